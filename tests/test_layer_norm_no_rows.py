"""Refusals of ufp4_layer_norm_backward on no rows: dgamma and dbeta are written then too, by a kernel that loads gamma (no GPU
needed, the addresses are made up)."""
import ctypes

import pytest

from rht_bit_block_gb300 import build, ufp4

P = ctypes.c_void_p


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return ufp4.load()


# one, two and four steps a lane, and rows whose sums are a kernel's of their own
@pytest.mark.parametrize("cols", [1, 96, 7168, 9000, 20000])
@pytest.mark.parametrize("gamma,gtype,status", [(0, 0, 1), (0, 1, 1), (0x5001, 0, 3), (0x5002, 1, 3)])
def test_gamma_is_checked_without_rows(lib, cols, gamma, gtype, status):
    got = lib.ufp4_layer_norm_backward(P(0), 0, 0, P(0), 0, 0, P(0), P(0), P(gamma), gtype, P(0), 0, 0, cols, P(0), 0, P(0x7000),
                                       P(0x40000), P(0x80000), 1 << 26, None)
    assert got == status
