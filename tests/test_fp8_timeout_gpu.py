"""The 8-bit product's bounded waits, without a GPU fault: ufp4_set_quantize_wait_limit(0) makes the first wait for a stage
of every cluster give up at once, with copies in flight into its shared memory.  The kernel records it, lets the copies
land and returns; ufp4_device_error reports it, and the next call gives what it gave before."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests.test_fp8_gemm_gpu import make

pytestmark = pytest.mark.gpu
DEV = "cuda"


# single CTAs and shares of each width, pairs, pairs with several tiles a cluster
@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (3, 2048, 1024), (30, 700, 4096), (60, 700, 4096), (200, 700, 4096),
                                   (2304, 2304, 512), (6000, 5000, 256)])
def test_a_wait_that_gives_up_is_reported_and_the_next_call_is_right(m, n, k):
    a, b = make(m, k, 1, 1), make(n, k, 128, 2)
    d = torch.empty((m, n), device=DEV)

    def call():
        ufp4.ufp4_fp8_gemm(a[2], b[2], d)
    call()
    torch.cuda.synchronize()
    assert ufp4.ufp4_device_error() == 0
    want = d.clone()
    ufp4.ufp4_set_quantize_wait_limit(0)
    try:
        call()
        torch.cuda.synchronize()
        assert ufp4.ufp4_device_error_status() == ufp4.UFP4_ERR_TIMEOUT
        assert ufp4.ufp4_device_error() == 0   # the read cleared it
    finally:
        ufp4.ufp4_set_quantize_wait_limit(-1)
    call()
    torch.cuda.synchronize()
    assert ufp4.ufp4_device_error() == 0
    assert torch.equal(d, want)
