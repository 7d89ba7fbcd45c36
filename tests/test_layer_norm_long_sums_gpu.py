"""dgamma and dbeta of rows above 16384 columns over many rows.  Every column of dy is one number, whose repeated fp32 addition
rounds the same way each time.

Tolerance, u = 2^-24.  A thread adds 256 rows at most; the shares' sums are added 32 apart and the 32 sums by halves, rows / 256 /
32 + 5 additions; a product and its factors round three times.  That many u of the sum of magnitudes; one chain of 2222 rows, an
eighteenth of 40000, is off by up to 550 u."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("rows,cols", [(40000, 16400), (40001, 16401), (20000, 32768)])
def test_sums_over_many_rows(rows, cols):
    g = torch.Generator().manual_seed(5)
    c = (0.1 + torch.rand(cols, generator=g)).to(DEV)
    dy = c.expand(rows, cols).contiguous()
    x = torch.ones((rows, cols), dtype=torch.bfloat16, device=DEV)
    mean, rstd = torch.zeros(rows, device=DEV), torch.ones(rows, device=DEV)  # h is 1
    gamma = torch.ones(cols, device=DEV)
    dx, dg, db = torch.empty_like(x), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.empty(ufp4.ufp4_layer_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=DEV)
    ufp4.ufp4_layer_norm_backward(dy, x, mean, rstd, gamma, dx, dg, db, ws)
    want = rows * c.double()
    for name, got in (("dgamma", dg), ("dbeta", db)):
        off = float(((got.double() - want) / want).abs().max()) * 2 ** 24
        assert off <= 256 + rows / 256 / 32 + 10, f"{name}: {off} u"
