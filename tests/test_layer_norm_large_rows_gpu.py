"""Gradients of the layer norm at constant rows of large elements (the mean times rstd is beyond fp32): h is 0 there, whether or not
a row is a whole number of lanes' elements.  Bounds of test_layer_norm_gpu."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests.test_layer_norm_gpu import _check_backward, _rows, _weights, EPS

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32


# copied rows of one, two and four steps a lane, rows read in place, sums by the columns' kernel
@pytest.mark.parametrize("cols", [5, 101, 104, 1027, 4999, 8193, 9001, 16383, 20001])
@pytest.mark.parametrize("dtype,xtype", [(BF, BF), (F, BF), (BF, F), (F, F)])
def test_large_constant_rows(cols, dtype, xtype):
    rows = 9
    x = torch.tensor([3e36, -3e36, 1e37, 3e38, -3e38, 2.0, 0.0, 1e30, 7e36]).to(DEV, xtype)[:, None].expand(-1, cols).contiguous()
    mean, rstd = x[:, 0].float().contiguous(), torch.full((rows,), EPS ** -0.5, device=DEV)
    dy = _rows(rows, cols, 101, dtype, std=1e-3)
    gamma, _ = _weights(cols, 102, F)
    dx, dg, db = torch.empty((rows, cols), dtype=BF, device=DEV), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.empty(ufp4.ufp4_layer_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=DEV)
    ufp4.ufp4_layer_norm_backward(dy, x, mean, rstd, gamma, dx, dg, db, ws)
    assert (dg == 0).all()
    _check_backward(x, dy, mean, rstd, gamma, None, dx, dg, db)
