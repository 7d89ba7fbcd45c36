"""ufp4_layer_norm and its gradients where every matrix starts and steps differently, none by whole vectors: results as everywhere
(bounds of test_layer_norm_gpu), and nothing written beside the rows."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests.test_layer_norm_gpu import _check_backward, _check_forward, _rows, _weights, EPS

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32


class Guarded:
    """A rows x cols bf16 matrix within a buffer of 9s."""

    def __init__(self, rows, cols, ld, offset):
        self.buf = torch.full((offset + rows * ld + 24,), 9.0, dtype=BF, device=DEV)
        self.m = self.buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]

    def check(self):
        left = self.buf.clone()
        off, (rows, cols), ld = self.m.storage_offset(), self.m.shape, self.m.stride(0)
        left[off:off + rows * ld].view(rows, ld)[:, :cols] = 9.0
        assert (left == 9).all()


@pytest.mark.parametrize("cols", [1, 5, 8, 255, 257, 511, 513, 1027, 4097, 8191, 8193, 9001, 12287, 16383, 17001])
@pytest.mark.parametrize("dtype,xtype", [(BF, BF), (F, BF), (BF, F), (F, F)])
def test_rows_that_start_anywhere(cols, dtype, xtype):
    rows = 11
    x = _rows(rows, cols, 81, xtype, shift=2.0, ld=cols + 2, offset=1)
    residual = _rows(rows, cols, 82, BF, ld=cols + 5, offset=3)
    dy = _rows(rows, cols, 83, dtype, std=1e-3, ld=cols, offset=5)
    dtotal = _rows(rows, cols, 84, BF, std=1e-3, ld=cols + 1, offset=2)
    gamma, beta = _weights(cols + 1, 85, F)
    gamma, beta = gamma[1:], beta[1:]
    y, total, dx = Guarded(rows, cols, cols + 3, 7), Guarded(rows, cols, cols + 1, 2), Guarded(rows, cols, cols, 9)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ufp4.ufp4_layer_norm(x, gamma, y.m, mean, rstd, beta=beta, residual=residual, total=total.m, eps=EPS)
    _check_forward(x, residual, gamma, beta, y.m, total.m, mean, rstd)
    dg, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.empty(ufp4.ufp4_layer_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=DEV)
    ufp4.ufp4_layer_norm(x, gamma, y.m, mean, rstd, beta=beta, eps=EPS)
    _check_forward(x, None, gamma, beta, y.m, None, mean, rstd)
    ufp4.ufp4_layer_norm_backward(dy, x, mean, rstd, gamma, dx.m, dg, db, ws, dtotal=dtotal)
    _check_backward(x, dy, mean, rstd, gamma, dtotal, dx.m, dg, db)
    for t in (y, total, dx):
        t.check()


@pytest.mark.parametrize("cols", [3, 101, 517, 5001])
def test_same_bits_wherever_the_rows_lie(cols):
    """Where a row starts changes neither the order of a sum nor a rounding."""
    x, dy = _rows(40, cols, 86, BF), _rows(40, cols, 87, BF, std=1e-3)
    gamma, beta = _weights(cols, 88, BF)
    seen = []
    for off in range(8):
        def at(t):
            buf = torch.empty(off + 40 * cols, dtype=BF, device=DEV)
            out = buf[off:].view(40, cols)
            return out.copy_(t)
        mx, mdy, y, dx = at(x), at(dy), at(x), at(x)
        mean, rstd, dg, db = (torch.empty(n, device=DEV) for n in (40, 40, cols, cols))
        ws = torch.empty(ufp4.ufp4_layer_norm_backward_workspace_size(40, cols), dtype=torch.uint8, device=DEV)
        ufp4.ufp4_layer_norm(mx, gamma, y, mean, rstd, beta=beta, eps=EPS)
        ufp4.ufp4_layer_norm_backward(mdy, mx, mean, rstd, gamma, dx, dg, db, ws)
        seen.append((y, mean, rstd, dx, dg, db))
    for other in seen[1:]:
        assert all(torch.equal(p, q) for p, q in zip(other, seen[0]))
