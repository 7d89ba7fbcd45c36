"""Layer norm and its gradients with several rows for every CTA and group: the next row copied ahead, a shift that differs from row
to row, the backward pass's two buffers in turn and its sums over rows.  Bounds of test_layer_norm_gpu."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests.test_layer_norm_gpu import _check_backward, _check_forward, _rows, _weights, EPS
from tests.test_layer_norm_rows_gpu import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32
ODD = [1, 127, 1027, 4999, 8193, 12289, 20001]
EVEN = [128, 2048, 5000, 8200, 16384, 16392, 32768]


def _count(cols):
    """Rows enough for three a CTA of the forward pass, which has up to 32 on an SM, 1024 threads and no fewer than 512 columns a
    warp, and for more of the backward pass."""
    warps = -(-cols // 512)
    return 3 * torch.cuda.get_device_properties(0).multi_processor_count * max(1, min(32, 32 // warps)) + 5


def _check(cols, dtype, xtype, lds):
    """lds: what the leading dimensions of x, residual, dy, dtotal, y, total and dx have beyond cols."""
    rows = _count(cols)
    x = _rows(rows, cols, 91, xtype, shift=2.0, ld=cols + lds[0], offset=lds[0])
    residual = _rows(rows, cols, 92, BF, ld=cols + lds[1], offset=lds[1])
    dy = _rows(rows, cols, 93, dtype, std=1e-3, ld=cols + lds[2], offset=lds[2])
    dtotal = _rows(rows, cols, 94, BF, std=1e-3, ld=cols + lds[3], offset=lds[3])
    y, total, dx = (Guarded(rows, cols, cols + n, n) for n in lds[4:])
    gamma, beta = _weights(cols, 95, F)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ufp4.ufp4_layer_norm(x, gamma, y.m, mean, rstd, beta=beta, residual=residual, total=total.m, eps=EPS)
    _check_forward(x, residual, gamma, beta, y.m, total.m, mean, rstd)
    ufp4.ufp4_layer_norm(x, gamma, y.m, mean, rstd, eps=EPS)
    _check_forward(x, None, gamma, None, y.m, None, mean, rstd)
    dg, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.full((ufp4.ufp4_layer_norm_backward_workspace_size(rows, cols),), 0xFF, dtype=torch.uint8, device=DEV)
    ufp4.ufp4_layer_norm_backward(dy, x, mean, rstd, gamma, dx.m, dg, db, ws, dtotal=dtotal)
    _check_backward(x, dy, mean, rstd, gamma, dtotal, dx.m, dg, db)
    ufp4.ufp4_layer_norm_backward(dy, x, mean, rstd, gamma, dx.m, dg, db, ws)
    _check_backward(x, dy, mean, rstd, gamma, None, dx.m, dg, db)
    for t in (y, total, dx):
        t.check()


@pytest.mark.parametrize("dtype,xtype", [(BF, BF), (F, BF), (BF, F), (F, F)])
@pytest.mark.parametrize("cols", ODD)
def test_rows_that_start_anywhere(cols, dtype, xtype):
    _check(cols, dtype, xtype, (2, 5, 0, 1, 3, 1, 0))  # even and odd distances: shifts that change from row to row


@pytest.mark.parametrize("dtype,xtype", [(BF, BF), (F, F)])
@pytest.mark.parametrize("cols", EVEN)
def test_aligned_rows(cols, dtype, xtype):
    _check(cols, dtype, xtype, (8, 0, 16, 0, 24, 8, 0))


@pytest.mark.parametrize("cols", [127, 1027, 2048, 4999, 8193, 16384, 20001])
def test_results_in_place_of_operands(cols):
    """Rows side by side: what one CTA copies ahead holds the ends of rows that others write."""
    rows = _count(cols)
    x, residual = _rows(rows, cols, 96, BF, shift=1.0), _rows(rows, cols, 97, BF)
    dy, dtotal = _rows(rows, cols, 98, BF), _rows(rows, cols, 99, BF)
    gamma, beta = _weights(cols, 65, BF)
    y, total = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ufp4.ufp4_layer_norm(x, gamma, y, mean, rstd, beta=beta, residual=residual, total=total, eps=EPS)
    x2, residual2 = x.clone(), residual.clone()
    ufp4.ufp4_layer_norm(x2, gamma, x2, beta=beta, residual=residual2, total=residual2, eps=EPS)
    assert torch.equal(x2, y) and torch.equal(residual2, total)
    ws = torch.empty(ufp4.ufp4_layer_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=DEV)
    want = None
    for place in (None, 0, 1, 2):
        ops = [t.clone() for t in (dy, total, dtotal)]
        dx = torch.empty_like(x) if place is None else ops[place]
        dg, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
        ufp4.ufp4_layer_norm_backward(ops[0], ops[1], mean, rstd, gamma, dx, dg, db, ws, dtotal=ops[2])
        want = [dx, dg, db] if want is None else want
        assert all(torch.equal(a, b) for a, b in zip((dx, dg, db), want)), place
