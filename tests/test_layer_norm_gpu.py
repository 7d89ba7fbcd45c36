"""ufp4_layer_norm and its gradients against the 64-bit formulas (tests/fp8_ref.py).

Tolerances, u = 2^-24.  A row's mean is a sum of up to 32 + 15 additions in sequence (32 elements a lane, then the lanes and
warps by halves): 64 u of the mean of magnitudes, A.  The variance is a mean of squares about that mean: another 64 u of
itself, and what the mean's error adds is of second order or 2 * 64 u A times the mean difference, 0.  rsqrtf is good to 2
ulp.  h = (s - m) r is then off by 64 u A r and 70 u |h|.  bf16 outputs add half a step, 2^-8 of themselves.  dgamma and
dbeta are sums of `rows` fp32 products: (rows + 70) u of the sums of magnitudes, and the given mean and rstd are the
forward's own."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests import fp8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, BF = 2.0 ** -24, 2.0 ** -8
EPS = 1e-5

SHAPES = [(1, 1), (3, 7), (5, 31), (4, 32), (9, 64), (33, 100), (2, 256), (17, 264), (7, 520), (37, 1408), (260, 2048),
          (2000, 128), (6, 5000), (3, 8192), (5, 8200), (2, 16384), (2, 16392), (3, 32768), (2, 20001)]


def _placed(x, ld=None, offset=0):
    rows, cols = x.shape
    ld = cols if ld is None else ld
    buf = torch.zeros(offset + rows * ld + 16, dtype=x.dtype, device=DEV)
    out = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    out.copy_(x)
    return out


def _rows(rows, cols, seed, dtype, shift=0.0, std=1.0, ld=None, offset=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * std
    x = torch.where(torch.rand((rows, cols), generator=g) < 2e-3, 50 * x, x) + shift * torch.randn((rows, 1), generator=g)
    return _placed(x.to(dtype), ld, offset)


def _weights(cols, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.1 * torch.randn(cols, generator=g)).to(DEV, dtype), (0.3 * torch.randn(cols, generator=g)).to(DEV, dtype)


def _within(got, want, lim, what):
    got, want = got.double().cpu(), want.double().cpu()
    bad = ~((got - want).abs() <= lim.double().cpu() + 1e-30)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, first {got[bad][0]} for {want[bad][0]}"


def _check_forward(x, residual, gamma, beta, y, total, mean, rstd):
    s = x.float()
    if residual is not None:
        s = s + residual.float()                  # an fp32 value by definition
    wy, wm, wr = ref.layer_norm(s, gamma, beta, EPS)
    s64 = s.double().cpu()
    big = s64.abs().mean(1)
    _within(mean, wm, 64 * U * big, "mean")
    _within(rstd, wr, wr * (100 * U + (64 * U * big * wr) ** 2), "rstd")
    if total is not None:
        assert torch.equal(total, s.bfloat16())
    w = gamma.double().cpu().abs()
    h = (wy - (0 if beta is None else beta.double().cpu())).abs()
    lim = 64 * U * (big * wr)[:, None] * w + 180 * U * h + BF * wy.abs() * (1 + 2.0 ** -8)
    _within(y, wy, lim * (1 + 2.0 ** -7), "y")


@pytest.mark.parametrize("parts", ["all", "plain"])
@pytest.mark.parametrize("wtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype, wtype, parts):
    rows, cols = shape
    x = _rows(rows, cols, 3 + rows, dtype, shift=2.0)
    gamma, beta = _weights(cols, 4, wtype)
    y = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    if parts == "all":
        residual, total = _rows(rows, cols, 5, torch.bfloat16), torch.empty_like(y)
        ufp4.ufp4_layer_norm(x, gamma, y, mean, rstd, beta=beta, residual=residual, total=total, eps=EPS)
        _check_forward(x, residual, gamma, beta, y, total, mean, rstd)
    else:
        ufp4.ufp4_layer_norm(x, gamma, y, mean, rstd, eps=EPS)
        _check_forward(x, None, gamma, None, y, None, mean, rstd)
        again = torch.empty_like(y)
        ufp4.ufp4_layer_norm(x, gamma, again, eps=EPS)            # statistics are optional
        assert torch.equal(again, y)


def test_rows_far_from_zero():
    """A mean of 1000 standard deviations: the mean square minus the squared mean would have no digit left."""
    g = torch.Generator().manual_seed(1)
    x = (torch.randn((50, 2048), generator=g) + 1000 * torch.randn((50, 1), generator=g)).to(DEV)
    gamma, beta = _weights(2048, 4, torch.float32)
    y, mean, rstd = torch.empty(x.shape, dtype=torch.bfloat16, device=DEV), torch.empty(50, device=DEV), torch.empty(50, device=DEV)
    ufp4.ufp4_layer_norm(x, gamma, y, mean, rstd, beta=beta, eps=EPS)
    _check_forward(x, None, gamma, beta, y, None, mean, rstd)


def test_constant_and_nonfinite_rows():
    x = torch.ones((6, 300), device=DEV)
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 299] = float("inf")
    x[5] = torch.randn(300, device=DEV)
    gamma, beta = _weights(300, 4, torch.float32)
    y, mean, rstd = torch.empty(x.shape, dtype=torch.bfloat16, device=DEV), torch.empty(6, device=DEV), torch.empty(6, device=DEV)
    ufp4.ufp4_layer_norm(x, gamma, y, mean, rstd, beta=beta, eps=EPS)
    assert torch.equal(y[0], beta.bfloat16()) and torch.equal(y[1], beta.bfloat16()) and torch.equal(y[4], y[0])
    assert torch.isnan(y[2:4]).all() and torch.isfinite(y[5]).all()
    assert (rstd[:2] - EPS ** -0.5).abs().max() < 1e-3
    # backward: such rows' dx is NaN, and so is dgamma; dbeta is not
    dx, dg, db = torch.empty_like(y), torch.empty(300, device=DEV), torch.empty(300, device=DEV)
    ws = torch.empty(ufp4.ufp4_layer_norm_backward_workspace_size(6, 300), dtype=torch.uint8, device=DEV)
    ufp4.ufp4_layer_norm_backward(torch.ones_like(x), x, mean, rstd, gamma, dx, dg, db, ws)
    assert torch.isnan(dx[2:4]).all() and torch.isfinite(dx[[0, 1, 4, 5]]).all()
    assert torch.isnan(dg).all() and (db == 6).all()


def _check_backward(x, dy, mean, rstd, gamma, dtotal, dx, dg, db):
    rows, cols = x.shape
    wdx, wdg, wdb, h, q = ref.layer_norm_backward(x, mean, rstd, gamma, dy)
    r = rstd.double().cpu()[:, None]
    terms = r * (q.abs() + q.abs().mean(1, keepdim=True) + h.abs() * (q * h).abs().mean(1, keepdim=True))
    if dtotal is not None:
        wdx = wdx + dtotal.double().cpu()
        terms = terms + dtotal.double().cpu().abs()
    # (s - m) of the given mean is one rounding of s - m; h has two, q one, the sums 64 and the result four more
    _within(dx, wdx, 80 * U * terms + BF * wdx.abs() * (1 + 2.0 ** -8), "dx")
    d = dy.double().cpu().abs()
    _within(dg, wdg, (rows + 70) * U * (d * h.abs()).sum(0), "dgamma")
    _within(db, wdb, (rows + 70) * U * d.sum(0), "dbeta")


def _backward(x, dy, gamma, dtotal, beta=None):
    rows, cols = x.shape
    y, mean, rstd = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ufp4.ufp4_layer_norm(x, gamma, y, mean, rstd, eps=EPS)
    dx, dg, db = torch.empty_like(y), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    need = ufp4.ufp4_layer_norm_backward_workspace_size(rows, cols)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=DEV)      # NaN patterns
    ufp4.ufp4_layer_norm_backward(dy, x, mean, rstd, gamma, dx, dg, db, ws[:need], dtotal=dtotal)
    assert (ws[need:] == 0xFF).all()
    return mean, rstd, dx, dg, db


@pytest.mark.parametrize("dtotal", [True, False])
@pytest.mark.parametrize("xtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dtype, xtype, dtotal):
    rows, cols = shape
    x, dy = _rows(rows, cols, 7, xtype, shift=2.0), _rows(rows, cols, 8, dtype, std=1e-3)
    gamma, _ = _weights(cols, 9, torch.bfloat16 if dtotal else torch.float32)
    add = _rows(rows, cols, 10, torch.bfloat16, std=1e-3) if dtotal else None
    mean, rstd, dx, dg, db = _backward(x, dy, gamma, add)
    _check_backward(x, dy, mean, rstd, gamma, add, dx, dg, db)
    again = _backward(x, dy, gamma, add)
    assert all(torch.equal(a, b) for a, b in zip(again, (mean, rstd, dx, dg, db)))


@pytest.mark.parametrize("ld,offset", [(None, 1), (301, 0), (304, 8), (320, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pitches_and_offsets(dtype, ld, offset):
    rows, cols = 50, 296
    x, dy = _rows(rows, cols, 11, dtype, ld=ld, offset=offset), _rows(rows, cols, 12, dtype, 1e-3, ld=ld, offset=offset)
    residual = _rows(rows, cols, 13, torch.bfloat16, ld=ld, offset=offset)
    gamma, beta = _weights(cols, 14, torch.float32)
    y, total, dx = (_placed(torch.full((rows, cols), 9.0, dtype=torch.bfloat16), ld, offset) for _ in range(3))
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ufp4.ufp4_layer_norm(x, gamma, y, mean, rstd, beta=beta, residual=residual, total=total, eps=EPS)
    _check_forward(x, residual, gamma, beta, y, total, mean, rstd)
    dg, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.empty(ufp4.ufp4_layer_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=DEV)
    ufp4.ufp4_layer_norm_backward(dy, total, mean, rstd, gamma, dx, dg, db, ws, dtotal=residual)
    _check_backward(total, dy, mean, rstd, gamma, residual, dx, dg, db)


def test_gradient_against_differences():
    """Central differences of the 64-bit forward along random directions, with the kernel's own gradients; the
    difference itself is good to h^2."""
    rows, cols, h = 6, 264, 1e-4
    x, dy = _rows(rows, cols, 21, torch.float32, shift=1.0), _rows(rows, cols, 22, torch.float32)
    gamma, beta = _weights(cols, 23, torch.float32)
    mean, rstd, dx, dg, db = _backward(x, dy, gamma, None)
    g = torch.Generator().manual_seed(24)
    d64, x64, w64, b64 = (t.double().cpu() for t in (dy, x, gamma, beta))
    for _ in range(4):
        vx, vg, vb = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((rows, cols), (cols,), (cols,)))

        def loss(e):
            return float((d64 * ref.layer_norm(x64 + e * vx, w64 + e * vg, b64 + e * vb, EPS)[0]).sum())
        num = (loss(h) - loss(-h)) / (2 * h)
        parts = [(dx.double().cpu() * vx), (dg.double().cpu() * vg), (db.double().cpu() * vb)]
        size = float(sum(p.abs().sum() for p in parts))
        # bf16 dx: half a step an element, random signs do not matter to the bound
        assert abs(float(sum(p.sum() for p in parts)) - num) <= BF * size + 1e-5 * size


@pytest.mark.parametrize("cols", [96, 101, 2048, 9000, 16384, 20000])
def test_results_in_place_of_operands(cols):
    """y over x, total over residual; dx over dy, over x and over dtotal."""
    rows = 40
    x, residual = _rows(rows, cols, 61, torch.bfloat16, shift=1.0), _rows(rows, cols, 62, torch.bfloat16)
    dy, dtotal = _rows(rows, cols, 63, torch.bfloat16), _rows(rows, cols, 64, torch.bfloat16)
    gamma, beta = _weights(cols, 65, torch.bfloat16)
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
        got = [dx, dg, db]
        want = got if want is None else want
        assert all(torch.equal(a, b) for a, b in zip(got, want)), place


def test_no_rows():
    x = torch.empty((0, 100), device=DEV)
    gamma, _ = _weights(100, 4, torch.float32)
    dg, db = torch.full((100,), 5.0, device=DEV), torch.full((100,), 5.0, device=DEV)
    for cols in (100,):
        ws = torch.empty(ufp4.ufp4_layer_norm_backward_workspace_size(0, cols), dtype=torch.uint8, device=DEV)
        none = torch.empty(0, device=DEV)
        y = torch.empty((0, cols), dtype=torch.bfloat16, device=DEV)
        ufp4.ufp4_layer_norm(x, gamma, y, none, none)
        ufp4.ufp4_layer_norm_backward(x, x, none, none, gamma, y, dg, db, ws)
        assert (dg == 0).all() and (db == 0).all()
    wide = 20000
    dg, db = torch.full((wide,), 5.0, device=DEV), torch.full((wide,), 5.0, device=DEV)
    ws = torch.empty(ufp4.ufp4_layer_norm_backward_workspace_size(0, wide), dtype=torch.uint8, device=DEV)
    x, y = torch.empty((0, wide), device=DEV), torch.empty((0, wide), dtype=torch.bfloat16, device=DEV)
    ufp4.ufp4_layer_norm_backward(x, x, torch.empty(0, device=DEV), torch.empty(0, device=DEV),
                                  torch.ones(wide, device=DEV), y, dg, db, ws)
    assert (dg == 0).all() and (db == 0).all()


def test_streams_and_captured_graphs():
    """Two captured backward passes, each with its workspace, replayed at once on two streams."""
    cases = []
    for i, (rows, cols) in enumerate(((700, 2048), (333, 1408))):
        x, dy = _rows(rows, cols, 31 + i, torch.bfloat16), _rows(rows, cols, 41 + i, torch.bfloat16, std=1e-3)
        gamma, _ = _weights(cols, 51, torch.bfloat16)
        mean, rstd, dx, dg, db = _backward(x, dy, gamma, None)
        ws = torch.empty(ufp4.ufp4_layer_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=DEV)
        got = [torch.empty_like(t) for t in (dx, dg, db)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ufp4.ufp4_layer_norm_backward(dy, x, mean, rstd, gamma, *got, ws)
        cases.append((graph, got, (dx, dg, db), (x, dy, gamma, mean, rstd, ws)))  # a graph's operands stay alive
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        for st, (graph, *_) in zip(streams, cases):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for _, got, want, _ in cases:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
