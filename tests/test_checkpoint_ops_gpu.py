"""ufp4_rms_norm and ufp4_glu, forward and backward, with their 8-bit
checkpoints, against the 64-bit formulas (tests/train_ref.py).

Tolerances.  bf16 outputs: half a unit in the last place of 8 significant
bits, 2^-8 relative, plus 2^-14 for the fp32 arithmetic in front of it; where terms cancel (dx, the
activations' derivatives) the fp32 part is relative to the terms.  dgamma is a
sum of `rows` fp32 products: (rows + 8) 2^-24 of the sum of magnitudes.  The
checkpoints and the bf16 sum are exact."""
import numpy as np
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests import train_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HALF = 2.0 ** -8, 2.0 ** -14
EPS = 1e-6


def _rand(rows, cols, seed, std=1.0, dtype=torch.bfloat16, ld=None, offset=0):
    """rows x cols on the GPU with leading dimension ld, starting `offset` elements into its storage; 1 in 500
    elements fifty times larger."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * std
    x = torch.where(torch.rand((rows, cols), generator=g) < 2e-3, 50 * x, x).to(dtype)
    return _placed(x, ld, offset)


def _placed(x, ld=None, offset=0):
    rows, cols = x.shape
    ld = cols if ld is None else ld
    buf = torch.zeros(offset + rows * ld + 16, dtype=x.dtype, device=DEV)
    out = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    out.copy_(x)
    return out


def _ckpt(rows, cols, codes_ld=None, scales_ld=None, offset=0):
    cl = cols if codes_ld is None else codes_ld
    nb = -(-cols // 32)
    sl = nb if scales_ld is None else scales_ld
    codes = torch.zeros(offset + rows * cl + 16, dtype=torch.uint8, device=DEV)[offset:offset + rows * cl].view(rows, cl)
    scales = torch.zeros((rows, sl), dtype=torch.uint8, device=DEV)
    return codes[:, :cols], scales[:, :nb], ufp4.QTensor(codes.data_ptr(), scales.data_ptr(), rows, cols, cl, sl)


def _near(got, want, terms=0.0, what="", rel=BF):
    got, want = got.double().cpu(), want.double().cpu()
    lim = (rel + HALF) * want.abs() + 2.0 ** -18 * (terms.cpu() if torch.is_tensor(terms) else terms) + 1e-30
    bad = ~((got - want).abs() <= lim) & ~(torch.isnan(got) & torch.isnan(want))
    assert not bad.any(), f"{what}: {int(bad.sum())} off, first {got[bad][0]} for {want[bad][0]}"


SHAPES = [(1, 1), (3, 7), (5, 31), (4, 32), (2, 33), (9, 64), (33, 100), (17, 264), (37, 1408), (260, 2048), (6, 5000),
          (3, 8200), (2, 16392), (2, 32768)]


# ------------------------------------------------------------------------- checkpoints
def _check_ckpt(codes, scales, v, what):
    c, s = ref.encode(v)
    assert torch.equal(scales.cpu(), s), f"{what}: scales"
    assert torch.equal(codes.cpu(), c), f"{what}: codes"


def test_checkpoint_of_every_scale_and_tie():
    """fp32 blocks over the whole exponent range, mantissas at and beside 1.75 (where the scale steps), exact ties of
    E4M3, subnormals, zeros and minus zeros."""
    rows = []
    for k in range(-149, 128):
        for f in (1.0, 1.75, float(np.nextafter(np.float32(1.75), np.float32(2))), 1.9999999):
            top = np.float32(min(f * 2.0 ** k, 3.4028234e38))
            t = np.concatenate([[1.0], (np.arange(1, 32) / 16.0) * 2.0 ** -(np.arange(31) % 12)]) * np.float64(top)
            t[1::2] *= -1
            rows.append(np.clip(t, -float(top), float(top)).astype(np.float32))
    rows.append(np.zeros(32, np.float32))
    rows.append(np.full(32, -0.0, np.float32))
    rows.append(np.array([448.0] + [(8 + i / 2) * 2.0 ** -6 for i in range(31)], np.float32))
    rows.append(np.array([448.0] + [-(i / 2) * 2.0 ** -9 for i in range(31)], np.float32))
    x = torch.from_numpy(np.stack(rows)).to(DEV)
    gc, gs, gq = _ckpt(*x.shape)
    uc, us, uq = _ckpt(*x.shape)
    ufp4.ufp4_glu(x, x, torch.empty_like(x, dtype=torch.bfloat16), ckpt_gate=gq, ckpt_up=uq)
    _check_ckpt(gc, gs, x, "gate")
    _check_ckpt(uc, us, x, "up")
    assert not (gc.cpu() == 0x80).any()


def test_checkpoint_reads_back_through_dequantize():
    """The checkpoint is an MXFP8 qtensor."""
    x = _rand(40, 256, 3)
    gc, gs, gq = _ckpt(40, 256)
    _, _, uq = _ckpt(40, 256)
    ufp4.ufp4_glu(x, x, torch.empty_like(x), ckpt_gate=gq, ckpt_up=uq)
    out = torch.empty((40, 256), device=DEV)
    desc = ufp4.make_desc(grid="mxfp8", block=(1, 32), n=1, scale_fmt=ufp4.SCALE_UE8M0)
    ufp4.ufp4_dequantize(gq, desc, False, out)
    assert torch.equal(out.double().cpu(), ref.decode(gc, gs))
    assert (out.double().cpu() - x.double().cpu()).abs().le(2.0 ** -4 * x.double().cpu().abs() +
                                                            2.0 ** -10 * ref.decode(gc, gs).abs().amax()).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("cols", [64, 70])
def test_nonfinite_blocks_read_back_as_nan(bad, cols):
    x = _rand(3, cols, 5, dtype=torch.float32)
    x[1, 40] = bad
    gc, gs, gq = _ckpt(3, cols)
    uc, us, uq = _ckpt(3, cols)
    ufp4.ufp4_glu(x, torch.ones_like(x), torch.empty_like(x, dtype=torch.bfloat16), ckpt_gate=gq, ckpt_up=uq)
    _check_ckpt(gc, gs, x, "gate")
    assert gs[1, 1] == 255 and (gc[1, 32:64] == 0x7F).all()
    dg, du, y = (torch.empty((3, cols), dtype=torch.bfloat16, device=DEV) for _ in range(3))
    ufp4.ufp4_glu_backward(torch.ones_like(x), gq, uq, dg, du, y=y)
    nan = torch.zeros((3, cols), dtype=torch.bool)
    nan[1, 32:64] = True
    for t in (dg, du, y):
        assert torch.equal(torch.isnan(t).cpu(), nan)
    # the norm's row is one sum: a NaN block takes its row (and every column of dgamma) with it, and no other row
    nc, ns, nq = _ckpt(3, cols)
    rstd, dgamma = torch.empty(3, device=DEV), torch.empty(cols, device=DEV)
    gamma = torch.ones(cols, device=DEV)
    ufp4.ufp4_rms_norm(x, gamma, y, rstd, ckpt=nq)
    _check_ckpt(nc, ns, x, "norm")
    ws = torch.empty(ufp4.ufp4_rms_norm_backward_workspace_size(3, cols), dtype=torch.uint8, device=DEV)
    ufp4.ufp4_rms_norm_backward(torch.ones_like(x), nq, torch.ones(3, device=DEV), gamma, dg, dgamma, ws)
    assert torch.isnan(dg[1]).all() and torch.isfinite(dg[0]).all() and torch.isfinite(dg[2]).all()
    assert torch.equal(torch.isnan(dgamma).cpu(), nan[1])


# --------------------------------------------------------------------------------- glu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_glu(shape, dtype, act):
    rows, cols = shape
    both = _rand(rows, 2 * cols, 7 + rows, dtype=dtype)
    gate, up = both[:, :cols], both[:, cols:]                # two halves of one output
    y = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    gc, gs, gq = _ckpt(rows, cols)
    uc, us, uq = _ckpt(rows, cols)
    ufp4.ufp4_glu(gate, up, y, act=act, ckpt_gate=gq, ckpt_up=uq)
    _near(y, ref.act(gate.double().cpu(), act)[0] * up.double().cpu(), what="y")
    _check_ckpt(gc, gs, gate, "gate")
    _check_ckpt(uc, us, up, "up")
    alone = torch.empty_like(y)
    ufp4.ufp4_glu(gate, up, alone, act=act)                  # without checkpoints
    assert torch.equal(alone, y)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_glu_backward(shape, dtype, act):
    rows, cols = shape
    gq = ref.encode(_rand(rows, cols, 11).float())
    uq = ref.encode(_rand(rows, cols, 12).float())
    g, u = ref.decode(*gq), ref.decode(*uq)
    dy = _rand(rows, cols, 13, 1e-3, dtype)
    keep = [t.to(DEV).contiguous() for t in (*gq, *uq)]
    both = torch.empty((rows, 2 * cols), dtype=torch.bfloat16, device=DEV)
    y = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    q = [ufp4.qtensor(keep[i], keep[i + 1], rows, cols) for i in (0, 2)]
    ufp4.ufp4_glu_backward(dy, *q, both[:, :cols], both[:, cols:], act=act, y=y)
    a, d = ref.act(g, act)
    d64 = dy.double().cpu()
    _near(both[:, cols:], d64 * a, what="dup")
    _near(both[:, :cols], d64 * u * d, terms=(d64 * u).abs(), what="dgate")
    _near(y, a * u, what="y")
    again = torch.empty_like(both)
    ufp4.ufp4_glu_backward(dy, *q, again[:, :cols], again[:, cols:], act=act)
    assert torch.equal(again, both)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_gradient_against_differences(act):
    """Central differences of the 64-bit forward along random directions; the step's own error is h^2 |f'''| / 6."""
    rows, cols = 8, 96
    gq = ref.encode(_rand(rows, cols, 21).clamp(-6, 6).float())
    uq = ref.encode(_rand(rows, cols, 22).clamp(-6, 6).float())
    g, u = ref.decode(*gq), ref.decode(*uq)
    dy = _rand(rows, cols, 23, dtype=torch.float32)
    keep = [t.to(DEV).contiguous() for t in (*gq, *uq)]
    dg, du = (torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ufp4.ufp4_glu_backward(dy, ufp4.qtensor(keep[0], keep[1], rows, cols), ufp4.qtensor(keep[2], keep[3], rows, cols), dg,
                           du, act=act)
    h = 1e-4
    d64 = dy.double().cpu()
    num_g = d64 * u * (ref.act(g + h, act)[0] - ref.act(g - h, act)[0]) / (2 * h)
    num_u = d64 * ref.act(g, act)[0] * ((u + h) - (u - h)) / (2 * h)
    _near(dg, num_g, terms=(d64 * u).abs(), what="dgate")
    _near(du, num_u, terms=d64.abs(), what="dup")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_extremes(act):
    """Saturated gates: exp overflows and underflows, g^2 overflows; nothing turns into NaN."""
    g = torch.tensor([[0.0, -0.0, 1e-30, -1e-30, 20, -20, 88.5, -88.5, 100, -100, 1e5, -1e5, 3e38, -3e38, 1e20, -1e20]],
                     device=DEV)
    u = torch.full_like(g, 0.5)
    y = torch.empty_like(g, dtype=torch.bfloat16)
    ufp4.ufp4_glu(g, u, y, act=act)
    _near(y, torch.nan_to_num(ref.act(g.double().cpu(), act)[0]) * 0.5, terms=1e-9, what="y")
    codes = torch.zeros((1, 16), dtype=torch.uint8, device=DEV)
    codes[0] = torch.tensor([0x00, 0x38, 0xB8, 0x7E, 0xFE, 0x50, 0xD0, 1, 0x81] + [0] * 7, dtype=torch.uint8)
    for byte in (0, 127, 190, 246):                          # units 2^-127, 1, 2^63, 2^119
        s = torch.full((1, 1), byte, dtype=torch.uint8, device=DEV)
        one = torch.full((1, 1), 127, dtype=torch.uint8, device=DEV)
        gq, uq = ufp4.qtensor(codes, s, 1, 16), ufp4.qtensor(codes, one, 1, 16)
        dg, du = torch.empty_like(y), torch.empty_like(y)
        ufp4.ufp4_glu_backward(u, gq, uq, dg, du, act=act)
        gv, uv = ref.decode(codes, s), ref.decode(codes, one)
        big = gv.abs() > 1e4                                  # there the formula is a step (g^3 may not be finite)
        a, d = ref.act(torch.where(big, torch.zeros_like(gv), gv), act)
        a = torch.where(big, gv.clamp_min(0), a)
        d = torch.where(big, (gv > 0).double(), d)
        _near(dg, 0.5 * uv * d, terms=uv.abs(), what=f"dgate {byte}")
        _near(du, 0.5 * a, terms=1e-9, what=f"dup {byte}")


# -------------------------------------------------------------------------------- norm
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_rms_norm(shape, dtype, residual):
    rows, cols = shape
    x = _rand(rows, cols, 31, dtype=dtype)
    r = _rand(rows, cols, 32, 2.0) if residual else None
    gamma = (1 + 0.1 * torch.randn(cols, generator=torch.Generator().manual_seed(1))).to(DEV)
    gamma = gamma if residual else gamma.bfloat16()
    y, total = (torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    rstd = torch.empty(rows, device=DEV)
    codes, scales, q = _ckpt(rows, cols)
    ufp4.ufp4_rms_norm(x, gamma, y, rstd, residual=r, total=total, ckpt=q, eps=EPS)
    s = x.float() + r.float() if residual else x.float()
    want, rs = ref.norm(s.cpu(), gamma.cpu(), EPS)
    _near(y, want, what="y")
    assert ((rstd.double().cpu() - rs).abs() <= 2.0 ** -20 * rs).all()
    assert torch.equal(total, s.bfloat16())
    _check_ckpt(codes, scales, s, "sum")
    alone = torch.empty_like(y)
    ufp4.ufp4_rms_norm(x, gamma, alone, residual=r, eps=EPS)  # only y
    assert torch.equal(alone, y)


def _norm_back(rows, cols, dtype, dtotal, remake, seed=41, **where):
    v = _rand(rows, cols, seed, 2.0).float()
    codes, scales = (t.to(DEV).contiguous() for t in ref.encode(v))
    s = ref.decode(codes, scales)
    rstd = (s.square().mean(1) + EPS).rsqrt().float()
    gamma = (1 + 0.1 * torch.randn(cols, generator=torch.Generator().manual_seed(2))).bfloat16()
    dy = _rand(rows, cols, seed + 1, 1e-3, dtype, **where)
    dt = _rand(rows, cols, seed + 2, 1e-3) if dtotal else None
    dx = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    y = torch.empty_like(dx) if remake else None
    dgamma = torch.full((cols,), 7.0, device=DEV)
    ws = torch.empty(max(1, ufp4.ufp4_rms_norm_backward_workspace_size(rows, cols)), dtype=torch.uint8, device=DEV)
    ufp4.ufp4_rms_norm_backward(dy, ufp4.qtensor(codes, scales, rows, cols), rstd.to(DEV), gamma.to(DEV), dx, dgamma, ws,
                                dtotal=dt, y=y)
    return s, rstd, gamma, dy, dt, dx, y, dgamma


@pytest.mark.parametrize("dtype,dtotal,remake", [(torch.bfloat16, False, False), (torch.bfloat16, True, True),
                                                 (torch.float32, True, False), (torch.float32, False, True)])
@pytest.mark.parametrize("shape", SHAPES + [(1500, 96), (700, 1000)])
def test_rms_norm_backward(shape, dtype, dtotal, remake):
    rows, cols = shape
    s, rstd, gamma, dy, dt, dx, y, dgamma = _norm_back(rows, cols, dtype, dtotal, remake)
    want, dg, yw = ref.norm_backward(s, rstd, gamma, dy.cpu())
    add = dt.double().cpu() if dtotal else torch.zeros_like(want)
    q, h = dy.double().cpu() * gamma.double(), s * rstd.double()[:, None]
    terms = rstd.double()[:, None] * (q.abs() + h.abs() * (q * h).abs().mean(1, keepdim=True)) + add.abs()
    _near(dx, want + add, terms=terms, what="dx")
    lim = (rows + 8) * 2.0 ** -24 * (dy.double().cpu() * h).abs().sum(0) + 1e-30
    assert ((dgamma.double().cpu() - dg).abs() <= lim).all()
    if remake:
        _near(y, yw, what="y")


def test_rms_norm_gradient_against_differences():
    """d(sum y * dy) along single elements of the row and of gamma, by central differences of the 64-bit forward."""
    rows, cols = 3, 40
    s, rstd, gamma, dy, _, dx, _, dgamma = _norm_back(rows, cols, torch.float32, False, False)
    h, d64 = 1e-4, dy.double().cpu()
    eps = EPS

    def f(t, g):
        return (ref.norm(t, g, eps)[0] * d64).sum()
    g64 = gamma.double()
    scale = (d64.abs().amax(1) * rstd.double()).max()
    for r in range(rows):
        for c in range(0, cols, 7):
            e = torch.zeros_like(s)
            e[r, c] = h
            num = (f(s + e, g64) - f(s - e, g64)) / (2 * h)
            assert abs(dx[r, c].double().cpu() - num) <= (BF + HALF) * abs(num) + 2e-5 * scale
    for c in range(0, cols, 7):
        e = torch.zeros_like(g64)
        e[c] = h
        num = (f(s, g64 + e) - f(s, g64 - e)) / (2 * h)
        assert abs(dgamma[c].double().cpu() - num) <= 1e-5 * (d64 * s * rstd.double()[:, None]).abs()[:, c].sum() + 1e-12


def test_rms_norm_without_rows():
    dgamma = torch.full((100,), 7.0, device=DEV)
    ws = torch.empty(ufp4.ufp4_rms_norm_backward_workspace_size(0, 100), dtype=torch.uint8, device=DEV)
    e = torch.empty((0, 100), dtype=torch.bfloat16, device=DEV)
    ufp4.ufp4_rms_norm_backward(e, ufp4.QTensor(None, None, 0, 100, 100, 4), torch.empty(0, device=DEV),
                                torch.ones(100, device=DEV), e, dgamma, ws)
    assert (dgamma == 0).all()
    ufp4.ufp4_rms_norm(e, torch.ones(100, device=DEV), e)
    ufp4.ufp4_glu(e, e, e)


def test_zero_rows_stay_finite():
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV)
    y, rstd = torch.empty_like(x), torch.empty(2, device=DEV)
    codes, scales, q = _ckpt(2, 64)
    ufp4.ufp4_rms_norm(x, torch.ones(64, device=DEV), y, rstd, ckpt=q, eps=1e-6)
    assert (y == 0).all() and (codes == 0).all() and (scales == 0).all()
    assert ((rstd - 1e3).abs() <= 1e3 * 2.0 ** -20).all()


# ------------------------------------------------------- strides, guards, streams, order
@pytest.mark.parametrize("cols,ld,offset", [(64, 72, 0), (64, 65, 0), (64, 64, 1), (96, 104, 3), (70, 71, 1), (1408, 1411, 5)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_and_unaligned_operands(cols, ld, offset, dtype):
    """Any row pitch and element alignment gives what contiguous operands give, and nothing outside the rows is written."""
    rows = 13
    gate, up = _rand(rows, cols, 51, dtype=dtype), _rand(rows, cols, 52, dtype=dtype)
    gamma = 1 + 0.1 * _rand(1, cols, 53, dtype=torch.float32)[0]
    dy = _rand(rows, cols, 54, dtype=dtype)

    def run(place, out):
        y, t, dg, du, yy, dx, ny = (out() for _ in range(7))
        ck = [_ckpt(rows, cols, *(() if place is None else (cols + 3, (cols + 31) // 32 + 2, offset))) for _ in range(3)]
        p = (lambda v: v) if place is None else place
        gm = gamma if place is None else _placed(gamma[None], None, offset)[0]
        rstd, dgamma = torch.empty(rows, device=DEV), torch.empty(cols, device=DEV)
        ws = torch.empty(ufp4.ufp4_rms_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=DEV)
        ufp4.ufp4_glu(p(gate), p(up), y, ckpt_gate=ck[0][2], ckpt_up=ck[1][2])
        ufp4.ufp4_glu_backward(p(dy), ck[0][2], ck[1][2], dg, du, y=yy)
        res = p(_rand(rows, cols, 55))
        ufp4.ufp4_rms_norm(p(gate), gm, ny, rstd, residual=res, total=t, ckpt=ck[2][2])
        ufp4.ufp4_rms_norm_backward(p(dy), ck[2][2], rstd, gm, dx, dgamma, ws, dtotal=res)
        return [y, t, dg, du, yy, dx, ny, rstd, dgamma] + [v for c in ck for v in c[:2]]

    bufs = []

    def guarded():
        buf = torch.full((offset + rows * ld + 64,), 3.0, dtype=torch.bfloat16, device=DEV)
        bufs.append(buf)
        return buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]

    plain = run(None, lambda: torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV))
    moved = run(lambda v: _placed(v, ld, offset), guarded)
    for i, (a, b) in enumerate(zip(plain, moved)):
        if i in (5, 7, 8, 6):   # a vector and a scalar path may order a row's sum differently: same bound as the formula
            assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-6)
        else:
            assert torch.equal(a, b), i
    for buf in bufs:
        body = buf[offset:offset + rows * ld].view(rows, ld)
        assert (buf[:offset] == 3).all() and (buf[offset + rows * ld:] == 3).all() and (body[:, cols:] == 3).all()


def test_runs_are_reproducible_and_follow_their_stream():
    rows, cols = 3000, 1000
    v = _rand(rows, cols, 61, dtype=torch.float32)
    side = torch.cuda.Stream()
    outs = []
    for i in range(3):
        big = torch.randn((4096, 4096), device=DEV)
        with torch.cuda.stream(side if i else torch.cuda.current_stream()):
            side.wait_stream(torch.cuda.default_stream())
            x = torch.zeros_like(v)
            for _ in range(4):
                big = big @ big * 1e-3                        # work in front on the same stream
            x.copy_(v)
            y, dx = (torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV) for _ in range(2))
            rstd, dgamma = torch.empty(rows, device=DEV), torch.empty(cols, device=DEV)
            _, _, q = ck = _ckpt(rows, cols)
            ws = torch.empty(ufp4.ufp4_rms_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=DEV)
            ufp4.ufp4_rms_norm(x, torch.ones(cols, device=DEV), y, rstd, ckpt=q)
            ufp4.ufp4_rms_norm_backward(y, q, rstd, torch.ones(cols, device=DEV), dx, dgamma, ws)
            outs.append([t.clone() for t in (y, dx, rstd, dgamma, ck[0], ck[1])])
        torch.cuda.synchronize()
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_operators_in_a_graph():
    """Captured and replayed on new inputs."""
    rows, cols = 64, 512
    x = _rand(rows, cols, 71)
    gamma = torch.ones(cols, device=DEV)
    y, rstd = torch.empty_like(x), torch.empty(rows, device=DEV)
    g = torch.empty_like(x)
    ufp4.ufp4_rms_norm(x, gamma, y, rstd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ufp4.ufp4_rms_norm(x, gamma, y, rstd)
        ufp4.ufp4_glu(y, y, g)
    x.copy_(_rand(rows, cols, 72))
    graph.replay()
    torch.cuda.synchronize()
    want, want_g = torch.empty_like(x), torch.empty_like(x)
    ufp4.ufp4_rms_norm(x, gamma, want)
    ufp4.ufp4_glu(want, want, want_g)
    assert torch.equal(y, want) and torch.equal(g, want_g)
