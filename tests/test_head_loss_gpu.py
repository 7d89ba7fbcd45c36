"""ufp4_head_loss and ufp4_head_loss_backward against the 64-bit formulas
(tests/train_ref.py), on the GPU.

Tolerances.  Logits are fp32 sums of exact bf16 products: 2^-19 of the largest
sum of magnitudes |h| |w|, plus 2^-20 of the result for the exponentials and
the logarithm.  dl is rounded to bf16 (8 significant bits: 2^-8 relative)
before it multiplies, so an entry of dh is within 2^-8 (1 + 2^-4) of sum |dl|
|w| (the 2^-4: the logits' error and the fp32 sums), plus 2^-8 of itself where
it is bf16; dw likewise.  Over many entries either rounding has a relative
2-norm of 2^-8 / sqrt(3 * 7/3) = 0.38 * 2^-8 (uniform in the unit, significands
uniform in [1, 2)), so with 10^4 entries of dl or more the difference's 2-norm
is within 2^-8 of the result's; with few, 2^-7."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests import train_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(tokens, vocab, hidden, seed=1, ignored=0.2, ldh=None, ldw=None, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r8 = -(-hidden // 8) * 8
    h = torch.full((tokens, ldh or r8), float("nan"), dtype=torch.bfloat16, device=DEV)
    h[:, :hidden] = std * torch.randn((tokens, hidden), generator=g, device=DEV)
    w = torch.full((vocab, ldw or r8), float("nan"), dtype=torch.bfloat16, device=DEV)
    w[:, :hidden] = torch.randn((vocab, hidden), generator=g, device=DEV) * hidden ** -0.5
    t = torch.randint(0, vocab, (tokens,), generator=g, device=DEV)
    skip = torch.rand((tokens,), generator=g, device=DEV) < ignored
    t = torch.where(skip, torch.full_like(t, -100), t)
    return h[:, :hidden], w[:, :hidden], t


def _forward(h, w, t, z=0.0):
    loss = torch.full((len(t),), 7.0, device=DEV)
    lse = torch.full_like(loss, 7.0)
    ws = torch.full((ufp4.ufp4_head_loss_workspace_size(len(t), *w.shape),), 255, dtype=torch.uint8, device=DEV)
    ufp4.ufp4_head_loss(h, w, t, loss, lse, ws, z_loss=z)
    return loss, lse


def _backward(h, w, t, lse, weight=None, scale=None, z=0.0, dh=torch.bfloat16, dw=torch.bfloat16):
    dh = torch.full(tuple(h.shape), 7.0, dtype=dh, device=DEV) if dh is not None else None
    dw = torch.full(tuple(w.shape), 7.0, dtype=dw, device=DEV) if dw is not None else None
    ws = torch.full((ufp4.ufp4_head_loss_backward_workspace_size(len(t), *w.shape),), 255, dtype=torch.uint8, device=DEV)
    ufp4.ufp4_head_loss_backward(h, w, t, lse, dh, dw, ws, token_weight=weight, scale=scale, z_loss=z)
    return dh, dw


def _check_forward(h, w, t, loss, lse, z=0.0):
    want, want_lse, _, keep = ref.head(h, w, t, z)
    mag = float((h[keep].double().abs() @ w.double().abs().T).max()) if keep.any() else 0.0
    lim = 2.0 ** -19 * mag + 2.0 ** -20 * (1 + want_lse.abs())
    assert ((lse.double() - want_lse).abs() <= lim).all()
    assert ((loss.double() - want).abs() <= 2 * lim * (1 + 2 * z * want_lse.abs())).all()
    assert (loss[~keep] == 0).all() and (lse[~keep] == 0).all()


def _check_grad(got, want, mag, entries):
    if got is None:
        return
    own = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    lim = 2.0 ** -8 * (1 + 2.0 ** -4) * mag + own * want.abs() + 1e-30
    err = (got.double() - want).abs()
    assert (err <= lim).all(), float((err - lim).max())
    norm = float(want.norm())
    assert float(err.norm()) <= (2.0 ** -8 if entries >= 10000 else 2.0 ** -7) * norm + 1e-30, float(err.norm()) / norm


def _check_backward(h, w, t, dh, dw, weight=None, scale=None, z=0.0):
    wh, ww, mh, mw = ref.head_backward(h, w, t, weight, scale, z)
    entries = int(((t >= 0) & (t < len(w))).sum()) * len(w)
    _check_grad(dh, wh, mh, entries)
    _check_grad(dw, ww, mw, entries)


SHAPES = [(1, 1, 1), (1, 7, 8), (3, 255, 63), (5, 256, 64), (64, 257, 72), (65, 1000, 130), (255, 300, 64), (256, 512, 256),
          (257, 5000, 100), (600, 1031, 520), (1, 20000, 1024), (1030, 130, 40)]


@pytest.mark.parametrize("z", [0.0, 1e-3])
@pytest.mark.parametrize("shape", SHAPES)
def test_loss_and_gradients(shape, z):
    h, w, t = _inputs(*shape, seed=sum(shape), ignored=0.0 if shape[0] < 4 else 0.2)
    loss, lse = _forward(h, w, t, z)
    _check_forward(h, w, t, loss, lse, z)
    weight = 0.5 + torch.rand(len(t), device=DEV)
    scale = torch.full((1,), 1.0 / len(t), device=DEV)
    dh, dw = _backward(h, w, t, lse, weight, scale, z)
    _check_backward(h, w, t, dh, dw, weight, scale, z)
    assert ufp4.ufp4_device_error() == 0


@pytest.mark.parametrize("tokens,vocab,hidden", [(4096, 20001, 72), (2300, 50001, 64), (9000, 9000, 136)])
def test_many_pieces_of_the_vocabulary(tokens, vocab, hidden):
    h, w, t = _inputs(tokens, vocab, hidden, ignored=0.05)
    loss, lse = _forward(h, w, t)
    _check_forward(h, w, t, loss, lse)
    dh, dw = _backward(h, w, t, lse, dh=torch.float32, dw=torch.float32)
    _check_backward(h, w, t, dh, dw)


@pytest.mark.parametrize("hd,wd", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32), (None, torch.bfloat16),
                                   (torch.float32, None)])
def test_types_and_single_gradients(hd, wd):
    h, w, t = _inputs(300, 700, 200, seed=4)
    _, lse = _forward(h, w, t)
    dh, dw = _backward(h, w, t, lse, dh=hd, dw=wd)
    _check_backward(h, w, t, dh, dw)


def test_accumulates_into_dw():
    h, w, t = _inputs(300, 700, 203, seed=5)
    _, lse = _forward(h, w, t)
    _, once = _backward(h, w, t, lse, dh=None, dw=torch.float32)
    start = torch.randn((700, 203), device=DEV)
    dw = start.clone()
    ws = torch.empty(ufp4.ufp4_head_loss_backward_workspace_size(300, 700, 203), dtype=torch.uint8, device=DEV)
    ufp4.ufp4_head_loss_backward(h, w, t, lse, None, dw, ws, accumulate_dw=True)
    assert torch.equal(dw, start + once)


def test_ignored_tokens_take_no_part():
    """Rows of h without a target may hold anything; targets past the vocabulary are no targets; the result is that of the
    other tokens alone."""
    h, w, t = _inputs(500, 900, 96, seed=6, ignored=0.5)
    t[7], t[11], t[13] = 900, 1 << 40, -(1 << 62)
    keep = (t >= 0) & (t < 900)
    clean = _forward(h, w, t)
    grads = _backward(h, w, t, clean[1])
    h2 = h.clone()
    h2[~keep] = torch.tensor([float("nan"), float("inf"), -float("inf")], device=DEV).bfloat16().repeat(32)
    dirty = _forward(h2, w, t)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])
    for a, b in zip(grads, _backward(h2, w, t, dirty[1])):
        assert torch.equal(a, b)
    assert (grads[0][~keep] == 0).all()
    hk, tk = h[keep].contiguous(), t[keep].contiguous()
    alone = _forward(hk, w, tk)
    assert torch.equal(alone[0], clean[0][keep])
    dh, dw = _backward(hk, w, tk, alone[1])
    assert torch.equal(dh, grads[0][keep]) and torch.equal(dw, grads[1])


@pytest.mark.parametrize("tokens", [0, 1, 70])
def test_no_token_has_a_target(tokens):
    h, w, _ = _inputs(tokens, 300, 72, seed=7)
    t = torch.full((tokens,), -1, device=DEV)
    loss, lse = _forward(h, w, t)
    assert (loss == 0).all() and (lse == 0).all()
    dh, dw = _backward(h, w, t, lse)
    assert (dh == 0).all() and (dw == 0).all()
    keep = torch.randn((300, 72), device=DEV)
    dw = keep.clone()
    ws = torch.empty(ufp4.ufp4_head_loss_backward_workspace_size(tokens, 300, 72), dtype=torch.uint8, device=DEV)
    ufp4.ufp4_head_loss_backward(h, w, t, lse, None, dw, ws, accumulate_dw=True)
    assert torch.equal(dw, keep)


def test_large_logits_and_equal_logits():
    """Logits in the thousands (the exponentials overflow without the maximum), and a row of zeros (lse = log vocab)."""
    h, w, t = _inputs(130, 500, 64, seed=8, ignored=0.0, std=300.0)
    h[3] = 0
    loss, lse = _forward(h, w, t)
    assert torch.isfinite(loss).all() and float(lse.abs().max()) > 200
    _check_forward(h, w, t, loss, lse)
    assert abs(float(lse[3]) - 6.214608098422191) < 1e-5
    dh, dw = _backward(h, w, t, lse)
    # a logit's absolute error is a relative one of its exponential: 2^-19 of the sum of magnitudes, here up to 2^-7
    wh, ww, mh, mw = ref.head_backward(h, w, t, None, None)
    slack = 2.0 ** -19 * float((h.double().abs() @ w.double().abs().T).max())
    assert ((dh.double() - wh).abs() <= (2.0 ** -8 * (1 + 2.0 ** -4) + slack) * mh + 2.0 ** -8 * wh.abs() + 1e-30).all()
    assert ((dw.double() - ww).abs() <= (2.0 ** -8 * (1 + 2.0 ** -4) + slack) * mw + 2.0 ** -8 * ww.abs() + 1e-30).all()


def test_nan_and_infinity_in_a_valid_row():
    h, w, t = _inputs(40, 300, 64, seed=9, ignored=0.0)
    h[5, 3] = float("nan")
    loss, lse = _forward(h, w, t)
    assert torch.isnan(loss[5]) and torch.isnan(lse[5])
    others = torch.arange(40, device=DEV) != 5
    assert torch.isfinite(loss[others]).all()
    dh, _ = _backward(h, w, t, lse)
    assert torch.isnan(dh[5].float()).all() and torch.isfinite(dh[others].float()).all()


def test_gradient_against_differences():
    """Central differences of the 64-bit loss along random directions of h and w."""
    h, w, t = _inputs(48, 200, 64, seed=10)
    weight = 0.5 + torch.rand(48, device=DEV)
    scale = torch.full((1,), 0.25, device=DEV)
    z = 1e-2
    _, lse = _forward(h, w, t, z)
    dh, dw = _backward(h, w, t, lse, weight, scale, z, torch.float32, torch.float32)
    _, _, mh, mw = ref.head_backward(h, w, t, weight, scale, z)
    g = torch.Generator(device=DEV).manual_seed(3)

    def f(a, b):
        return float((ref.head(a, b, t, z)[0] * weight.double()).sum() * scale.double())
    for got, mag, which in ((dh, mh, 0), (dw, mw, 1)):
        x = (h.double(), w.double())
        for _ in range(4):
            d = torch.randn(tuple(got.shape), generator=g, device=DEV, dtype=torch.float64)
            e = 1e-5
            hi, lo = list(x), list(x)
            hi[which], lo[which] = x[which] + e * d, x[which] - e * d
            num = (f(*hi) - f(*lo)) / (2 * e)
            # independent roundings of the entries add up as a norm; 1e-6: the differences' own error
            lim = 2.0 ** -8 * float((mag * d).norm()) + 1e-6 * float((mag * d).abs().sum())
            assert abs(float((got.double() * d).sum()) - num) <= lim


@pytest.mark.parametrize("ld", [72, 80, 200])
def test_leading_dimensions_and_guards(ld):
    """Padded operands (NaN in the padding), outputs of any pitch and alignment, nothing written outside their rows."""
    tokens, vocab, hidden = 100, 333, 70
    h, w, t = _inputs(tokens, vocab, hidden, seed=11, ldh=ld, ldw=ld)
    loss, lse = _forward(h, w, t)
    _check_forward(h, w, t, loss, lse)
    for dtype in (torch.bfloat16, torch.float32):
        bufs = [torch.full((5 + n * (hidden + 3) + 64,), 3.0, dtype=dtype, device=DEV) for n in (tokens, vocab)]
        outs = [b[5:5 + n * (hidden + 3)].view(n, hidden + 3)[:, :hidden] for b, n in zip(bufs, (tokens, vocab))]
        ws = torch.full((ufp4.ufp4_head_loss_backward_workspace_size(tokens, vocab, hidden) + 512,), 255, dtype=torch.uint8,
                        device=DEV)
        ufp4.ufp4_head_loss_backward(h, w, t, lse, *outs, ws[:-512])
        _check_backward(h, w, t, *outs)
        assert (ws[-512:] == 255).all()
        for b, n in zip(bufs, (tokens, vocab)):
            body = b[5:5 + n * (hidden + 3)].view(n, hidden + 3)
            assert (b[:5] == 3).all() and (b[5 + n * (hidden + 3):] == 3).all() and (body[:, hidden:] == 3).all()


def test_reproducible_on_another_stream():
    h, w, t = _inputs(700, 3000, 256, seed=12)
    loss, lse = _forward(h, w, t)
    dh, dw = _backward(h, w, t, lse)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        loss2, lse2 = _forward(h, w, t)
        dh2, dw2 = _backward(h, w, t, lse2)
    side.synchronize()
    for a, b in ((loss, loss2), (lse, lse2), (dh, dh2), (dw, dw2)):
        assert torch.equal(a, b)


def test_in_a_graph():
    """Forward and backward captured, replayed on new inputs (the count of valid tokens is read on the device)."""
    tokens, vocab, hidden = 300, 900, 128
    h, w, t = _inputs(tokens, vocab, hidden, seed=13)
    h2, w2, t2 = _inputs(tokens, vocab, hidden, seed=14, ignored=0.6)
    loss, lse = torch.empty(tokens, device=DEV), torch.empty(tokens, device=DEV)
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    ws = torch.empty(max(ufp4.ufp4_head_loss_workspace_size(tokens, vocab, hidden),
                         ufp4.ufp4_head_loss_backward_workspace_size(tokens, vocab, hidden)), dtype=torch.uint8, device=DEV)

    def run():
        ufp4.ufp4_head_loss(h, w, t, loss, lse, ws)
        ufp4.ufp4_head_loss_backward(h, w, t, lse, dh, dw, ws)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for a, b in ((h, h2), (w, w2), (t, t2)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    _check_forward(h2, w2, t2, loss, lse)
    _check_backward(h2, w2, t2, dh, dw)


@pytest.mark.parametrize("tokens", [1, 31, 127, 128, 129])
@pytest.mark.parametrize("vocab", [33, 4000, 40001])
def test_few_tokens(tokens, vocab):
    """The tiles of up to 128 tokens: one or several per CTA, ragged widths, tokens in place."""
    h, w, t = _inputs(tokens, vocab, 192, seed=tokens, ignored=0.3)
    loss, lse = _forward(h, w, t)
    _check_forward(h, w, t, loss, lse)


@pytest.mark.parametrize("tokens", [1, 100, 128, 129, 200, 256, 300, 384, 385])
@pytest.mark.parametrize("vocab,hidden", [(33, 64), (4000, 200), (40001, 136)])
def test_up_to_a_few_hundred_tokens(tokens, vocab, hidden):
    """Both sides of the steps from single CTAs' tiles to pairs', forward (128 tokens) and backward (384)."""
    h, w, t = _inputs(tokens, vocab, hidden, seed=tokens, ignored=0.3)
    loss, lse = _forward(h, w, t)
    _check_forward(h, w, t, loss, lse)
    dh, dw = _backward(h, w, t, lse)
    _check_backward(h, w, t, dh, dw)
