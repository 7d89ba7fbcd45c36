"""Gradients of the vocabulary loss on few tokens, where no rounding of dl is averaged away: the entry at a token's target,
weight (p - 1), dominates its row of dl, and one rounding of it moves the token's whole gradient.

Tolerances, of fp32 gradients, element by element.  Up to 128 tokens dl is kept in two bf16 parts for dw: each entry within
2^-16 of itself.  For dh it is rounded to bf16 but at the target, where the remainder is added back, so what is left is the
rounding of the entries w a p of the others, each spread over +-2^-8 of its power of two with a standard deviation of at
most 2^-8 / sqrt(3) of the entry, independent of one another: six standard deviations of their sum.  To both: the exponential's error,
2^-19 of the largest sum of magnitudes |h| |w| (a logit's error is an absolute one of the exponent) and 2^-20 of p, and
2^-20 of the sum of magnitudes for the fp32 sums.  bf16 gradients: their own rounding is all that shows, so their distance
from the exact ones is within a tenth of that of the exact ones rounded."""
import math

import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests import train_ref as ref
from tests.test_head_loss_gpu import _backward, _forward, _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _dl(h, w, t, weight, z):
    """dl of the valid tokens and its part w a p, in 64 bits."""
    _, lse, logits, keep = ref.head(h, w, t, z)
    l = lse[keep][:, None]
    part = torch.exp(logits - l) * (1 + 2 * z * l) * weight.double()[keep][:, None]
    dl = part.clone()
    dl[torch.arange(len(dl), device=DEV), t[keep]] -= weight.double()[keep]
    return dl, part, keep


@pytest.mark.parametrize("tokens,vocab,hidden,ignored", [
    (1, 7243, 2272, 0.0), (2, 1000, 256, 0.0), (10, 12140, 3200, 0.0), (16, 32000, 264, 0.2), (31, 5000, 136, 0.0),
    (32, 3001, 200, 0.0), (33, 3001, 200, 0.0), (64, 2000, 72, 0.0), (65, 4000, 70, 0.1), (100, 9000, 64, 0.5),
    (127, 1500, 136, 0.0), (128, 1500, 135, 0.0), (128, 40001, 64, 0.3)])
@pytest.mark.parametrize("z", [0.0, 1e-3])
def test_no_rounding_moves_a_tokens_gradient(tokens, vocab, hidden, ignored, z):
    h, w, t = _inputs(tokens, vocab, hidden, seed=tokens, ignored=ignored)
    g = torch.Generator(device=DEV).manual_seed(hidden)
    weight = 0.5 + torch.rand((tokens,), generator=g, device=DEV)
    scale = torch.full((1,), 1.0 / tokens, device=DEV)
    _, lse = _forward(h, w, t, z)
    dl, part, keep = _dl(h, w, t, weight, z)
    s, hk, w64 = float(scale), h[keep].double(), w.double()
    want = torch.zeros_like(h, dtype=torch.float64)
    want[keep] = s * (dl @ w64)
    want_dw = s * (dl.T @ hk)
    p_error = 2.0 ** -19 * float((hk.abs() @ w64.abs().T).max()) + 2.0 ** -20 if keep.any() else 0.0
    lim = torch.zeros_like(want)
    lim[keep] = s * (6 * 2.0 ** -8 / math.sqrt(3) * (part.square() @ w64.square()).sqrt() + p_error * (part @ w64.abs())
                     + 2.0 ** -20 * (dl.abs() @ w64.abs()))
    lim_dw = s * ((2.0 ** -16 + 2.0 ** -20) * (dl.abs().T @ hk.abs()) + p_error * (part.T @ hk.abs()))
    dh, dw = _backward(h, w, t, lse, weight, scale, z, torch.float32, torch.float32)
    assert ((dh.double() - want).abs() <= lim + 1e-30).all()
    assert ((dw.double() - want_dw).abs() <= lim_dw + 1e-30).all()
    half = _backward(h, w, t, lse, weight, scale, z)
    for got, exact in zip(half, (want, want_dw)):
        rounded = float((exact.bfloat16().double() - exact).norm())
        assert float((got.double() - exact).norm()) <= 1.1 * rounded
    assert ufp4.ufp4_device_error() == 0


def test_gradients_alone_and_accumulated():
    """Each gradient by itself, added to what is there, and with ignored tokens of any content, has the same bits."""
    tokens, vocab, hidden = 90, 3000, 200
    h, w, t = _inputs(tokens, vocab, hidden, seed=5, ignored=0.4)
    g = torch.Generator(device=DEV).manual_seed(6)
    weight = 0.5 + torch.rand((tokens,), generator=g, device=DEV)
    _, lse = _forward(h, w, t)
    dh, dw = _backward(h, w, t, lse, weight, None, 0.0, torch.float32, torch.float32)
    assert torch.equal(_backward(h, w, t, lse, weight, None, 0.0, torch.float32, None)[0], dh)
    assert torch.equal(_backward(h, w, t, lse, weight, None, 0.0, None, torch.float32)[1], dw)
    start = torch.randn((vocab, hidden), generator=g, device=DEV)
    total = start.clone()
    ws = torch.full((ufp4.ufp4_head_loss_backward_workspace_size(tokens, vocab, hidden) + 512,), 255, dtype=torch.uint8,
                    device=DEV)
    ufp4.ufp4_head_loss_backward(h, w, t, lse, None, total, ws[:-512], token_weight=weight, accumulate_dw=True)
    assert torch.equal(total, start + dw) and (ws[-512:] == 255).all()
    keep = t >= 0
    h2 = h.clone()
    h2[~keep] = float("nan")
    again = _backward(h2, w, t, lse, weight, None, 0.0, torch.float32, torch.float32)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw) and (dh[~keep] == 0).all()
    alone = _backward(h[keep].contiguous(), w, t[keep].contiguous(), lse[keep].contiguous(), weight[keep].contiguous(), None,
                      0.0, torch.float32, torch.float32)
    assert torch.equal(alone[0], dh[keep]) and torch.equal(alone[1], dw)
