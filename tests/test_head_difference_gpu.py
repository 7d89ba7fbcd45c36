"""The vocabulary loss's gradients against central differences of the 64-bit loss, along random directions of h and w.

Tolerance.  An entry of dl is rounded to bf16: 8 significant bits, so an error spread over +-2^-8 of its power of two, with a
standard deviation of at most 2^-8 / sqrt(3) of the entry.  Along a direction the entries' errors add up with the factors
x = dl * (direction . w) (or h), independent of one another, so the sum has a standard deviation of at most 2^-8 / sqrt(3)
* |x|_2; the limit is six of them.  Beside it, relative to sum |x|: 2^-19 of the largest sum of magnitudes |h| |w| for a
logit's error (an absolute error of the exponent), 2^-20 for the exponential and the fp32 sums, and 1e-6 for the differences
(step 1e-5: truncation 1e-10, and 2^-53 of the loss over the step)."""
import math

import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests import train_ref as ref
from tests.test_head_loss_gpu import _backward, _forward, _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("tokens,vocab,hidden,z", [(48, 200, 64, 1e-2), (300, 700, 40, 0.0), (130, 1500, 200, 1e-3)])
def test_gradients_against_differences(tokens, vocab, hidden, z):
    h, w, t = _inputs(tokens, vocab, hidden, seed=tokens)
    g = torch.Generator(device=DEV).manual_seed(vocab)
    weight = 0.5 + torch.rand((tokens,), generator=g, device=DEV)
    scale = torch.full((1,), 0.25, device=DEV)
    _, lse = _forward(h, w, t, z)
    dh, dw = _backward(h, w, t, lse, weight, scale, z, torch.float32, torch.float32)
    _, l64, logits, keep = ref.head(h, w, t, z)
    dl = torch.exp(logits - l64[keep][:, None]) * (1 + 2 * z * l64[keep])[:, None]
    dl[torch.arange(len(dl), device=DEV), t[keep]] -= 1
    dl *= (weight.double() * scale.double())[keep][:, None]
    logit = 2.0 ** -19 * float((h[keep].double().abs() @ w.double().abs().T).max())

    def f(a, b):
        return float((ref.head(a, b, t, z)[0] * weight.double()).sum() * scale.double())
    e = 1e-5
    x = (h.double(), w.double())
    for which, got in ((0, dh), (1, dw)):
        for _ in range(8):
            d = torch.randn(tuple(got.shape), generator=g, device=DEV, dtype=torch.float64)
            hi, lo = list(x), list(x)
            hi[which], lo[which] = x[which] + e * d, x[which] - e * d
            num = (f(*hi) - f(*lo)) / (2 * e)
            terms = dl * (d[keep] @ w.double().T if which == 0 else h[keep].double() @ d.T)
            lim = 6 * 2.0 ** -8 / math.sqrt(3) * float(terms.norm()) + (logit + 2.0 ** -20 + 1e-6) * float(terms.abs().sum())
            assert abs(float((got.double() * d).sum()) - num) <= lim
    assert ufp4.ufp4_device_error() == 0
