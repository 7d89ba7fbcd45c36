"""ufp4_layer_norm on constant and nearly constant rows far from zero, against 64 bits, with limits that go by the row's
deviations.

Tolerances, u = 2^-24.  The first mean is off by at most E = 64 u A, A the row's mean magnitude (test_layer_norm_gpu).  The
differences from it, of mean magnitude D <= mean |s - m| + E, are off by u of themselves, their mean by 64 u D for the sum and 3 u
D for the differences, the product and the reciprocal.  So (s - first) - rest is off by 70 u (D + |s - m|) at most.  The variance
is mean d^2 - rest^2: 70 u (var + E^2) and 2 E times rest's error, 140 u E D; half of that, relative to var + eps, is rstd's
error, with 4 u for rsqrtf and products.  mean is written as one fp32 number: half a step, u |m|, and rest's error.  A bf16 y adds
2^-8 of itself."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests import fp8_ref as ref
from tests.test_layer_norm_gpu import _weights, _within, EPS

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, BF = 2.0 ** -24, 2.0 ** -8


def _check(s, gamma, beta, y, mean, rstd):
    wy, wm, wr = ref.layer_norm(s, gamma, beta, EPS)
    c = (s.double().cpu() - wm[:, None]).abs()
    var = c.square().mean(1)
    E = 64 * U * s.double().cpu().abs().mean(1)
    D = c.mean(1) + E
    off = (70 * U * (var + E * E) + 140 * U * E * D) / (var + EPS)
    rel = 0.5 * off / (1 - off) + 4 * U
    _within(mean, wm, U * wm.abs() + 70 * U * D, "mean")
    _within(rstd, wr, wr * rel, "rstd")
    w, b = gamma.double().cpu().abs(), (0 if beta is None else beta.double().cpu().abs())
    h = c * wr[:, None]
    lim = w * (70 * U * (D[:, None] + c) * (wr * (1 + rel))[:, None] + h * (rel[:, None] + 4 * U)) + 2 * U * (w * h + b)
    _within(y, wy, (lim + BF * wy.abs()) * (1 + 2.0 ** -7), "y")


VALUES = [0.0, 1.0, -3.0, 176.0, 1000.0, -30000.0, 99840.0, 1e-3]  # bf16 numbers but the last


@pytest.mark.parametrize("cols", [7, 257, 1792, 7167, 7168, 8200, 14336, 16384, 28672])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_constant_rows(cols, dtype):
    x = torch.tensor(VALUES).to(DEV, dtype)[:, None].expand(-1, cols).contiguous()
    gamma, beta = _weights(cols, 4, torch.float32)
    rows = x.shape[0]
    y, mean, rstd = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    for b in (None, beta):
        ufp4.ufp4_layer_norm(x, gamma, y, mean, rstd, beta=b, eps=EPS)
        _check(x, gamma, b, y, mean, rstd)
    # the sum of two constants, and its bf16 rounding
    residual, total = torch.full((rows, cols), 0.75, dtype=torch.bfloat16, device=DEV), torch.empty_like(y)
    ufp4.ufp4_layer_norm(x, gamma, y, mean, rstd, residual=residual, total=total, eps=EPS)
    s = x.float() + residual.float()
    _check(s, gamma, None, y, mean, rstd)
    assert torch.equal(total, s.bfloat16())


@pytest.mark.parametrize("noise", [1e-4, 1e-2, 1.0])
@pytest.mark.parametrize("cols", [300, 1027, 7168, 7169, 14336, 28672])
def test_small_deviations_far_from_zero(cols, noise):
    g = torch.Generator().manual_seed(cols)
    x = (torch.tensor(VALUES)[:, None] * 1.0 + noise * torch.randn((len(VALUES), cols), generator=g)).to(DEV)
    gamma, beta = _weights(cols, 4, torch.float32)
    rows = x.shape[0]
    y, mean, rstd = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ufp4.ufp4_layer_norm(x, gamma, y, mean, rstd, beta=beta, eps=EPS)
    _check(x, gamma, beta, y, mean, rstd)


@pytest.mark.parametrize("cols", [1792, 7168, 7169])
def test_a_constant_row_has_no_gradient_but_the_common_one(cols):
    """Backward at the mean that the forward call wrote: h is 0 on a constant row, so dgamma is 0 and dx = rstd (q - mean q)."""
    x = torch.tensor(VALUES[:7], device=DEV)[:, None].expand(-1, cols).contiguous()
    g = torch.Generator().manual_seed(3)
    dy = torch.randn((7, cols), generator=g).to(DEV, torch.bfloat16)
    gamma, _ = _weights(cols, 4, torch.float32)
    y, mean, rstd = torch.empty((7, cols), dtype=torch.bfloat16, device=DEV), torch.empty(7, device=DEV), torch.empty(7, device=DEV)
    ufp4.ufp4_layer_norm(x, gamma, y, mean, rstd, eps=EPS)
    assert torch.equal(mean, x[:, 0])
    dx, dg, db = torch.empty_like(y), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.empty(ufp4.ufp4_layer_norm_backward_workspace_size(7, cols), dtype=torch.uint8, device=DEV)
    ufp4.ufp4_layer_norm_backward(dy, x, mean, rstd, gamma, dx, dg, db, ws)
    assert (dg == 0).all()
    wdx, _, _, _, q = ref.layer_norm_backward(x, mean, rstd, gamma, dy)
    terms = rstd.double().cpu()[:, None] * (q.abs() + q.abs().mean(1, keepdim=True))
    _within(dx, wdx, 80 * U * terms + BF * wdx.abs() * (1 + 2.0 ** -8), "dx")
