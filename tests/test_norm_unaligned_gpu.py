"""The norm on operands off alignment and of other pitches, against the 64-bit formulas, at the tolerances that
tests/test_checkpoint_ops_gpu.py derives: rstd 2^-20 of itself, dgamma (rows + 8) 2^-24 of its sum of magnitudes, the bf16
results a unit of bf16 and 2^-18 of their terms; the checkpoint and the bf16 sum are exact."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests import train_ref as ref
from tests.test_checkpoint_ops_gpu import EPS, _check_ckpt, _ckpt, _near, _placed, _rand

pytestmark = pytest.mark.gpu
DEV = "cuda"


# columns, pitch, first element; one operand off alignment, or all of them
@pytest.mark.parametrize("cols,ld,offset", [(64, 72, 0), (64, 65, 0), (64, 64, 1), (96, 104, 3), (70, 71, 1), (1408, 1411, 5),
                                            (2047, 2047, 0), (9001, 9003, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("which", ["x", "residual", "gamma", "y", "ckpt", "all"])
def test_norm_passes(cols, ld, offset, dtype, which):
    rows = 13

    def put(t, name):
        return _placed(t, ld, offset) if which in (name, "all") else t.to(DEV)
    x, res, dy = _rand(rows, cols, 81, dtype=dtype), _rand(rows, cols, 82, 2.0), _rand(rows, cols, 83, 1e-3, dtype)
    gamma = (1 + 0.1 * torch.randn((1, cols), generator=torch.Generator().manual_seed(84))).to(DEV)
    gm = _placed(gamma, None, offset)[0] if which in ("gamma", "all") else gamma[0]
    y, total, dx, again = (put(torch.full((rows, cols), 3.0, dtype=torch.bfloat16, device=DEV), "y") for _ in range(4))
    rstd, dgamma = torch.empty(rows, device=DEV), torch.empty(cols, device=DEV)
    where = (cols + 3, -(-cols // 32) + 2, offset) if which in ("ckpt", "all") else ()
    codes, scales, q = _ckpt(rows, cols, *where)
    ufp4.ufp4_rms_norm(put(x, "x"), gm, y, rstd, residual=put(res, "residual"), total=total, ckpt=q, eps=EPS)
    s = x.float() + res.float()
    want, rs = ref.norm(s.cpu(), gamma[0].cpu(), EPS)
    assert ((rstd.double().cpu() - rs).abs() <= 2.0 ** -20 * rs).all()
    _near(y, want, what="y")
    assert torch.equal(total, s.bfloat16())
    _check_ckpt(codes, scales, s, "sum")
    ws = torch.empty(ufp4.ufp4_rms_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=DEV)
    ufp4.ufp4_rms_norm_backward(put(dy, "x"), q, rstd, gm, dx, dgamma, ws, dtotal=put(res, "residual"), y=again)
    saved, r = ref.decode(codes, scales), rstd.cpu()
    d, dg, yw = ref.norm_backward(saved, r, gamma[0].cpu(), dy.cpu())
    add, qq, h = res.double().cpu(), dy.double().cpu() * gamma.double().cpu(), saved * r.double()[:, None]
    terms = r.double()[:, None] * (qq.abs() + h.abs() * (qq * h).abs().mean(1, keepdim=True)) + add.abs()
    _near(dx, d + add, terms=terms, what="dx")
    lim = (rows + 8) * 2.0 ** -24 * (dy.double().cpu() * h).abs().sum(0) + 1e-30
    assert ((dgamma.double().cpu() - dg).abs() <= lim).all()
    _near(again, yw, what="y again")
