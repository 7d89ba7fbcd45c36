"""The example's training step: its loss and gradients against the same block in
fp32 torch autograd, and a few steps of descent.

The 4-bit operands dominate the error (E1M2 with 16-element blocks: about 10 %
per operand, so a gradient that went through two GEMMs keeps a cosine of 0.9
with the fp32 one); the head's gradient has only the bf16 h and w and one 4-bit
forward in front of it."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("mlp_head_step", os.path.join(ROOT, "examples", "mlp_head_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _reference(model, x, targets, f):
    p = {n: t.float().requires_grad_() for n, t in (("gate_up", model.gate_up.w), ("down", model.down.w),
                                                    ("head", model.head), ("x", x), ("gamma1", model.norm1.gamma),
                                                    ("gamma2", model.norm2.gamma))}

    def norm(t, gamma):
        return t * (t.square().mean(1, keepdim=True) + 1e-6).rsqrt() * gamma
    both = norm(p["x"], p["gamma1"]) @ p["gate_up"].T
    act = torch.sigmoid(both[:, :f]) * both[:, :f] * both[:, f:]
    logits = norm(act @ p["down"].T + p["x"], p["gamma2"]) @ p["head"].T
    keep = targets >= 0
    loss = (torch.logsumexp(logits[keep], 1) - logits[keep].gather(1, targets[keep][:, None])[:, 0]).mean()
    loss.backward()
    return loss.detach(), {n: t.grad for n, t in p.items()}


def test_step_against_autograd(ex):
    t, hidden, f, vocab = 512, 256, 512, 1000
    model = ex.Model(t, hidden, f, vocab)
    x, targets = ex.data(t, hidden, vocab)
    loss = model.forward(x, targets)
    want, grads = _reference(model, x, targets, f)
    assert abs(float(loss) - float(want)) <= 0.02 * float(want)
    got = model.backward(targets)
    for name, g in got.items():
        cos = torch.nn.functional.cosine_similarity(g.float().flatten(), grads[name].flatten(), dim=0)
        assert float(cos) > 0.9, (name, float(cos))
        assert 0.8 < float(g.float().norm() / grads[name].norm()) < 1.25, name


def test_steps_lower_the_loss(ex):
    model = ex.Model(256, 256, 512, 700)
    x, targets = ex.data(256, 256, 700)
    losses = []
    for step in range(8):
        losses.append(float(model.forward(x, targets)))
        model.update(model.backward(targets, seed=2 * step + 1), 2.0)
    assert losses[-1] < 0.7 * losses[0], losses
