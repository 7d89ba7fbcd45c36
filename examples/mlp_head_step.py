"""A training step of one feed-forward block and the vocabulary head, all through the library:

  x -> RMS norm -> gate/up GEMM -> gated activation -> down GEMM -> + x, RMS norm -> loss over the vocabulary

and back.  The three GEMMs of each linear layer run on 4-bit operands (FPROP and WGRAD operands rounded
to nearest, the gradient stochastically); between the passes the step keeps only 8-bit checkpoints, one
fp32 number per row and token, and x itself.

  python examples/mlp_head_step.py [--tokens 2048 --hidden 1024 --ffn 2816 --vocab 16384 --steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from rht_bit_block_gb300 import ufp4  # noqa: E402

SIGN_SEED = 0x5EED0001
EPS = 1e-6


def _desc(rounding=ufp4.ROUND_RTNE, sr_seed=0, out_mask=ufp4.OUT_ROWWISE):
    return ufp4.make_desc(grid="e1m2", block=(1, 16), n=16, sign_seed=SIGN_SEED, rounding=rounding, sr_seed=sr_seed,
                          scale_fmt=ufp4.SCALE_UE8M0, out_mask=out_mask)


def _gemm(a, b, M, N, K):
    """D[M, N] = Q(A) Q(B)^T of two quantized operands (codes, scales) along K."""
    desc = _desc()
    d = torch.empty((M, N), dtype=torch.float32, device="cuda")
    ws = torch.empty(max(1, ufp4.ufp4_gemm_workspace_size(M, N, K, desc)), dtype=torch.uint8, device="cuda")
    ufp4.ufp4_gemm(ufp4.qtensor(*a, M, K), ufp4.qtensor(*b, N, K), desc, d, ws)
    return d


class Linear:
    """y = x w^T with quantized FPROP, DGRAD and WGRAD; w: bf16 [out, in]."""

    def __init__(self, out, inp, gen):
        self.w = (torch.randn((out, inp), generator=gen, device="cuda") * inp ** -0.5).bfloat16()

    def forward(self, x):
        self.q = ufp4.quantize(self.w, _desc(out_mask=ufp4.OUT_ROWWISE | ufp4.OUT_COLWISE))
        return _gemm(ufp4.quantize(x, _desc())["row"], self.q["row"], len(x), *self.w.shape)

    def backward_input(self, dy, seed):
        """dx = dy w; keeps dy's column-wise quantization for backward_weight."""
        out, inp = self.w.shape
        q = ufp4.quantize(dy, _desc(ufp4.ROUND_SR, seed, ufp4.OUT_ROWWISE | ufp4.OUT_COLWISE))
        self.dy = q["col"]
        return _gemm(q["row"], self.q["col"], len(dy), inp, out)

    def backward_weight(self, x):
        """dw = dy^T x."""
        out, inp = self.w.shape
        return _gemm(self.dy, ufp4.quantize(x, _desc(out_mask=ufp4.OUT_COLWISE))["col"], out, inp, len(x))


class Checkpoint:
    def __init__(self, rows, cols):
        self.codes, self.scales = ufp4.alloc_checkpoint(rows, cols, "cuda")
        self.q = ufp4.qtensor(self.codes, self.scales, rows, cols)


class Norm:
    """RMS norm of x + residual, from an 8-bit checkpoint in the backward pass."""

    def __init__(self, rows, cols):
        self.gamma = torch.ones(cols, device="cuda")
        self.rstd = torch.empty(rows, device="cuda")
        self.saved = Checkpoint(rows, cols)
        self.ws = torch.empty(ufp4.ufp4_rms_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")

    def forward(self, x, residual=None):
        y = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
        ufp4.ufp4_rms_norm(x, self.gamma, y, self.rstd, residual=residual, ckpt=self.saved.q, eps=EPS)
        return y

    def backward(self, dy, dtotal=None, remake=False):
        dx = torch.empty(dy.shape, dtype=torch.bfloat16, device="cuda")
        y = torch.empty_like(dx) if remake else None
        dgamma = torch.empty_like(self.gamma)
        ufp4.ufp4_rms_norm_backward(dy, self.saved.q, self.rstd, self.gamma, dx, dgamma, self.ws, dtotal=dtotal, y=y)
        return dx, dgamma, y


class Model:
    def __init__(self, tokens, hidden, ffn, vocab, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.gate_up, self.down = Linear(2 * ffn, hidden, gen), Linear(hidden, ffn, gen)
        self.head = (torch.randn((vocab, hidden), generator=gen, device="cuda") * hidden ** -0.5).bfloat16()
        self.norm1, self.norm2 = Norm(tokens, hidden), Norm(tokens, hidden)
        self.gate, self.up = Checkpoint(tokens, ffn), Checkpoint(tokens, ffn)
        self.loss, self.lse = (torch.empty(tokens, device="cuda") for _ in range(2))
        sizes = (tokens, vocab, hidden)
        need = max(ufp4.ufp4_head_loss_workspace_size(*sizes), ufp4.ufp4_head_loss_backward_workspace_size(*sizes))
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        self.ffn = ffn

    def forward(self, x, targets):
        f = self.ffn
        both = self.gate_up.forward(self.norm1.forward(x))
        act = torch.empty((len(x), f), dtype=torch.bfloat16, device="cuda")
        ufp4.ufp4_glu(both[:, :f], both[:, f:], act, ckpt_gate=self.gate.q, ckpt_up=self.up.q)
        self.h = self.norm2.forward(self.down.forward(act), residual=x)
        ufp4.ufp4_head_loss(self.h, self.head, targets, self.loss, self.lse, self.ws)
        return self.loss.sum() / (targets >= 0).sum()

    def backward(self, targets, seed=1):
        """Gradients of the mean loss over the tokens that have a target."""
        f, g = self.ffn, {}
        scale = ((targets >= 0).sum().float().reciprocal()).reshape(1)
        dh, g["head"] = torch.empty_like(self.h), torch.empty(self.head.shape, device="cuda")
        ufp4.ufp4_head_loss_backward(self.h, self.head, targets, self.lse, dh, g["head"], self.ws, scale=scale)
        stream, g["gamma2"], _ = self.norm2.backward(dh)
        dact = self.down.backward_input(stream, seed)
        dboth = torch.empty((len(dh), 2 * f), dtype=torch.bfloat16, device="cuda")
        act = torch.empty((len(dh), f), dtype=torch.bfloat16, device="cuda")
        ufp4.ufp4_glu_backward(dact, self.gate.q, self.up.q, dboth[:, :f], dboth[:, f:], y=act)
        g["down"] = self.down.backward_weight(act)
        dnorm = self.gate_up.backward_input(dboth, seed + 1)
        g["x"], g["gamma1"], normed = self.norm1.backward(dnorm, dtotal=stream, remake=True)
        g["gate_up"] = self.gate_up.backward_weight(normed)
        return g

    def update(self, g, rate):
        for name, w in (("head", self.head), ("down", self.down.w), ("gate_up", self.gate_up.w)):
            w -= (rate * g[name]).to(w.dtype)
        self.norm1.gamma -= rate * g["gamma1"]
        self.norm2.gamma -= rate * g["gamma2"]


def data(tokens, hidden, vocab, ignored=0.1, seed=7):
    """Token embeddings, and targets that follow from them (each of 64 tokens has one successor)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    table = torch.randn((64, hidden), generator=gen, device="cuda")
    follows = torch.randint(0, vocab, (64,), generator=gen, device="cuda")
    ids = torch.randint(0, 64, (tokens,), generator=gen, device="cuda")
    skip = torch.rand((tokens,), generator=gen, device="cuda") < ignored
    return table[ids].bfloat16(), torch.where(skip, torch.full_like(ids, -100), follows[ids])


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 2048), ("hidden", 1024), ("ffn", 2816), ("vocab", 16384), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--rate", type=float, default=0.05)
    a = ap.parse_args()
    model = Model(a.tokens, a.hidden, a.ffn, a.vocab)
    x, targets = data(a.tokens, a.hidden, a.vocab)
    for step in range(a.steps):
        loss = model.forward(x, targets)
        model.update(model.backward(targets, seed=2 * step + 1), a.rate)
        print(f"step {step}: loss {float(loss):.4f}")


if __name__ == "__main__":
    main()
