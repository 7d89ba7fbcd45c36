"""Layer norm and an 8-bit projection as a training step uses them: norm of the residual stream, quantization of its output and
of the weight, FPROP, and back through DGRAD, WGRAD (added to a running gradient) and the norm's gradients; eagerly, and captured
into one graph that is replayed on other values.

Tolerances.  Each step is held against 64 bits at its own inputs with the bounds of its operator's tests.  The whole is held
against the unquantized 64-bit step: E4M3 rounds an element by at most 2^-4 of itself, 2^-4 / sqrt(3) in the mean square, and two
operands of a product by sqrt(2) times that, 0.051 of its norm (the products' signs are random); the norm's backward pass only
takes two directions out of its input."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests import fp8_ref as ref
from tests.test_fp8_gemm_gpu import check
from tests.test_layer_norm_gpu import _check_backward, _check_forward, EPS

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Operand:
    """Both 8-bit forms of a matrix."""

    def __init__(self, rows, cols, block):
        self.block = block
        self.row, self.col = ufp4.alloc_fp8(rows, cols, block, DEV), ufp4.alloc_fp8(cols, rows, block, DEV)
        self.r, self.c = ufp4.qtensor(*self.row, rows, cols), ufp4.qtensor(*self.col, cols, rows)

    def write(self, v):
        ufp4.ufp4_fp8_quantize(v, self.r, self.c, block_rows=self.block)

    def values(self):
        return ref.restore(*self.row, self.block).to(DEV), ref.restore(*self.col, self.block).to(DEV)


class Step:
    def __init__(self, tokens, hidden, out):
        bf, f = torch.bfloat16, torch.float32

        def buf(shape, dtype):
            return torch.empty(shape, dtype=dtype, device=DEV)
        self.x, self.residual, self.dout = buf((tokens, hidden), f), buf((tokens, hidden), bf), buf((tokens, out), f)
        self.dstream, self.w = buf((tokens, hidden), bf), buf((out, hidden), bf)
        self.gamma, self.beta = buf((hidden,), f), buf((hidden,), f)
        self.y, self.total, self.dx = (buf((tokens, hidden), bf) for _ in range(3))
        self.mean, self.rstd = buf((tokens,), f), buf((tokens,), f)
        self.result, self.dy, self.dw = buf((tokens, out), bf), buf((tokens, hidden), f), buf((out, hidden), f)
        self.dgamma, self.dbeta = buf((hidden,), f), buf((hidden,), f)
        self.qy, self.qw, self.qd = Operand(tokens, hidden, 1), Operand(out, hidden, 128), Operand(tokens, out, 1)
        self.ws = buf((ufp4.ufp4_layer_norm_backward_workspace_size(tokens, hidden),), torch.uint8)

    def fill(self, seed):
        g = torch.Generator().manual_seed(seed)
        for t, std in ((self.x, 1.0), (self.residual, 2.0), (self.dout, 1e-3), (self.dstream, 1e-3), (self.w, 0.05),
                       (self.gamma, 0.1), (self.beta, 0.1), (self.dw, 1e-2)):
            t.copy_((torch.randn(t.shape, generator=g) * std).to(t.dtype))
        self.gamma += 1.0

    def run(self):
        ufp4.ufp4_layer_norm(self.x, self.gamma, self.y, self.mean, self.rstd, beta=self.beta, residual=self.residual,
                             total=self.total, eps=EPS)
        self.qy.write(self.y)
        self.qw.write(self.w)
        ufp4.ufp4_fp8_gemm(self.qy.r, self.qw.r, self.result)
        self.qd.write(self.dout)
        ufp4.ufp4_fp8_gemm(self.qd.r, self.qw.c, self.dy)
        ufp4.ufp4_fp8_gemm(self.qd.c, self.qy.c, self.dw, b_block_rows=1, accumulate=True)
        ufp4.ufp4_layer_norm_backward(self.dy, self.total, self.mean, self.rstd, self.gamma, self.dx, self.dgamma, self.dbeta,
                                      self.ws, dtotal=self.dstream)

    def outputs(self):
        return [t.clone() for t in (self.result, self.dx, self.dw, self.dgamma, self.dbeta)]

    def check(self, before):
        _check_forward(self.x, self.residual, self.gamma, self.beta, self.y, self.total, self.mean, self.rstd)
        (yr, yc), (wr, wc), (dr, dc) = self.qy.values(), self.qw.values(), self.qd.values()
        check(self.result, yr, wr, what="result")
        check(self.dy, dr, wc, what="dy")
        check(self.dw, dc, yc, before, what="dw")
        _check_backward(self.total, self.dy, self.mean, self.rstd, self.gamma, self.dstream, self.dx, self.dgamma, self.dbeta)
        # the unquantized step
        s = (self.x + self.residual.float()).double()
        s.requires_grad_()
        w, gamma, beta = (t.double().requires_grad_() for t in (self.w, self.gamma, self.beta))
        d = s - s.mean(1, keepdim=True)
        y = d * (d.square().mean(1, keepdim=True) + EPS).rsqrt() * gamma + beta
        result = y @ w.T
        (result * self.dout.double()).sum().backward()
        dx = s.grad + self.dstream.double()
        for name, got, want in (("result", self.result, result), ("dx", self.dx.double() - self.dstream.double(), s.grad),
                                ("dw", self.dw.double() - before.double(), w.grad), ("dgamma", self.dgamma, gamma.grad),
                                ("dbeta", self.dbeta, beta.grad)):
            rel = float((got.double() - want.detach()).norm() / want.detach().norm())
            assert rel < 2.0 ** -4, (name, rel)
        assert float((self.dx.double() - dx).norm() / dx.norm()) < 2.0 ** -4


# a token's worth, an expert's ragged share, a batch on pairs of CTAs
@pytest.mark.parametrize("tokens,hidden,out", [(1, 256, 384), (37, 392, 520), (300, 1408, 2816), (2300, 2048, 2304)])
def test_step(tokens, hidden, out):
    step = Step(tokens, hidden, out)
    step.fill(1)
    before = step.dw.clone()
    step.run()
    step.check(before)
    want = step.outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    step.fill(2)
    before = step.dw.clone()
    graph.replay()
    step.check(before)
    step.fill(1)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(step.outputs(), want))
