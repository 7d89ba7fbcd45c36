"""The 8-bit projection and the layer norm where rows lie further apart than 32 bits reach, and with every kernel of theirs at work
at once.  Results have to be those of close rows and of calls alone, bit for bit."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests.test_fp8_gemm_gpu import make
from tests.test_layer_norm_gpu import _rows, _weights, EPS

pytestmark = pytest.mark.gpu
DEV = "cuda"


def far(t, ld):
    """The values of t, rows ld elements apart."""
    rows, cols = t.shape
    out = torch.empty((rows - 1) * ld + cols, dtype=t.dtype, device=DEV).as_strided((rows, cols), (ld, 1))
    return out.copy_(t)


def far_operand(op, ld, scales_ld):
    codes, scales = far(op[0], ld), far(op[1], scales_ld)
    return codes, scales, ufp4.qtensor(codes, scales, *op[0].shape)


# few tokens, shares of a single tile, pairs
@pytest.mark.parametrize("shape,ld", [((3, 300, 1024), 1 << 30), ((100, 300, 1024), 1 << 25), ((2304, 2304, 256), 1 << 21)])
@pytest.mark.parametrize("blocks", [(1, 128), (1, 1)])
def test_far_rows_of_a_product(shape, ld, blocks):
    m, n, k = shape
    a, b = make(m, k, blocks[0], 3), make(n, k, blocks[1], 4)
    near = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    ufp4.ufp4_fp8_gemm(a[2], b[2], near, *blocks)
    apart = 1 << 23 if n < 1000 else 1 << 21  # of B's rows: 2.5 or 4.8 GB
    fa, fb = far_operand(a, ld, ld // 4), far_operand(b, apart, apart // 8)
    d = far(torch.full_like(near, 7.0), ld)
    ufp4.ufp4_fp8_gemm(fa[2], fb[2], d, *blocks)
    assert torch.equal(d, near)


@pytest.mark.parametrize("block", [1, 128])
def test_far_rows_of_the_quantizer(block):
    x = _rows(3, 700, 5, torch.bfloat16)
    near, out = ufp4.alloc_fp8(3, 700, block, DEV), ufp4.alloc_fp8(3, 700, block, DEV)
    ufp4.ufp4_fp8_quantize(x, ufp4.qtensor(*near, 3, 700), block_rows=block)
    out = [far(t, 1 << 30) for t in out]
    ufp4.ufp4_fp8_quantize(far(x, 1 << 30), ufp4.qtensor(*out, 3, 700), block_rows=block)
    assert all(torch.equal(p, q) for p, q in zip(out, near))


@pytest.mark.parametrize("cols", [1408, 1407, 20000])
def test_far_rows_of_the_norm(cols):
    x, res = _rows(3, cols, 6, torch.bfloat16), _rows(3, cols, 7, torch.bfloat16)
    gamma, beta = _weights(cols, 8, torch.bfloat16)

    def forward(x, res, y, total):
        mean, rstd = torch.empty(3, device=DEV), torch.empty(3, device=DEV)
        ufp4.ufp4_layer_norm(x, gamma, y, mean, rstd, beta=beta, residual=res, total=total, eps=EPS)
        return y, total, mean, rstd
    ld = 1 << 30
    near = forward(x, res, torch.empty_like(x), torch.empty_like(x))
    got = forward(far(x, ld), far(res, ld), far(x, ld), far(x, ld))
    assert all(torch.equal(p, q) for p, q in zip(got, near))
    _, total, mean, rstd = near

    def backward(dy, s, dx):
        sums = [torch.empty(cols, device=DEV) for _ in range(2)]
        ws = torch.empty(ufp4.ufp4_layer_norm_backward_workspace_size(3, cols), dtype=torch.uint8, device=DEV)
        ufp4.ufp4_layer_norm_backward(dy, s, mean, rstd, gamma, dx, *sums, ws, dtotal=dy)
        return (dx, *sums)
    near = backward(res, total, torch.empty_like(x))
    got = backward(far(res, ld), far(total, ld), far(x, ld))
    assert all(torch.equal(p, q) for p, q in zip(got, near))


def test_all_kernels_at_once():
    """Products of every kind, the quantizer and the norm on streams of their own, together."""
    calls = []
    for i, (m, n, k, blocks) in enumerate([(1, 2816, 2048, (1, 128)), (30, 2816, 2048, (1, 1)), (60, 7168, 1024, (1, 128)),
                                           (200, 1408, 2048, (1, 128)), (2304, 2304, 512, (1, 128)), (2304, 2304, 512, (1, 1))]):
        a, b = make(m, k, blocks[0], 60 + i), make(n, k, blocks[1], 70 + i)
        d = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
        calls.append(([d], lambda a=a, b=b, d=d, blocks=blocks: ufp4.ufp4_fp8_gemm(a[2], b[2], d, *blocks)))
    x = _rows(1000, 1408, 9, torch.bfloat16)
    row, col = ufp4.alloc_fp8(1000, 1408, 1, DEV), ufp4.alloc_fp8(1408, 1000, 1, DEV)
    q = ufp4.qtensor(*row, 1000, 1408), ufp4.qtensor(*col, 1408, 1000)
    calls.append(([*row, *col], lambda: ufp4.ufp4_fp8_quantize(x, *q)))
    gamma, beta = _weights(1408, 10, torch.bfloat16)
    y, mean, rstd = torch.empty_like(x), torch.empty(1000, device=DEV), torch.empty(1000, device=DEV)
    calls.append(([y, mean, rstd], lambda: ufp4.ufp4_layer_norm(x, gamma, y, mean, rstd, beta=beta, eps=EPS)))
    want = []
    for out, call in calls:
        call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
        for t in out:
            t.zero_()
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (_, call) in zip(streams, calls):
            with torch.cuda.stream(st):
                call()
    torch.cuda.synchronize()
    for (out, _), alone in zip(calls, want):
        assert all(torch.equal(p, q) for p, q in zip(out, alone))
    assert ufp4.ufp4_device_error_status() == 0
