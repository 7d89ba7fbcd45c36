"""ufp4_fp8_gemm against the 64-bit product of the restored operands.

Tolerances.  With S the sum of the products' magnitudes: a block's 128 products (each exact) are summed by four tensor
core instructions that keep at least 22 bits of the largest term, 4 * 2^-21 of S; the scaled additions round once a block
and once for each scale, (blocks + 3) 2^-24 of S.  A bf16 result adds half a step, 2^-8 of itself."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests import fp8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(rows, cols, block, seed, spread=3.0):
    """A random operand: every code byte but the NaNs, log-normal scales; (codes, scales, qtensor, values in 64 bits)."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 256, (rows, cols), generator=g, dtype=torch.uint8)
    c = torch.where((c & 0x7F) == 0x7F, torch.zeros_like(c), c)
    s = torch.exp(torch.randn((-(-rows // block), -(-cols // 128)), generator=g) * spread) * 1e-3
    codes, scales = ufp4.alloc_fp8(rows, cols, block, DEV)
    codes.copy_(c)
    scales.copy_(s)
    return codes, scales, ufp4.qtensor(codes, scales, rows, cols), ref.restore(c, s, block).to(DEV)


def check(d, a, b, before=None, what=""):
    want = a @ b.T
    if before is not None:
        want = want + before.double()
    s = a.abs() @ b.abs().T
    blocks = -(-a.shape[1] // 128)
    lim = (4 * 2.0 ** -21 + (blocks + 3) * 2.0 ** -24) * s + 1e-30
    if before is not None:
        lim = lim + 2.0 ** -24 * (want.abs() + before.double().abs())
    if d.dtype == torch.bfloat16:
        lim = lim * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    bad = ~((d.double() - want).abs() <= lim)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {tuple(bad.nonzero()[0].tolist())}: "
                           f"{d[bad][0].item()} for {want[bad][0].item()}, worst {float(((d.double() - want).abs() / s).max())} of S")


# one token to many, odd and even, around the tiles' edges, blocks that end short, one and several shares, pairs
SHAPES = [(1, 1, 1), (1, 128, 128), (1, 130, 7), (3, 257, 1000), (16, 129, 640), (17, 2048, 512), (33, 500, 333),
          (64, 1408, 2048), (65, 300, 129), (100, 1000, 4109), (128, 128, 256), (129, 127, 384), (200, 2816, 130),
          (256, 256, 1024), (300, 4000, 257), (777, 1999, 1111), (2000, 2050, 129), (2304, 2304, 640), (5, 20000, 256)]


@pytest.mark.parametrize("blocks", [(1, 128), (1, 1), (128, 128), (128, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_product(shape, dtype, blocks):
    m, n, k = shape
    a, b = make(m, k, blocks[0], 1 + m), make(n, k, blocks[1], 2 + n)
    d = torch.full((m + 1, n + 3), 7.0, dtype=dtype, device=DEV)
    ufp4.ufp4_fp8_gemm(a[2], b[2], d[:m, :n], *blocks)
    check(d[:m, :n], a[3], b[3])
    assert (d[m] == 7).all() and (d[:, n:] == 7).all()


@pytest.mark.parametrize("shape", [(1, 200, 500), (40, 300, 700), (600, 700, 300), (2100, 2300, 200)])
@pytest.mark.parametrize("blocks", [(1, 128), (1, 1)])
def test_accumulate(shape, blocks):
    m, n, k = shape
    a, b = make(m, k, blocks[0], 3, 0.5), make(n, k, blocks[1], 4, 0.5)
    d = torch.randn((m, n), device=DEV)
    before = d.clone()
    ufp4.ufp4_fp8_gemm(a[2], b[2], d, *blocks, accumulate=True)
    check(d, a[3], b[3], before)


@pytest.mark.parametrize("shape", [(1, 300, 2048), (48, 1408, 2048), (100, 512, 4096), (500, 600, 640), (2304, 2560, 512)])
def test_same_bits_every_time(shape):
    m, n, k = shape
    a, b = make(m, k, 1, 5), make(n, k, 128, 6)
    d = [torch.empty((m, n), device=DEV) for _ in range(4)]
    for t in d:
        ufp4.ufp4_fp8_gemm(a[2], b[2], t)
    assert all(torch.equal(t, d[0]) for t in d)


def test_whole_numbers_are_exact():
    """Codes of small whole numbers and scales of powers of two: every sum is exact in fp32."""
    g = torch.Generator().manual_seed(7)
    for m, n, k in ((5, 300, 1000), (128, 640, 384), (2200, 2400, 512)):
        ops = []
        for rows, block in ((m, 1), (n, 128)):
            v = torch.randint(-4, 5, (rows, k), generator=g).float()
            s = torch.pow(2.0, torch.randint(-2, 3, (-(-rows // block), -(-k // 128)), generator=g).float())
            codes, scales = ufp4.alloc_fp8(rows, k, block, DEV)
            codes.copy_(v.to(torch.float8_e4m3fn).view(torch.uint8))
            scales.copy_(s)
            ops.append((codes, scales, ufp4.qtensor(codes, scales, rows, k), ref.restore(codes, scales, block).to(DEV)))
        d = torch.empty((m, n), device=DEV)
        ufp4.ufp4_fp8_gemm(ops[0][2], ops[1][2], d)
        assert torch.equal(d.double(), ops[0][3] @ ops[1][3].T)


def test_nan_stays_in_its_row_and_column():
    for m, n, k in ((20, 300, 500), (150, 300, 500), (2300, 2400, 300)):
        a, b = make(m, k, 1, 8, 0.5), make(n, k, 128, 9, 0.5)
        a[0][7, 130] = 0x7F
        b[0][200, 3] = 0xFF
        d = torch.empty((m, n), device=DEV)
        ufp4.ufp4_fp8_gemm(a[2], b[2], d)
        want = torch.zeros((m, n), dtype=torch.bool, device=DEV)
        want[7] = want[:, 200] = True
        assert torch.equal(torch.isnan(d), want)


def test_bytes_behind_the_columns_are_not_read():
    """NaN codes and scales behind K, in the pitch."""
    m, n, k = 40, 200, 300
    a, b = make(m, k, 1, 10), make(n, k, 128, 11)
    ops = []
    for codes, scales, _, v in (a, b):
        c = torch.full((codes.shape[0], 400), 0x7F, dtype=torch.uint8, device=DEV)
        s = torch.full((scales.shape[0], 7), float("nan"), device=DEV)
        c[:, :k] = codes
        s[:, :3] = scales
        ops.append((c, s, ufp4.QTensor(c.data_ptr(), s.data_ptr(), codes.shape[0], k, 400, 7)))
    d = torch.empty((m, n), device=DEV)
    ufp4.ufp4_fp8_gemm(ops[0][2], ops[1][2], d)
    check(d, a[3], b[3])


def test_no_columns_and_no_rows():
    q = ufp4.QTensor(0, 0, 5, 0, 0, 0)
    d = torch.full((5, 9), 3.0, device=DEV)
    ufp4.ufp4_fp8_gemm(q, q, d[:, 2:7], 1, 1, accumulate=True)
    assert (d == 3).all()
    ufp4.ufp4_fp8_gemm(q, q, d[:, 2:7], 1, 1)
    assert (d[:, 2:7] == 0).all() and (d[:, :2] == 3).all() and (d[:, 7:] == 3).all()
    empty = ufp4.QTensor(0, 0, 0, 64, 64, 1)
    ufp4.ufp4_fp8_gemm(empty, ufp4.QTensor(0, 0, 5, 64, 64, 1), torch.empty((0, 5), device=DEV))


@pytest.mark.parametrize("shape", [(2, 640, 1024), (90, 400, 1024), (2304, 2304, 256)])
def test_streams_and_captured_graphs(shape):
    """Calls on two streams at once, and one captured and replayed on new values of the same operands."""
    m, n, k = shape
    ops = [(make(m, k, 1, 20 + i), make(n, k, 128, 30 + i)) for i in range(2)]
    alone = []
    for a, b in ops:
        d = torch.empty((m, n), device=DEV)
        ufp4.ufp4_fp8_gemm(a[2], b[2], d)
        alone.append(d)
    torch.cuda.synchronize()
    streams, out = [torch.cuda.Stream() for _ in range(2)], [torch.empty((m, n), device=DEV) for _ in range(2)]
    for _ in range(5):
        for st, (a, b), d in zip(streams, ops, out):
            with torch.cuda.stream(st):
                ufp4.ufp4_fp8_gemm(a[2], b[2], d)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, alone))
    (a, b), (a2, b2) = ops
    graph, d = torch.cuda.CUDAGraph(), torch.empty((m, n), device=DEV)
    with torch.cuda.graph(graph):
        ufp4.ufp4_fp8_gemm(a[2], b[2], d)
    for mine, other in ((a, a2), (b, b2)):
        mine[0].copy_(other[0])
        mine[1].copy_(other[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(d, alone[1])


def test_quantized_linear_layer():
    """FPROP, DGRAD and WGRAD of a linear layer on its quantized operands."""
    t, out, inp = 300, 520, 392
    g = torch.Generator().manual_seed(40)
    x, w, dy = (torch.randn(s, generator=g).to(DEV, torch.bfloat16) for s in ((t, inp), (out, inp), (t, out)))

    def both(v, block):
        rows, cols = v.shape
        r, c = ufp4.alloc_fp8(rows, cols, block, DEV), ufp4.alloc_fp8(cols, rows, block, DEV)
        qr, qc = ufp4.qtensor(*r, rows, cols), ufp4.qtensor(*c, cols, rows)
        ufp4.ufp4_fp8_quantize(v, qr, qc, block_rows=block)
        kept.append((r, c))  # a qtensor holds addresses only
        return (qr, ref.restore(*r, block).to(DEV)), (qc, ref.restore(*c, block).to(DEV))
    kept = []
    (xr, xrv), (xc, xcv) = both(x, 1)
    (wr, wrv), (wc, wcv) = both(w, 128)
    (dr, drv), (dc, dcv) = both(dy, 1)
    assert torch.equal(wrv, wcv.T)
    y, dx = (torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in ((t, out), (t, inp)))
    dw = torch.empty((out, inp), device=DEV)
    ufp4.ufp4_fp8_gemm(xr, wr, y)
    ufp4.ufp4_fp8_gemm(dr, wc, dx)
    ufp4.ufp4_fp8_gemm(dc, xc, dw, b_block_rows=1)
    check(y, xrv, wrv, what="y")
    check(dx, drv, wcv, what="dx")
    check(dw, dcv, xcv, what="dw")
    # against the unquantized layer: E4M3 keeps 4 bits, 2^-4 of an element at most, about a third of it in the mean
    # square, of either operand, and products add up with random signs
    for got, want in ((y, x.double() @ w.double().T), (dx, dy.double() @ w.double()), (dw, dy.double().T @ x.double())):
        assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -4
