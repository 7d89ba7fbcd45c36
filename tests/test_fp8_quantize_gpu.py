"""ufp4_fp8_quantize against its definition in 64 bits (tests/fp8_ref.py): codes and scales are exact."""
import numpy as np
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests import fp8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rand(rows, cols, seed, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * std
    return torch.where(torch.rand((rows, cols), generator=g) < 2e-3, 50 * x, x).to(dtype)


def _placed(x, ld=None, offset=0):
    rows, cols = x.shape
    ld = cols if ld is None else ld
    buf = torch.zeros(offset + rows * ld + 16, dtype=x.dtype, device=DEV)
    out = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    out.copy_(x)
    return out


def _operand(rows, cols, block, extra=16):
    """A whole buffer of 0xA5 / -1 around an operand: (all codes, all scales, qtensor); one row and some columns more."""
    pitch = (cols + 15) // 16 * 16 + extra
    codes = torch.full((rows + 1, pitch), 0xA5, dtype=torch.uint8, device=DEV)
    nb = -(-cols // 128)
    scales = torch.full((-(-rows // block) + 1, nb + 3), -1.0, device=DEV)
    return codes, scales, ufp4.QTensor(codes.data_ptr(), scales.data_ptr(), rows, cols, pitch, nb + 3)


def _check(buffers, x, block, what):
    codes, scales, _ = buffers
    rows, cols = x.shape
    c, s = ref.quantize(x, block)
    want_c, want_s = torch.full(codes.shape, 0xA5, dtype=torch.uint8), torch.full(scales.shape, -1.0)
    want_c[:rows, :cols] = c
    want_s[:s.shape[0], :s.shape[1]] = s
    assert torch.equal(torch.nan_to_num(scales.cpu(), nan=-7.0, posinf=-8.0),
                       torch.nan_to_num(want_s, nan=-7.0, posinf=-8.0)), f"{what}: scales"
    assert torch.equal(codes.cpu(), want_c), f"{what}: codes"      # and nothing beside them is written


def _run(x, block, row=True, col=True):
    rows, cols = x.shape
    r, c = _operand(rows, cols, block), _operand(cols, rows, block)
    ufp4.ufp4_fp8_quantize(x, r[2] if row else None, c[2] if col else None, block_rows=block)
    if row:
        _check(r, x.cpu(), block, "rowwise")
    if col:
        _check(c, x.cpu().T.contiguous(), block, "colwise")
    return r, c


SHAPES = [(1, 1), (1, 128), (3, 7), (7, 129), (16, 2048), (33, 100), (127, 127), (128, 128), (129, 257), (260, 1408),
          (513, 384), (1, 7168), (2049, 5)]


@pytest.mark.parametrize("outputs", ["row", "col", "both"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize(shape, dtype, block, outputs):
    x = _placed(_rand(*shape, 5 + shape[0], dtype))
    _run(x, block, row=outputs != "col", col=outputs != "row")


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ld,offset", [(None, 1), (301, 0), (304, 4), (312, 8), (320, 2)])
def test_quantize_pitches_and_offsets(dtype, ld, offset, block):
    x = _placed(_rand(140, 296, 9, dtype), ld, offset)
    _run(x, block)
    _run(x, block, col=False)


def test_every_scale_and_tie():
    """fp32 blocks over the whole exponent range (subnormal ones among them, whose scale is the least), exact ties of
    E4M3 and the values beside them, zeros and minus zeros."""
    rows = []
    for k in range(-149, 128):
        for f in (1.0, 1.75, float(np.nextafter(np.float32(1.75), np.float32(2))), 1.9999999):
            top = np.float32(min(f * 2.0 ** k, 3.4028234e38))
            t = np.concatenate([[1.0], (np.arange(1, 128) / 64.0) * 2.0 ** -(np.arange(127) % 20)]) * np.float64(top)
            t[1::2] *= -1
            rows.append(np.clip(t, -float(top), float(top)).astype(np.float32))
    ties = np.array([448.0] + [(8 + i / 2) * 2.0 ** (i % 9 - 6) for i in range(63)] + [-(i / 2) * 2.0 ** -9 for i in range(64)])
    for scale in (1.0, 2.0 ** -20, 2.0 ** 30):
        rows.append((ties * scale).astype(np.float32))
    rows.append(np.nextafter(ties.astype(np.float32), np.float32(1e9)))
    rows.append(np.zeros(128, np.float32))
    rows.append(np.full(128, -0.0, np.float32))
    x = torch.from_numpy(np.stack(rows)).to(DEV)
    r, _ = _run(x, 1)
    _run(x, 1, col=False)
    _run(x.T.contiguous(), 1)
    assert not (r[0][:, :128] == 0x80).any()


@pytest.mark.parametrize("bad", [float("nan"), -float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nonfinite_blocks(bad, block, dtype):
    x = _rand(140, 300, 5, dtype)
    x[131, 140] = bad
    x[1, 299] = bad
    _run(x.to(DEV), block)
    r, _ = _run(x.to(DEV), block, col=False)
    back = ref.restore(r[0][:140, :300], r[1][:r[1].shape[0] - 1, :3], block)
    assert torch.isnan(back[131, 128:256]).all() and torch.isfinite(back[131 if block == 1 else 2, :128]).all()


def test_empty_matrices_write_nothing():
    for shape in ((0, 40), (40, 0)):
        x = torch.zeros(shape, device=DEV)
        codes, scales, q = _operand(max(shape), max(shape), 1)
        q.rows, q.cols = shape
        ufp4.ufp4_fp8_quantize(x, q)
        assert (codes == 0xA5).all() and (scales == -1).all()


def test_many_rows():
    """More than 2^31 elements: 64-bit offsets of both outputs (sampled)."""
    rows, cols = 270_000, 8192
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    x.view(torch.int16).random_(0x3000, 0x4200)
    r, c = ufp4.alloc_fp8(rows, cols, 1, DEV), ufp4.alloc_fp8(cols, rows, 1, DEV)
    ufp4.ufp4_fp8_quantize(x, ufp4.qtensor(*r, rows, cols), ufp4.qtensor(*c, cols, rows))
    alone = ufp4.alloc_fp8(rows, cols, 1, DEV)
    ufp4.ufp4_fp8_quantize(x, ufp4.qtensor(*alone, rows, cols))
    for at in (0, 131_072, rows - 3):
        want = ref.quantize(x[at:at + 3].cpu(), 1)
        for got in (r, alone):
            assert torch.equal(got[0][at:at + 3].cpu(), want[0]) and torch.equal(got[1][at:at + 3].cpu(), want[1])
    last = rows // 128 * 128  # a short block
    want = ref.quantize(x[last:].T.contiguous().cpu(), 1)
    assert torch.equal(c[0][:, last:].cpu(), want[0]) and torch.equal(c[1][:, last // 128:].cpu(), want[1])
