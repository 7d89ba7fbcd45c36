"""The binding's check that an 8-bit operand's scales are those of the block_rows it is used with (no GPU needed: the library is
not called, or its call is recorded)."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4


@pytest.fixture
def calls(monkeypatch):
    """Host tensors pass for the device's; the library's calls are recorded."""
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: made.append(name) or 0
    monkeypatch.setattr(ufp4, "_stream", lambda s: 0)
    monkeypatch.setattr(ufp4, "_check_devices", lambda *a: None)
    monkeypatch.setattr(ufp4, "load", lambda: Library())
    return made


def _operand(rows, cols, block):
    return ufp4.qtensor(*ufp4.alloc_fp8(rows, cols, block, "cpu"), rows, cols)


@pytest.mark.parametrize("rows,cols", [(2, 1), (7, 300), (128, 128), (129, 257), (300, 128)])
def test_quantizer_takes_what_the_operand_was_allocated_for(calls, rows, cols):
    x = torch.zeros((rows, cols))
    for block, other in ((1, 128), (128, 1)):
        row, col = _operand(rows, cols, block), _operand(cols, rows, block)
        ufp4.ufp4_fp8_quantize(x, row, col, block_rows=block)
        ufp4.ufp4_fp8_quantize(x, row, None, block_rows=block)
        with pytest.raises(ValueError, match="rowwise"):
            ufp4.ufp4_fp8_quantize(x, row, None, block_rows=other)
        if cols > 1:
            with pytest.raises(ValueError, match="colwise"):
                ufp4.ufp4_fp8_quantize(x, None, col, block_rows=other)
    with pytest.raises(ValueError):
        ufp4.ufp4_fp8_quantize(x, _operand(rows, cols, 128))      # the default is 1
    assert len(calls) == 4


def test_one_row_is_the_same_in_either_block(calls):
    x = torch.zeros((1, 300))
    for block in (1, 128):
        ufp4.ufp4_fp8_quantize(x, _operand(1, 300, 129 - block), block_rows=block)
    assert len(calls) == 2


@pytest.mark.parametrize("a,b", [(1, 1), (1, 128), (128, 1), (128, 128)])
def test_product_takes_what_its_operands_were_quantized_with(calls, a, b):
    A, B, d = _operand(40, 300, a), _operand(200, 300, b), torch.zeros((40, 200))
    for ga in (1, 128):
        for gb in (1, 128):
            if (ga, gb) == (a, b):
                ufp4.ufp4_fp8_gemm(A, B, d, ga, gb)
            else:
                with pytest.raises(ValueError, match="A has" if ga != a else "B has"):
                    ufp4.ufp4_fp8_gemm(A, B, d, ga, gb)
    assert calls == ["ufp4_fp8_gemm"]


def test_a_weight_gradient_needs_its_block_rows(calls):
    A, B = _operand(64, 300, 1), _operand(96, 300, 1)
    with pytest.raises(ValueError, match="B has scales .* block_rows is 1"):
        ufp4.ufp4_fp8_gemm(A, B, torch.zeros((64, 96)))
    ufp4.ufp4_fp8_gemm(A, B, torch.zeros((64, 96)), b_block_rows=1)


def test_scales_of_too_few_columns_or_another_type(calls):
    codes, scales = ufp4.alloc_fp8(40, 300, 1, "cpu")
    x = torch.zeros((40, 300))
    with pytest.raises(ValueError, match="too few"):
        ufp4.ufp4_fp8_quantize(x, ufp4.qtensor(codes, scales[:, :2], 40, 300))
    with pytest.raises(ValueError, match="too few"):
        ufp4.ufp4_fp8_quantize(x, ufp4.qtensor(codes, scales[:39], 40, 300))
    for other in (torch.bfloat16, torch.uint8, torch.float64):
        with pytest.raises(TypeError, match="float32 scales"):
            ufp4.ufp4_fp8_quantize(x, ufp4.qtensor(codes, scales.to(other), 40, 300))
    with pytest.raises(TypeError, match="one byte"):
        ufp4.ufp4_fp8_quantize(x, ufp4.qtensor(codes.short(), scales, 40, 300))
    ufp4.ufp4_fp8_quantize(x, ufp4.qtensor(codes.view(torch.float8_e4m3fn), scales, 40, 300))
    assert len(calls) == 1


def test_room_for_more_and_addresses_alone_are_taken(calls):
    """Scales of more rows than the operand has, as a buffer for the most tokens is used; a QTensor that no tensors made; none
    of either kind of rows."""
    codes, scales = ufp4.alloc_fp8(500, 300, 1, "cpu")
    ufp4.ufp4_fp8_quantize(torch.zeros((40, 300)), ufp4.qtensor(codes, scales, 40, 300))
    codes, scales = ufp4.alloc_fp8(500, 300, 128, "cpu")
    ufp4.ufp4_fp8_quantize(torch.zeros((40, 300)), ufp4.qtensor(codes, scales, 40, 300), block_rows=128)
    bare = ufp4.QTensor(codes.data_ptr(), scales.data_ptr(), 40, 300, 304, 3)
    ufp4.ufp4_fp8_quantize(torch.zeros((40, 300)), bare)
    ufp4.ufp4_fp8_quantize(torch.zeros((40, 300)), bare, block_rows=128)
    ufp4.ufp4_fp8_quantize(torch.zeros((0, 300)), _operand(0, 300, 128))
    # one block of columns: its scales may be one dimension
    ufp4.ufp4_fp8_quantize(torch.zeros((40, 100)), ufp4.qtensor(codes[:40], torch.zeros(40), 40, 100))
    assert len(calls) == 6


def test_other_block_rows_are_left_to_the_library():
    from rht_bit_block_gb300 import build
    build.build()
    q = _operand(40, 300, 1)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(ufp4, "_stream", lambda s: 0)
        m.setattr(ufp4, "_check_devices", lambda *a: None)
        for block in (0, 32, -1):
            with pytest.raises(ufp4.Ufp4Error) as e:
                ufp4.ufp4_fp8_quantize(torch.zeros((40, 300)), q, block_rows=block)
            assert e.value.status == 1
