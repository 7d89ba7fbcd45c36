"""Refusals of the 8-bit operands' and the layer norm's entry points: every bad argument is an error code before
anything is launched (no GPU needed, the addresses are made up), and the binding's own checks."""
import ctypes

import pytest
import torch

from rht_bit_block_gb300 import build, ufp4

P = ctypes.c_void_p


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return ufp4.load()


def _op(rows=64, cols=300, codes=0x100000, scales=0x200000, codes_ld=304, scales_ld=3):
    return ufp4.QTensor(codes, scales, rows, cols, codes_ld, scales_ld)


def _ref(q):
    return ctypes.byref(q) if q is not None else None


def test_quantize_refusals(lib):
    def call(x=0x1000, ld=300, dt=0, rows=64, cols=300, block=1, row=_op(), col=_op(300, 64, codes_ld=64, scales_ld=1)):
        return lib.ufp4_fp8_quantize(P(x), ld, dt, rows, cols, block, _ref(row), _ref(col), None)
    assert call(rows=0) == 0 and call(cols=0) == 0 and call(rows=0, x=0) == 0      # nothing to do
    for bad in (dict(rows=-1), dict(cols=-1), dict(dt=2), dict(dt=-1), dict(block=0), dict(block=32), dict(block=64),
                dict(row=None, col=None), dict(x=0), dict(ld=299), dict(row=_op(rows=63)), dict(row=_op(cols=299)),
                dict(row=_op(codes=0)), dict(row=_op(scales=0)), dict(row=_op(codes_ld=288)), dict(row=_op(scales_ld=2)),
                dict(col=_op()), dict(col=_op(300, 64, codes_ld=48, scales_ld=1)), dict(col=_op(300, 64, codes_ld=64, scales_ld=0))):
        assert call(**bad) == 1, bad
    for bad in (dict(x=0x1001), dict(x=0x1002, dt=1), dict(row=_op(codes=0x100008)), dict(row=_op(codes_ld=312)),
                dict(row=_op(scales=0x200002)), dict(col=_op(300, 64, codes=0x100001, codes_ld=64, scales_ld=1))):
        assert call(**bad) == 3, bad
    assert call(rows=(1 << 30) + 1) == 2 and call(cols=(1 << 30) + 1, ld=1 << 31) == 2


def test_gemm_refusals(lib):
    def call(a=_op(), ab=1, b=_op(90, 300), bb=128, d=0x300000, ldd=90, dt=0, acc=0):
        return lib.ufp4_fp8_gemm(_ref(a), ab, _ref(b), bb, P(d), ldd, dt, acc, None)
    assert call(a=_op(rows=0)) == 0 and call(b=_op(0, 300), ldd=0) == 0              # no results
    for bad in (dict(a=None), dict(b=None), dict(ab=0), dict(ab=2), dict(bb=64), dict(dt=2), dict(acc=2), dict(acc=-1),
                dict(a=_op(rows=-1)), dict(b=_op(-1, 300)), dict(b=_op(90, 299)), dict(a=_op(cols=-5), b=_op(90, -5)),
                dict(d=0), dict(ldd=89), dict(a=_op(codes=0)), dict(b=_op(90, 300, scales=0)), dict(a=_op(codes_ld=288)),
                dict(b=_op(90, 300, scales_ld=2))):
        assert call(**bad) == 1, bad
    assert call(acc=1) == 2                                                          # only an fp32 D is added to
    for bad in (dict(d=0x300001), dict(d=0x300002, dt=1), dict(a=_op(codes=0x100004)), dict(b=_op(90, 300, codes_ld=308)),
                dict(a=_op(scales=0x200001))):
        assert call(**bad) == 3, bad
    assert call(a=_op((1 << 30) + 1)) == 2
    assert call(a=_op(1 << 24), b=_op(1 << 24, 300), ldd=1 << 24) == 2               # tiles
    # no sum and accumulation: D stays; its operands are not looked at
    assert call(a=_op(cols=0, codes=0), b=_op(90, 0, codes=0), dt=1, acc=1) == 0


def test_layer_norm_refusals(lib):
    def call(x=0x1000, ldx=96, dt=0, res=None, ldr=0, gamma=0x5000, beta=0x5800, gt=1, rows=64, cols=96, eps=1e-5, y=0x20000,
             ldy=96, tot=None, ldt=0, mean=0x6000, rstd=0x7000):
        return lib.ufp4_layer_norm(P(x), ldx, dt, P(res), ldr, P(gamma), P(beta), gt, rows, cols, eps, P(y), ldy, P(tot), ldt,
                                   P(mean), P(rstd), None)
    assert call(rows=0) == 0
    for bad in (dict(rows=-1), dict(cols=0), dict(dt=3), dict(gt=3), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(x=0), dict(gamma=0), dict(y=0), dict(ldx=95), dict(ldy=95),
                dict(res=0x70000, ldr=95), dict(tot=0x70000, ldt=95)):
        assert call(**bad) == 1, bad
    assert call(cols=32769, ldx=40000, ldy=40000) == 2
    for bad in (dict(x=0x1001), dict(gamma=0x5002), dict(beta=0x5802), dict(mean=0x6002), dict(rstd=0x7001), dict(y=0x20001)):
        assert call(**bad) == 3, bad


def test_layer_norm_backward_refusals(lib):
    size = ctypes.c_size_t(0)
    f = lib.ufp4_layer_norm_backward_workspace_size
    assert f(64, 96, ctypes.byref(size)) == 0 and size.value >= 2 * 96 * 4
    assert f(0, 96, ctypes.byref(size)) == 0 and size.value >= 2 * 96 * 4
    assert f(-1, 96, ctypes.byref(size)) == 1 and f(1, 0, ctypes.byref(size)) == 1 and f(1, 96, None) == 1
    assert f(1, 32769, ctypes.byref(size)) == 2

    def call(dy=0x1000, ldd=96, dt=0, x=0x9000, ldx=96, xt=0, mean=0x6000, rstd=0x6400, gamma=0x5000, gt=0, dtot=None, ldt=0,
             rows=64, cols=96, dx=0x20000, ldo=96, dg=0x7000, db=0x7400, ws=0x80000, n=1 << 24):
        return lib.ufp4_layer_norm_backward(P(dy), ldd, dt, P(x), ldx, xt, P(mean), P(rstd), P(gamma), gt, P(dtot), ldt, rows,
                                            cols, P(dx), ldo, P(dg), P(db), P(ws), n, None)
    for bad in (dict(rows=-1), dict(cols=0), dict(dt=2), dict(xt=-1), dict(gt=2), dict(dy=0), dict(x=0), dict(mean=0),
                dict(rstd=0), dict(gamma=0), dict(dx=0), dict(dg=0), dict(db=0), dict(ws=0), dict(n=64), dict(ldd=95),
                dict(ldx=95), dict(ldo=95), dict(dtot=0x90000, ldt=95)):
        assert call(**bad) == 1, bad
    for bad in (dict(ws=0x80010), dict(dg=0x7002), dict(db=0x7401), dict(dy=0x1001), dict(x=0x9002, xt=1), dict(mean=0x6001)):
        assert call(**bad) == 3, bad
    assert call(cols=40000) == 2


def _host_calls():
    m, v, g = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros(4), torch.ones(64)
    codes, scales = ufp4.alloc_fp8(4, 64, 1, "cpu")
    q = ufp4.qtensor(codes, scales, 4, 64)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    return {
        "quantize": lambda: ufp4.ufp4_fp8_quantize(m, q),
        "gemm": lambda: ufp4.ufp4_fp8_gemm(q, q, torch.zeros((4, 4)), b_block_rows=1),
        "norm": lambda: ufp4.ufp4_layer_norm(m, g, m.clone(), v, v.clone(), beta=g, residual=m, total=m.clone()),
        "norm_backward": lambda: ufp4.ufp4_layer_norm_backward(m, m, v, v, g, m.clone(), g.clone(), g.clone(), ws, dtotal=m),
    }


@pytest.mark.parametrize("name", list(_host_calls()))
def test_host_tensors_are_refused(name, monkeypatch):
    monkeypatch.setattr(ufp4, "_stream", lambda s: 0)
    monkeypatch.setattr(ufp4, "load", lambda: pytest.fail("the library was called"))
    with pytest.raises(ValueError, match="host memory"):
        _host_calls()[name]()


def test_binding_checks_shapes_and_types():
    x, v, g = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros(4), torch.ones(64)
    q = ufp4.qtensor(*ufp4.alloc_fp8(4, 64, 1, "cpu"), 4, 64)
    with pytest.raises(TypeError):
        ufp4.ufp4_fp8_quantize(x.half(), q)
    with pytest.raises(ValueError):
        ufp4.ufp4_fp8_quantize(x.T.contiguous().T, q)            # columns are strided
    with pytest.raises(ValueError):
        ufp4.ufp4_fp8_gemm(q, q, torch.zeros((4, 5)))
    with pytest.raises(TypeError):
        ufp4.ufp4_fp8_gemm(q, q, torch.zeros((4, 4), dtype=torch.float16))
    with pytest.raises(TypeError):
        ufp4.ufp4_layer_norm(x, g, x, beta=g.bfloat16())         # gamma's type
    with pytest.raises(ValueError):
        ufp4.ufp4_layer_norm(x, g[:32], x)
    with pytest.raises(TypeError):
        ufp4.ufp4_layer_norm(x, g, x.float())
    with pytest.raises(ValueError):
        ufp4.ufp4_layer_norm_backward(x, x[:, :32], v, v, g, x, g, g, torch.zeros(1, dtype=torch.uint8))
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 20, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            ufp4.ufp4_layer_norm_backward(x, x, v, v, g, x, g, g, ws)


@pytest.mark.parametrize("rows,cols,block", [(1, 1, 1), (7, 300, 1), (129, 257, 128)])
def test_alloc_fp8(rows, cols, block):
    codes, scales = ufp4.alloc_fp8(rows, cols, block, "cpu")
    q = ufp4.qtensor(codes, scales, rows, cols)
    assert codes.shape == (rows, cols) and q.codes_ld % 16 == 0 and q.codes_ld >= cols
    assert scales.shape == (-(-rows // block), -(-cols // 128)) and scales.dtype == torch.float32
