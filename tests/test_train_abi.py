"""Refusals of the training-step operators: every bad argument is an error
code before anything is launched (no GPU needed, the addresses are made up),
and the binding's own checks of shapes and types."""
import ctypes

import pytest
import torch

from rht_bit_block_gb300 import build, ufp4

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ufp4.load()


def _ckpt(rows=64, cols=96, codes=0x100000, scales=0x200000, codes_ld=None, scales_ld=None):
    return ufp4.QTensor(codes, scales, rows, cols, cols if codes_ld is None else codes_ld,
                        (cols + 31) // 32 if scales_ld is None else scales_ld)


def _ref(q):
    return ctypes.byref(q) if q is not None else None


def test_glu_refusals(lib):
    def call(gate=0x1000, ldg=96, up=0x9000, ldu=96, dt=0, rows=64, cols=96, act=0, y=0x20000, ldy=96, cg=_ckpt(),
             cu=_ckpt()):
        return lib.ufp4_glu(P(gate), ldg, P(up), ldu, dt, rows, cols, act, P(y), ldy, _ref(cg), _ref(cu), None)
    assert call(rows=0) == 0 and call(cols=0) == 0          # nothing to do
    for bad in (dict(rows=-1), dict(cols=-1), dict(dt=2), dict(act=2), dict(act=-1), dict(gate=0), dict(up=0), dict(y=0),
                dict(ldg=95), dict(ldu=95), dict(ldy=95), dict(cg=None), dict(cu=None), dict(cg=_ckpt(rows=63)),
                dict(cu=_ckpt(cols=95)), dict(cg=_ckpt(codes=0)), dict(cu=_ckpt(scales=0)), dict(cg=_ckpt(codes_ld=95)),
                dict(cu=_ckpt(scales_ld=2))):
        assert call(**bad) == 1, bad
    for bad in (dict(gate=0x1001), dict(up=0x9002, dt=1), dict(y=0x20001)):
        assert call(**bad) == 3, bad
    assert call(cols=(1 << 30) + 1) == 2


def test_glu_backward_refusals(lib):
    def call(dy=0x1000, ldd=96, dt=0, cg=_ckpt(), cu=_ckpt(), rows=64, cols=96, act=1, dg=0x20000, ldg=96, du=0x30000,
             ldu=96, y=None, ldy=0):
        return lib.ufp4_glu_backward(P(dy), ldd, dt, _ref(cg), _ref(cu), rows, cols, act, P(dg), ldg, P(du), ldu, P(y),
                                     ldy, None)
    assert call(rows=0) == 0
    for bad in (dict(rows=-1), dict(dt=-1), dict(act=7), dict(dy=0), dict(cg=None), dict(cu=None), dict(dg=0), dict(du=0),
                dict(ldd=1), dict(ldg=1), dict(ldu=1), dict(y=0x40000, ldy=95), dict(cg=_ckpt(rows=1))):
        assert call(**bad) == 1, bad
    assert call(dy=0x1002, dt=1) == 3 and call(dg=0x20001) == 3 and call(y=0x40001, ldy=96) == 3


def test_rms_norm_refusals(lib):
    def call(x=0x1000, ldx=96, dt=0, res=None, ldr=0, gamma=0x5000, gt=1, rows=64, cols=96, eps=1e-6, y=0x20000, ldy=96,
             tot=None, ldt=0, rstd=0x6000, ck=_ckpt()):
        return lib.ufp4_rms_norm(P(x), ldx, dt, P(res), ldr, P(gamma), gt, rows, cols, eps, P(y), ldy, P(tot), ldt,
                                 P(rstd), _ref(ck), None)
    assert call(rows=0) == 0
    for bad in (dict(rows=-1), dict(cols=0), dict(dt=3), dict(gt=3), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(x=0), dict(gamma=0), dict(y=0), dict(rstd=0),
                dict(ldx=95), dict(ldy=95), dict(res=0x70000, ldr=95), dict(tot=0x70000, ldt=95), dict(ck=_ckpt(cols=95))):
        assert call(**bad) == 1, bad
    assert call(cols=32769, ldx=40000, ldy=40000, ck=None) == 2
    assert call(x=0x1001) == 3 and call(gamma=0x5002) == 3 and call(rstd=0x6002) == 3


def test_rms_norm_backward_refusals(lib):
    size = ctypes.c_size_t(0)
    assert lib.ufp4_rms_norm_backward_workspace_size(64, 96, ctypes.byref(size)) == 0
    assert size.value >= 96 * 4
    assert lib.ufp4_rms_norm_backward_workspace_size(-1, 96, ctypes.byref(size)) == 1
    assert lib.ufp4_rms_norm_backward_workspace_size(1, 0, ctypes.byref(size)) == 1
    assert lib.ufp4_rms_norm_backward_workspace_size(1, 96, None) == 1
    assert lib.ufp4_rms_norm_backward_workspace_size(1, 32769, ctypes.byref(size)) == 2

    def call(dy=0x1000, ldd=96, dt=0, ck=_ckpt(), rstd=0x6000, gamma=0x5000, gt=0, dtot=None, ldt=0, rows=64, cols=96,
             dx=0x20000, ldx=96, dg=0x7000, y=None, ldy=0, ws=0x80000, n=1 << 24):
        return lib.ufp4_rms_norm_backward(P(dy), ldd, dt, _ref(ck), P(rstd), P(gamma), gt, P(dtot), ldt, rows, cols,
                                          P(dx), ldx, P(dg), P(y), ldy, P(ws), n, None)
    for bad in (dict(rows=-1), dict(cols=0), dict(dt=2), dict(gt=2), dict(dy=0), dict(ck=None), dict(rstd=0),
                dict(gamma=0), dict(dx=0), dict(dg=0), dict(ws=0), dict(n=64), dict(ldd=95), dict(ldx=95),
                dict(dtot=0x90000, ldt=95), dict(y=0x90000, ldy=95)):
        assert call(**bad) == 1, bad
    assert call(ws=0x80010) == 3 and call(dg=0x7002) == 3 and call(cols=40000) == 2


def test_head_loss_refusals(lib):
    size = ctypes.c_size_t(0)
    for f in (lib.ufp4_head_loss_workspace_size, lib.ufp4_head_loss_backward_workspace_size):
        assert f(64, 1000, 128, ctypes.byref(size)) == 0 and size.value > 0
        assert f(0, 1000, 128, ctypes.byref(size)) == 0 and size.value > 0
        assert f(-1, 1000, 128, ctypes.byref(size)) == 1
        assert f(64, 0, 128, ctypes.byref(size)) == 1
        assert f(64, 1000, 0, ctypes.byref(size)) == 1
        assert f(64, 1000, 128, None) == 1
        assert f((1 << 30) + 1, 1000, 128, ctypes.byref(size)) == 2

    def fwd(h=0x1000, ldh=128, w=0x90000, ldw=128, t=0x8000, T=64, V=1000, K=128, z=0.0, loss=0xA000, lse=0xB000,
            ws=0x100000, n=1 << 40):
        return lib.ufp4_head_loss(P(h), ldh, P(w), ldw, P(t), T, V, K, z, P(loss), P(lse), P(ws), n, None)
    assert fwd(T=0, h=0, t=0, loss=0, lse=0, ws=0) == 0        # no tokens: nothing to do
    for bad in (dict(T=-1), dict(V=0), dict(K=0), dict(h=0), dict(w=0), dict(t=0), dict(loss=0), dict(lse=0), dict(ws=0),
                dict(n=1024), dict(ldh=120), dict(ldw=120), dict(z=float("nan")), dict(z=float("inf"))):
        assert fwd(**bad) == 1, bad
    for bad in (dict(h=0x1008), dict(w=0x90002), dict(ldh=130), dict(ldw=132), dict(t=0x8004), dict(loss=0xA002),
                dict(lse=0xB001), dict(ws=0x100080)):
        assert fwd(**bad) == 3, bad
    assert fwd(V=(1 << 30) + 1) == 2 and fwd(T=1 << 24, V=1 << 24) == 2   # extents, and tiles of the product

    def bwd(lse=0xB000, weight=None, scale=None, dh=0x20000, ldd=128, ht=0, dw=0x30000, ldw=128, wt=0, acc=0,
            ws=0x100000, n=1 << 40, T=64):
        return lib.ufp4_head_loss_backward(P(0x1000), 128, P(0x90000), 128, P(0x8000), T, 1000, 128, 0.0, P(lse),
                                           P(weight), P(scale), P(dh), ldd, ht, P(dw), ldw, wt, acc, P(ws), n, None)
    for bad in (dict(lse=0), dict(dh=0, dw=0), dict(ht=2), dict(wt=-1), dict(acc=2), dict(ldd=127), dict(ldw=127),
                dict(ws=0), dict(n=1024)):
        assert bwd(**bad) == 1, bad
    assert bwd(acc=1) == 2                                     # only an fp32 dw is added to
    for bad in (dict(weight=0x2), dict(scale=0x2), dict(dh=0x20001), dict(dw=0x30002, wt=1), dict(ws=0x100010)):
        assert bwd(**bad) == 3, bad


def test_binding_checks_shapes_and_types(lib):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ufp4.ufp4_glu(x, x[:, :32], x)
    with pytest.raises(TypeError):
        ufp4.ufp4_glu(x.half(), x.half(), x)
    with pytest.raises(TypeError):
        ufp4.ufp4_glu(x, x.float(), x)
    with pytest.raises(ValueError):
        ufp4.ufp4_glu(x.T.contiguous().T, x, x)              # columns are strided
    with pytest.raises(TypeError):
        ufp4.ufp4_rms_norm(x, x[0], x.float())
    with pytest.raises(ValueError):
        ufp4.ufp4_rms_norm(x, x[0, :32], x)
    with pytest.raises(TypeError):
        ufp4.ufp4_head_loss(x, x, torch.zeros(4, dtype=torch.int32), x[0], x[0], x)
