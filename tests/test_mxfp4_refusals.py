"""The MXFP4 calls and the gated activation reject bad arguments on the host (no GPU work is enqueued by these calls), and the
Python functions reject tensors of another place, type or shape before the library is called."""

import ctypes

import pytest
import torch

P = ctypes.c_void_p
NULL, SHAPE, DTYPE, WORKSPACE, VALUE, ALIGN = -1, -2, -3, -5, -6, -8

fake, other = P(4096), P(8192)   # never dereferenced: validation fails first, or there is nothing to do


@pytest.fixture(scope="module")
def nvq():
    import post_nvfp4_weight_amd as m
    return m


def test_quantize(nvq):
    def f(X=fake, xd=1, n=4, k=64, ldx=64, codes=other, scales=other):
        return nvq.lib.mxfp4_quantize(X, xd, n, k, ldx, codes, scales, None)

    assert f(xd=2) == DTYPE and f(xd=-1) == DTYPE
    for bad in (dict(k=48), dict(k=0), dict(k=-32), dict(ldx=63), dict(n=-1), dict(n=1 << 31), dict(k=4000032, ldx=4000032)):
        assert f(**bad) == SHAPE, bad
    for name in ("X", "codes", "scales"):
        assert f(**{name: None}) == NULL, name
    assert f(X=P(4097)) == ALIGN and f(X=P(4098), xd=0) == ALIGN and f(codes=P(4104)) == ALIGN
    assert f(n=0, X=None, codes=None, scales=None) == 0
    assert b"mxfp4_quantize" in nvq.lib.nvq_last_error()


def test_dequantize(nvq):
    def f(codes=fake, scales=fake, n=4, k=64, out=other, od=0):
        return nvq.lib.mxfp4_dequantize(codes, scales, n, k, out, od, None)

    assert f(od=2) == DTYPE and f(k=16) == SHAPE and f(n=-1) == SHAPE
    for name in ("codes", "scales", "out"):
        assert f(**{name: None}) == NULL, name
    assert f(codes=P(4104)) == ALIGN and f(out=P(4104)) == ALIGN
    assert f(n=0, codes=None, scales=None, out=None) == 0


def test_gemm(nvq):
    def f(X=fake, xd=1, xs=None, n=4, k=64, ldx=64, codes=fake, scales=fake, m=16, Y=other, yd=0, ldy=16, ws=None, wb=0):
        return nvq.lib.mxfp4_gemm(X, xd, xs, n, k, ldx, codes, scales, m, Y, yd, ldy, ws, wb, None)

    assert f(xd=3) == DTYPE and f(yd=2) == DTYPE and f(yd=-1) == DTYPE
    for bad in (dict(k=48), dict(k=0), dict(ldx=32), dict(n=-1), dict(n=1 << 31), dict(m=0), dict(m=4000001, ldy=4000001), dict(ldy=15),
                dict(xd=2, xs=fake, ldx=96), dict(xd=2, xs=fake, ldx=32)):
        assert f(**bad) == SHAPE, bad
    for name in ("X", "codes", "scales", "Y"):
        assert f(**{name: None}) == NULL, name
    assert f(xd=2) == NULL      # codes without their scales
    assert f(X=P(4097)) == ALIGN and f(xd=2, xs=fake, X=P(4104)) == ALIGN and f(codes=P(4104)) == ALIGN and f(Y=P(4098)) == ALIGN
    assert f(Y=fake) == VALUE
    assert f(n=0, X=None, codes=None, scales=None, Y=None) == 0
    size = nvq.lib.mxfp4_gemm_workspace_size
    need = size(1, 4096, 64, 16)
    assert need >= 4096 * 34 and size(2, 0, 64, 16) == 0 and size(1, 1, 64, 16) == 0 and size(7, 4096, 64, 16) == 0
    assert f(n=4096) == WORKSPACE
    assert f(n=4096, ws=P(1 << 20), wb=need // 2) == WORKSPACE
    assert f(n=4096, ws=P((1 << 20) + 8), wb=need) == WORKSPACE


def test_gemm_dx(nvq):
    def f(dY=fake, dd=1, n=4, m=16, lddy=16, codes=fake, scales=fake, k=64, dX=other, xd=0, lddx=64, ws=None, wb=0):
        return nvq.lib.mxfp4_gemm_dx(dY, dd, n, m, lddy, codes, scales, k, dX, xd, lddx, ws, wb, None)

    assert f(dd=0) == DTYPE and f(xd=2) == DTYPE
    for bad in (dict(k=48), dict(m=0), dict(lddy=15), dict(lddx=63), dict(n=-1), dict(n=1 << 31), dict(m=4000001, lddy=4000001)):
        assert f(**bad) == SHAPE, bad
    for name in ("dY", "codes", "scales", "dX"):
        assert f(**{name: None}) == NULL, name
    assert f(dY=P(4097)) == ALIGN and f(codes=P(4104)) == ALIGN and f(dX=P(4098)) == ALIGN
    assert f(dX=fake) == VALUE
    assert f(n=0, dY=None, codes=None, scales=None, dX=None) == 0
    need = nvq.lib.mxfp4_gemm_dx_workspace_size(65536, 16, 64)
    assert need >= 16 * 64 * 2 and nvq.lib.mxfp4_gemm_dx_workspace_size(0, 16, 64) == 0
    for bad in (dict(), dict(ws=P(1 << 20), wb=16 * 64 * 2 - 1), dict(ws=P((1 << 20) + 8), wb=need)):
        assert f(n=65536, **bad) == WORKSPACE, bad


def test_swiglu(nvq):
    def f(X=fake, xd=1, n=4, h=8, ldx=16, out=other, od=1, ldo=8):
        return nvq.lib.swiglu(X, xd, n, h, ldx, out, od, ldo, None)

    assert f(xd=2) == DTYPE and f(od=2) == DTYPE
    for bad in (dict(n=-1), dict(n=1 << 31), dict(h=0), dict(ldx=15), dict(ldo=7), dict(h=4000001, ldx=1 << 30, ldo=1 << 30)):
        assert f(**bad) == SHAPE, bad
    assert f(X=None) == NULL and f(out=None) == NULL
    assert f(X=P(4097)) == ALIGN and f(out=P(4098), od=0) == ALIGN
    assert f(out=fake) == VALUE
    assert f(n=0, X=None, out=None) == 0


def test_swiglu_backward(nvq):
    def f(d=fake, ldd=8, X=fake, dt=1, n=4, h=8, ldx=16, dX=other, lddx=16):
        return nvq.lib.swiglu_backward(d, ldd, X, dt, n, h, ldx, dX, lddx, None)

    assert f(dt=2) == DTYPE
    for bad in (dict(n=-1), dict(n=1 << 31), dict(h=0), dict(ldx=15), dict(ldd=7), dict(lddx=15), dict(h=4000001, ldx=1 << 30)):
        assert f(**bad) == SHAPE, bad
    for name in ("d", "X", "dX"):
        assert f(**{name: None}) == NULL, name
    assert f(d=P(4097)) == ALIGN and f(dX=P(4098), dt=0) == ALIGN
    assert f(dX=fake) == VALUE
    assert f(n=0, d=None, X=None, dX=None) == 0


def test_python_refuses_host_tensors_and_types(nvq):
    z = torch.zeros(4, 64)
    c = torch.zeros(4, 32, dtype=torch.uint8)
    s = torch.zeros(4, 2, dtype=torch.uint8)
    for call in (lambda: nvq.mxfp4_quantize(z), lambda: nvq.mxfp4_dequantize(c, s), lambda: nvq.mxfp4_gemm(z, c, s),
                 lambda: nvq.mxfp4_gemm(c, c, s, x_scales=s), lambda: nvq.mxfp4_gemm_dx(z, c, s), lambda: nvq.swiglu(z),
                 lambda: nvq.swiglu_backward(z, z)):
        with pytest.raises(ValueError, match="HIP device"):
            call()


def test_moe_mlp(nvq):
    def f(X=fake, xd=1, T=4, d=64, ldx=64, logits=fake, ld=0, E=8, ldl=8, K=2, ids=fake, w=fake, uc=fake, us=fake, ug=fake, h=32, dc=fake,
          ds=fake, dg=fake, m=24, out=other, od=1, ldo=24, ws=P(1 << 20), wb=1 << 20):
        return nvq.lib.nvfp4_moe_mlp(X, xd, T, d, ldx, logits, ld, E, ldl, K, 1, ids, w, uc, us, ug, h, dc, ds, dg, m, out, od, ldo, ws, wb,
                                     None)

    assert f(xd=0) == DTYPE and f(ld=2) == DTYPE and f(od=2) == DTYPE
    for bad in (dict(T=-1), dict(T=65), dict(d=40), dict(d=16, ldx=16), dict(d=0), dict(ldx=48), dict(ldx=68), dict(E=0), dict(E=1025, ldl=1025), dict(ldl=7),
                dict(h=0), dict(h=16), dict(h=40), dict(m=0), dict(ldo=23), dict(T=64, ldx=1 << 25), dict(d=4000016, ldx=4000016), dict(h=4000016),
                dict(m=4000001, ldo=4000001)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(K=0), dict(K=-1), dict(K=9), dict(K=65, E=1024, ldl=1024), dict(K=65, logits=None), dict(K=1 << 40)):
        assert f(**bad) == VALUE, bad
    for name in ("X", "ids", "w", "uc", "us", "ug", "dc", "ds", "dg", "out"):
        assert f(**{name: None}) == NULL, name
    assert f(X=P(4104)) == ALIGN and f(uc=P(4100)) == ALIGN and f(dc=P(4100)) == ALIGN and f(ids=P(4098)) == ALIGN
    assert f(logits=P(4098)) == ALIGN and f(out=P(4097)) == ALIGN
    assert f(out=fake) == VALUE
    need = nvq.lib.nvfp4_moe_mlp_workspace_size(4, 8, 2, 32)
    assert need > 0 and need % 256 == 0
    for bad in ((0, 8, 2, 32), (65, 8, 2, 32), (4, 0, 2, 32), (4, 8, 0, 32), (4, 8, 65, 32), (4, 8, 2, 16), (4, 8, 2, 40)):
        assert nvq.lib.nvfp4_moe_mlp_workspace_size(*bad) == 0, bad
    assert f(ws=None) == WORKSPACE and f(wb=need - 1) == WORKSPACE and f(ws=P((1 << 20) + 8)) == WORKSPACE
    assert f(T=0, X=None, ids=None, w=None, uc=None, us=None, ug=None, dc=None, ds=None, dg=None, out=None, ws=None, wb=0) == 0
