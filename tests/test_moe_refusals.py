"""The mixture-of-experts calls reject bad arguments on the host (no GPU work is enqueued by these calls), and the Python
functions reject tensors of another place, type or shape before the library is called."""

import ctypes

import pytest
import torch

P = ctypes.c_void_p
NULL, SHAPE, DTYPE, WORKSPACE, VALUE, ALIGN = -1, -2, -3, -5, -6, -8


@pytest.fixture(scope="module")
def nvq():
    import post_nvfp4_weight_amd as m
    return m


fake = P(4096)   # never dereferenced: validation fails first, or there is nothing to do


def test_topk(nvq):
    f = nvq.lib.moe_topk
    assert f(fake, 2, 4, 8, 8, 2, 1, fake, fake, None) == DTYPE
    assert f(fake, 0, -1, 8, 8, 2, 1, fake, fake, None) == SHAPE
    assert f(fake, 0, 1 << 31, 8, 8, 2, 1, fake, fake, None) == SHAPE
    assert f(fake, 0, 4, 0, 8, 1, 1, fake, fake, None) == SHAPE
    assert f(fake, 0, 4, 1025, 1025, 2, 1, fake, fake, None) == SHAPE
    assert f(fake, 0, 4, 8, 7, 2, 1, fake, fake, None) == SHAPE
    for k in (0, -1, 9):
        assert f(fake, 0, 4, 8, 8, k, 1, fake, fake, None) == VALUE
    assert f(fake, 0, 4, 1024, 1024, 65, 1, fake, fake, None) == VALUE
    for bad in ((None, fake, fake), (fake, None, fake), (fake, fake, None)):
        assert f(bad[0], 0, 4, 8, 8, 2, 1, bad[1], bad[2], None) == NULL
    assert f(P(4098), 0, 4, 8, 8, 2, 1, fake, fake, None) == ALIGN
    assert f(P(4097), 1, 4, 8, 8, 2, 1, fake, fake, None) == ALIGN
    assert f(None, 0, 0, 8, 8, 2, 1, None, None, None) == 0
    assert b"moe_topk" in nvq.lib.nvq_last_error()


def test_topk_backward(nvq):
    f = nvq.lib.moe_topk_backward
    assert f(fake, 5, 4, 8, 8, fake, fake, fake, 2, 1, fake, 8, None) == DTYPE
    assert f(fake, 0, 4, 8, 8, fake, fake, fake, 9, 1, fake, 8, None) == VALUE
    assert f(fake, 0, 4, 8, 8, fake, fake, fake, 2, 1, fake, 7, None) == SHAPE
    assert f(fake, 0, 4, 8, 8, fake, fake, None, 2, 1, fake, 8, None) == NULL
    assert f(fake, 0, 4, 8, 8, fake, fake, fake, 2, 1, P(4098), 8, None) == ALIGN
    assert f(None, 0, 0, 8, 8, None, None, None, 2, 1, None, 8, None) == 0


def test_sort(nvq):
    f, size = nvq.lib.moe_sort, nvq.lib.moe_sort_workspace_size
    assert f(fake, -1, 2, 8, fake, fake, fake, None, 0, None) == SHAPE
    assert f(fake, 4, 0, 8, fake, fake, fake, None, 0, None) == SHAPE
    assert f(fake, 1 << 30, 2, 8, fake, fake, fake, None, 0, None) == SHAPE      # 2^31 slots
    assert f(fake, 4, 2, 0, fake, fake, fake, None, 0, None) == SHAPE
    assert f(fake, 4, 2, 1025, fake, fake, fake, None, 0, None) == SHAPE
    assert f(fake, 4, 2, 8, fake, None, fake, None, 0, None) == NULL
    assert f(None, 4, 2, 8, fake, fake, fake, None, 0, None) == NULL
    assert f(fake, 4, 2, 8, fake, P(4100), fake, None, 0, None) == ALIGN
    need = size(262144, 8, 256)
    assert need > 0 and size(4, 2, 8) == 0 and size(-1, 2, 8) == 0 and size(4, 2, 0) == 0
    assert f(fake, 262144, 8, 256, fake, fake, fake, None, 0, None) == WORKSPACE
    assert f(fake, 262144, 8, 256, fake, fake, fake, P(1 << 20), need // 2, None) == WORKSPACE
    assert f(fake, 262144, 8, 256, fake, fake, fake, P((1 << 20) + 8), need, None) == WORKSPACE


def test_grouped_products(nvq):
    f = nvq.lib.nvfp4_gemm_grouped

    def fwd(X=fake, xd=1, n=10, k=32, ldx=32, tok=fake, rows=20, off=fake, G=4, codes=fake, scales=fake, g=fake, m=16,
            Y=fake, yd=1, ldy=16):
        return f(X, xd, n, k, ldx, tok, rows, off, G, codes, scales, g, m, Y, yd, ldy, None)

    assert fwd(xd=0) == DTYPE and fwd(yd=3) == DTYPE
    for bad in (dict(k=24), dict(k=0), dict(ldx=16), dict(ldx=36), dict(rows=-1), dict(rows=1 << 31), dict(G=0),
                dict(m=0), dict(ldy=15), dict(n=-1), dict(n=0), dict(tok=None), dict(n=1 << 31)):
        assert fwd(**bad) == SHAPE, bad
    for name in ("X", "off", "codes", "scales", "g", "Y"):
        assert fwd(**{name: None}) == NULL, name
    assert fwd(X=P(4104)) == ALIGN and fwd(codes=P(4100)) == ALIGN and fwd(off=P(4100)) == ALIGN
    assert fwd(Y=P(4097)) == ALIGN and fwd(tok=P(4098)) == ALIGN
    assert fwd(rows=0, X=None, tok=None, off=None, codes=None, scales=None, g=None, Y=None) == 0

    b = nvq.lib.nvfp4_gemm_grouped_dx

    def bwd(dY=fake, dd=1, rows=20, m=16, lddy=16, off=fake, G=4, codes=fake, scales=fake, g=fake, k=32, dX=fake, xd=1,
            lddx=32):
        return b(dY, dd, rows, m, lddy, off, G, codes, scales, g, k, dX, xd, lddx, None)

    assert bwd(dd=0) == DTYPE and bwd(xd=2) == DTYPE
    for bad in (dict(k=24), dict(lddy=15), dict(lddx=31), dict(rows=-1), dict(G=0), dict(m=0)):
        assert bwd(**bad) == SHAPE, bad
    for name in ("dY", "off", "codes", "scales", "g", "dX"):
        assert bwd(**{name: None}) == NULL, name
    assert bwd(dY=P(4097)) == ALIGN and bwd(dX=P(4097)) == ALIGN
    assert bwd(rows=0, dY=None, off=None, codes=None, scales=None, g=None, dX=None) == 0


def test_combine(nvq):
    f, b = nvq.lib.moe_combine, nvq.lib.moe_combine_backward
    assert f(fake, 2, 8, 16, 16, fake, fake, 4, 2, fake, 0, 16, None) == DTYPE
    assert f(fake, 0, 8, 16, 15, fake, fake, 4, 2, fake, 0, 16, None) == SHAPE
    assert f(fake, 0, 8, 16, 16, fake, fake, 4, 2, fake, 0, 15, None) == SHAPE
    assert f(fake, 0, 8, 0, 16, fake, fake, 4, 2, fake, 0, 16, None) == SHAPE
    assert f(fake, 0, 8, 16, 16, fake, fake, 4, 0, fake, 0, 16, None) == SHAPE
    assert f(None, 0, 8, 16, 16, fake, fake, 4, 2, fake, 0, 16, None) == NULL
    assert f(fake, 0, 8, 16, 16, None, fake, 4, 2, fake, 0, 16, None) == NULL
    assert f(P(4098), 0, 8, 16, 16, fake, fake, 4, 2, fake, 0, 16, None) == ALIGN
    assert f(None, 0, 0, 16, 16, None, None, 0, 2, None, 0, 16, None) == 0
    assert b(fake, 0, 4, 16, 16, fake, 0, 8, 16, fake, fake, 2, None, 16, None, None) == NULL
    assert b(fake, 0, 4, 16, 16, None, 0, 8, 16, fake, fake, 2, fake, 16, fake, None) == NULL
    assert b(fake, 0, 4, 16, 16, fake, 0, 8, 16, fake, fake, 2, fake, 15, fake, None) == SHAPE
    assert b(fake, 0, 4, 16, 15, fake, 0, 8, 16, fake, fake, 2, fake, 16, fake, None) == SHAPE
    assert b(fake, 9, 4, 16, 16, fake, 0, 8, 16, fake, fake, 2, fake, 16, fake, None) == DTYPE
    assert b(fake, 0, 4, 16, 16, fake, 0, 8, 16, fake, fake, 2, P(4098), 16, fake, None) == ALIGN
    assert b(None, 0, 0, 16, 16, None, 0, 0, 16, None, None, 2, fake, 16, None, None) == 0


def test_python_functions_refuse_host_tensors(nvq):
    z = torch.zeros(4, 8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    u = torch.zeros(2, 16, 16, dtype=torch.uint8)
    off = torch.zeros(3, dtype=torch.int64)
    for call in (lambda: nvq.moe_topk(z, 2), lambda: nvq.moe_topk_backward(z, i, z[:, :2], z[:, :2]),
                 lambda: nvq.moe_sort(i, 4), lambda: nvq.nvfp4_gemm_grouped(z, u, u[:, :, :2], z[0, :2], off),
                 lambda: nvq.nvfp4_gemm_grouped_dx(z, u, u[:, :, :2], z[0, :2], off), lambda: nvq.moe_combine(z, i),
                 lambda: nvq.moe_combine_backward(z, z, i)):
        with pytest.raises(ValueError, match="HIP device"):
            call()


def test_output_may_not_be_an_input(nvq):
    l, other = nvq.lib, P(8192)
    assert l.moe_topk_backward(fake, 0, 4, 8, 8, other, other, other, 2, 1, fake, 8, None) == VALUE
    assert l.nvfp4_gemm_grouped(fake, 1, 10, 32, 32, other, 20, other, 4, other, other, other, 32, fake, 1, 32, None) == VALUE
    assert l.nvfp4_gemm_grouped_dx(fake, 1, 20, 32, 32, other, 4, other, other, other, 32, fake, 1, 32, None) == VALUE
    assert l.moe_combine(fake, 0, 8, 16, 16, other, other, 4, 2, fake, 0, 16, None) == VALUE
    assert l.moe_combine_backward(other, 0, 4, 16, 16, fake, 0, 8, 16, other, other, 2, fake, 16, None, None) == VALUE
    assert l.moe_combine_backward(fake, 0, 4, 16, 16, other, 0, 8, 16, other, other, 2, fake, 16, None, None) == VALUE
