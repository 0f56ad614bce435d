"""GPU parity of MXFP4 quantization, product and gradient against the fp64 oracle.

Quantization and the values are exact (equal).  Products: both operands are exact, so an output's error is that of its sum.
A matrix-core instruction adds 64 (or 128) k to the accumulator; taken as two roundings of 2^-23 of everything it holds,
k / 32 of them, and at most 16 additions that join partial sums: (k / 32 + 16) 2^-23 sum |x w|.  The gradient's instruction
adds 16 bf16 products: (m / 16 + 16) 2^-23 sum |dy w|, as in the NVFP4 products' tests.  A bf16 result adds 2^-8 relative.
"""

import numpy as np
import pytest
import torch

from oracle import mxfp4

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def nvq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import post_nvfp4_weight_amd as m
    return m


def _np(t):
    return t.double().cpu().numpy() if t.dtype.is_floating_point else t.cpu().numpy()


def _same(a, b):
    assert np.array_equal(np.nan_to_num(a, nan=1e300, posinf=1e301, neginf=-1e301), np.nan_to_num(b, nan=1e300, posinf=1e301, neginf=-1e301))


def _check_quantize(nvq, X):
    codes, scales = nvq.mxfp4_quantize(X)
    rc, rs = mxfp4.quantize(_np(X))
    assert np.array_equal(_np(scales), rs)
    got = mxfp4.unpack(_np(codes))
    _same(mxfp4.values(got, rs), mxfp4.values(rc, rs))      # the same values (a zero may have either sign)
    return codes, scales


# ---- quantization ---------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,k,gap", [(1, 32, 0), (1, 4096, 0), (3, 32, 5), (7, 96, 0), (33, 160, 3), (5, 1056, 1), (130, 64, 0),
                                     (2, 8224, 8)])
def test_quantize(nvq, n, k, gap, dtype):
    rng = np.random.default_rng([n, k])
    x = rng.standard_normal((n, k + gap)) * np.exp(3 * rng.standard_normal((n, 1)))
    x[:, ::7] = 0
    X = torch.from_numpy(x.astype(np.float32)).to(DTYPES[dtype]).to(DEV)[:, :k]
    codes, scales = _check_quantize(nvq, X)
    ref = mxfp4.values(mxfp4.unpack(_np(codes)), _np(scales))
    for out in DTYPES.values():
        v = nvq.mxfp4_dequantize(codes, scales, out_dtype=out)
        assert v.dtype == out and v.shape == (n, k)
        assert np.array_equal(_np(v), ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_every_exponent_and_tie(nvq, dtype):
    """Blocks whose largest value has each exponent, with every midpoint of the grid, its neighbours and both signs."""
    dt = DTYPES[dtype]
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    base = np.concatenate((mids, mids * (1 + step), mids * (1 - step), [4.0]))
    rows = []
    for e in range(-149 if dtype == "f32" else -133, 126):
        r = np.zeros(64)
        r[:len(base)] = np.ldexp(base, e)
        r[32:32 + len(base)] = -np.ldexp(base[::-1] / 8, e)
        rows.append(r)
    X = torch.from_numpy(np.array(rows)).to(torch.float32).to(dt).to(DEV)
    codes, scales = _check_quantize(nvq, X)
    for out in DTYPES.values():
        v = _np(nvq.mxfp4_dequantize(codes, scales, out_dtype=out))
        assert np.array_equal(v, mxfp4.values(mxfp4.unpack(_np(codes)), _np(scales)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_special(nvq, dtype):
    X = torch.zeros(6, 128, dtype=DTYPES[dtype])
    X[1, 5] = float("nan")
    X[2, 40] = float("inf")
    X[2, 41] = 1.0
    X[3, 127] = -float("inf")
    X[4] = torch.finfo(DTYPES[dtype]).max
    X[5, 64:] = -0.0
    X[5, 0] = torch.finfo(DTYPES[dtype]).tiny
    codes, scales = _check_quantize(nvq, X.to(DEV))
    s = _np(scales)
    assert s[0].tolist() == [0] * 4 and s[1].tolist() == [255, 0, 0, 0] and s[2].tolist() == [0, 255, 0, 0] and s[3, 3] == 255
    assert not mxfp4.unpack(_np(codes))[1, :32].any()
    v = _np(nvq.mxfp4_dequantize(codes, scales))
    assert np.isnan(v[1, :32]).all() and not np.isnan(v[1, 32:]).any()


def test_dequantize_every_byte(nvq):
    """Every code under every scale byte, infinities and NaN included."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8).repeat_interleave(16).reshape(256, 16).contiguous()
    ref = mxfp4.values(mxfp4.unpack(codes.numpy()), scales.numpy())
    for out, dt in ((torch.float32, np.float32), (torch.bfloat16, np.float32)):
        v = _np(nvq.mxfp4_dequantize(codes.to(DEV), scales.to(DEV), out_dtype=out))
        with np.errstate(over="ignore"):
            _same(v, ref.astype(dt).astype(np.float64))


# ---- product ----------------------------------------------------------------------
def _weights(rng, m, k, wide=False):
    w = rng.standard_normal((m, k)) * 0.05
    if wide:
        w *= np.exp(4 * rng.standard_normal((m, 1)))
    codes, scales = mxfp4.quantize(w)
    return torch.from_numpy(mxfp4.pack(codes)).to(DEV), torch.from_numpy(scales).to(DEV), mxfp4.values(codes, scales)


def _random_codes(rng, n, k, lo=110, hi=140):
    codes = rng.integers(0, 16, (n, k), dtype=np.uint8)
    scales = rng.integers(lo, hi, (n, k // 32), dtype=np.uint8)
    return torch.from_numpy(mxfp4.pack(codes)).to(DEV), torch.from_numpy(scales).to(DEV), mxfp4.values(codes, scales)


def _bound(x, w, terms, ref, dtype):
    return (terms + 16) * 2.0 ** -23 * (np.abs(x) @ np.abs(w)) + (2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 0) + 1e-37


SHAPES = [(1, 1, 32), (1, 17, 64), (1, 64, 512), (2, 33, 544), (5, 100, 1024), (16, 64, 4128), (17, 48, 96), (31, 130, 2048),
          (33, 16, 512), (64, 257, 1056), (65, 128, 256), (100, 130, 288), (128, 256, 512), (129, 1003, 1056), (257, 300, 160),
          (300, 129, 8192)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,m,k", SHAPES)
def test_gemm_packed(nvq, n, m, k, dtype):
    """Random codes under random scales on both sides: every lane's block must meet its own scale."""
    rng = np.random.default_rng([n, m, k])
    xc, xs, x = _random_codes(rng, n, k)
    wc, ws, w = _random_codes(rng, m, k)
    dt = DTYPES[dtype]
    Y = nvq.mxfp4_gemm(xc, wc, ws, x_scales=xs, out_dtype=dt)
    assert Y.dtype == dt
    ref = x @ w.T
    assert np.all(np.abs(_np(Y) - ref) <= _bound(x, w.T, k / 32, ref, dt))


@pytest.mark.parametrize("xtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,m,k", SHAPES)
def test_gemm_quantizes(nvq, n, m, k, xtype):
    """X in bf16 or fp32, rows apart: the product of mxfp4_quantize's values."""
    rng = np.random.default_rng([n, m, k, 1])
    X = torch.from_numpy((rng.standard_normal((n, k + 3)) * np.exp(rng.standard_normal(k + 3))).astype(np.float32)).to(DTYPES[xtype])
    X = X.to(DEV)[:, 1:1 + k]
    wc, ws, w = _weights(rng, m, k)
    Y = nvq.mxfp4_gemm(X, wc, ws)
    x = mxfp4.values(*mxfp4.quantize(_np(X)))
    ref = x @ w.T
    assert np.all(np.abs(_np(Y) - ref) <= _bound(x, w.T, k / 32, ref, torch.float32))


@pytest.mark.parametrize("n", [3, 40, 200])
def test_gemm_exact_integers(nvq, n):
    """Values whose sums fp32 holds exactly, one block after another: equality, so no block is lost or met twice."""
    k, m = 1120, 70
    rng = np.random.default_rng(n)
    xc, xs, x = _random_codes(rng, n, k, 127, 129)
    wc, ws, w = _random_codes(rng, m, k, 127, 129)
    assert np.array_equal(_np(nvq.mxfp4_gemm(xc, wc, ws, x_scales=xs)), x @ w.T)


@pytest.mark.parametrize("n", [2, 50, 150])
def test_gemm_nan_blocks(nvq, n):
    """A NaN block of X makes its row NaN, one of W its column; nothing else changes."""
    k, m = 352, 40
    rng = np.random.default_rng(n)
    xc, xs, x = _random_codes(rng, n, k)
    wc, ws, w = _random_codes(rng, m, k)
    clean = _np(nvq.mxfp4_gemm(xc, wc, ws, x_scales=xs))
    for block in (0, 7, 10):
        a, b = xs.clone(), ws.clone()
        a[n - 1, block] = 255
        b[m - 2, block] = 255
        y = _np(nvq.mxfp4_gemm(xc, wc, b, x_scales=a))
        want = clean.copy()
        want[n - 1] = np.nan
        want[:, m - 2] = np.nan
        _same(y, want)
    X = torch.ones(n, k, dtype=torch.bfloat16, device=DEV)
    X[0, 33] = float("nan")
    y = _np(nvq.mxfp4_gemm(X, wc, ws))
    assert np.isnan(y[0]).all() and not np.isnan(y[1:]).any()


@pytest.mark.parametrize("n", [4, 90])
def test_gemm_extreme_scales(nvq, n):
    """Scales whose product leaves fp32's range on either side, and ones that cancel."""
    k, m = 64, 8
    one = np.full((n, k), 2, dtype=np.uint8)      # 1.0
    xc = torch.from_numpy(mxfp4.pack(one)).to(DEV)
    wc = torch.from_numpy(mxfp4.pack(np.full((m, k), 2, dtype=np.uint8))).to(DEV)
    for a, b in ((0, 254), (254, 0), (127, 127), (20, 234), (190, 190), (10, 10)):
        xs = torch.full((n, 2), a, dtype=torch.uint8, device=DEV)
        ws = torch.full((m, 2), b, dtype=torch.uint8, device=DEV)
        y = _np(nvq.mxfp4_gemm(xc, wc, ws, x_scales=xs))
        want = np.float32(min(64 * 2.0 ** (a + b - 254), 3e39)) if a + b < 400 else np.inf
        if a + b - 254 > 122:
            assert np.all(np.isinf(y)) and np.all(y > 0)
        elif a + b - 254 < -149 - 6:
            assert np.all(y == 0)
        else:
            assert np.all(y == want), (a, b)


@pytest.mark.parametrize("n", [3, 60, 140])
def test_gemm_output_rows_apart(nvq, n):
    """Y with gaps between its rows and at an odd element: only its own elements are written."""
    k, m = 96, 77
    rng = np.random.default_rng(n)
    xc, xs, x = _random_codes(rng, n, k)
    wc, ws, w = _random_codes(rng, m, k)
    for dt in DTYPES.values():
        buf = torch.full((n + 2, m + 10), 7.0, dtype=dt, device=DEV)
        Y = buf[1:n + 1, 3:3 + m]
        nvq.mxfp4_gemm(xc, wc, ws, x_scales=xs, Y=Y)
        ref = x @ w.T
        assert np.all(np.abs(_np(Y) - ref) <= _bound(x, w.T, k / 32, ref, dt))
        Y.fill_(7.0)
        assert bool((buf == 7.0).all())


def test_gemm_empty(nvq):
    wc, ws, _ = _weights(np.random.default_rng(0), 8, 64)
    assert nvq.mxfp4_gemm(torch.zeros(0, 64, device=DEV), wc, ws).shape == (0, 8)
    c, s = nvq.mxfp4_quantize(torch.zeros(0, 64, device=DEV))
    assert c.shape == (0, 32) and s.shape == (0, 2) and nvq.mxfp4_dequantize(c, s).shape == (0, 64)
    assert nvq.mxfp4_gemm_dx(torch.zeros(0, 8, dtype=torch.bfloat16, device=DEV), wc, ws).shape == (0, 64)


# ---- gradient -----------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,m,k", [(1, 1, 32), (1, 64, 256), (3, 65, 64), (64, 100, 288), (65, 128, 1056), (100, 1003, 96), (129, 77, 512),
                                   (600, 64, 352), (700, 200, 544), (1, 5000, 64)])
def test_gemm_dx(nvq, n, m, k, dtype):
    rng = np.random.default_rng([n, m, k, 2])
    wc, ws, w = _random_codes(rng, m, k)
    dY = torch.from_numpy(rng.standard_normal((n, m + 1)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    dt = DTYPES[dtype]
    for d in (dY[:, :m], dY[:, 1:], dY[:, :m].contiguous()):
        dX = nvq.mxfp4_gemm_dx(d, wc, ws, out_dtype=dt)
        dy = _np(d)
        ref = dy @ w
        assert np.all(np.abs(_np(dX) - ref) <= _bound(dy, w, m / 16, ref, dt))


def test_gemm_dx_scales(nvq):
    """Every scale byte that bf16 and fp32 hold with the codes' range, zero codes, and NaN blocks."""
    m, k = 256, 64
    rng = np.random.default_rng(5)
    codes = rng.integers(0, 16, (m, k), dtype=np.uint8)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 2, axis=1)
    wc, ws = torch.from_numpy(mxfp4.pack(codes)).to(DEV), torch.from_numpy(scales).to(DEV)
    w = mxfp4.values(codes, scales)
    dY = torch.eye(m, dtype=torch.bfloat16, device=DEV)[:253]
    dX = _np(nvq.mxfp4_gemm_dx(dY[:, :253].contiguous(), wc[:253].contiguous(), ws[:253].contiguous()))
    assert np.array_equal(dX[1:], w[1:253])      # (byte 0 and 1 reach bf16's subnormals)
    b = ws.clone()
    b[:] = 127
    b[7, 1] = 255
    dX = _np(nvq.mxfp4_gemm_dx(dY, wc, b))
    assert np.isnan(dX[:, 32:]).all() and not np.isnan(dX[:, :32]).any()


def test_gemm_dx_against_differences(nvq):
    """The product is linear in its quantized activations: a difference of two products is the gradient's product."""
    n, m, k = 6, 48, 96
    rng = np.random.default_rng(6)
    xc, xs, x = _random_codes(rng, n, k, 125, 129)
    wc, ws, w = _random_codes(rng, m, k, 125, 129)
    dY = torch.from_numpy(rng.integers(-2, 3, (n, m)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    dX = _np(nvq.mxfp4_gemm_dx(dY, wc, ws))
    base = (_np(nvq.mxfp4_gemm(xc, wc, ws, x_scales=xs)) * _np(dY)).sum()
    for t, j in ((0, 0), (3, 50), (5, 95)):
        c = mxfp4.unpack(_np(xc))
        c[t, j] ^= 8                                # x -> -x
        moved = (_np(nvq.mxfp4_gemm(torch.from_numpy(mxfp4.pack(c)).to(DEV), wc, ws, x_scales=xs)) * _np(dY)).sum()
        assert moved - base == -2 * x[t, j] * dX[t, j]      # small integers and halves: exact
