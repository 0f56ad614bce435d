"""The experts' products at the edges of what their callers may pass, on each of the kernels that the library chooses from:
few rows, 64 x 128 tiles and 128 x 256 tiles of the product, 64- and 128-row tiles of its gradient, each with rows that the
copies to LDS can and cannot bring.  Error bounds as for the products at other sizes: (depth / 16 + 16) 2^-23 of
sum |x w|, and 2^-8 of the result where it is bf16."""

import numpy as np
import pytest
import torch

from oracle import moe

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def nvq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import post_nvfp4_weight_amd as m
    return m


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def _np(t):
    return t.double().cpu().numpy() if t.dtype.is_floating_point else t.cpu().numpy()


def _most_tiles(rows, G, height, columns):
    return ((rows // height + min(rows, G)) * columns + 7) // 8 * 8


def _kernel(rows, G, m):
    """The product's kernel for X below 4 GiB, by the rule that nvfp4_gemm_grouped_launch goes by."""
    if _most_tiles(rows, G, 16, -(-m // 32)) <= 768:
        return "few rows"
    if rows >= 32 * min(rows, G) and _most_tiles(rows, G, 128, -(-m // 256)) >= 448:
        return "128 x 256"
    return "64 x 128"


# Rows of each expert, so that experts end at and around every height that a tile can have; outputs.
SMALL = [0, 1, 2, 15, 16, 17, 0, 31, 32, 33]
LARGE = SMALL + [47, 48, 49, 63, 64, 65, 95, 96, 97, 127, 128, 129, 159, 160, 161, 0, 191, 192, 193, 255, 256, 257, 0]
PRODUCTS = {"few rows": (SMALL, 70), "64 x 128": (LARGE, 203), "128 x 256": (LARGE, 2563)}


def _sized(kernel, counts, m, lead, tail):
    """grp_off of the counts behind `lead` rows of no expert, and the rows with `tail` more; checks the kernel chosen."""
    off = (lead + np.concatenate([[0], np.cumsum(counts)])).astype(np.int64)
    rows = int(off[-1]) + tail
    assert _kernel(rows, len(counts), m) == kernel
    return off, rows


def _experts(rng, G, m, k):
    packed = rng.integers(0, 256, (G, m, k // 2), dtype=np.uint8)
    scales = rng.integers(0x20, 0x7F, (G, m, k // 16), dtype=np.uint8)
    return packed, scales, (rng.random(G) + 0.5).astype(np.float32) * np.float32(1e-3)


def _normal(rng, shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DEV, torch.bfloat16)


def _product(X, W, off, tok):
    """The oracle's product, an expert at a time."""
    Y = np.zeros((len(tok), W.shape[1]))
    for e in range(len(W)):
        r = slice(int(off[e]), int(off[e + 1]))
        Y[r] = moe.grouped_matmul(X, W[e:e + 1], [0, r.stop - r.start], tok[r]) if r.stop > r.start else 0
    return Y


def _close(Y, ref, mag, depth, dtype):
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert np.all(np.abs(_np(Y) - ref) <= mag * ((depth / 16 + 16) * 2.0 ** -23) + np.abs(ref) * half + 1e-30)


@pytest.mark.parametrize("kernel", PRODUCTS)
def test_rows_without_a_token_under_rejected_weights(nvq, kernel):
    """A row whose token is outside [0, n) is zeros, also in the channel of a rejected weight row and under an infinite g."""
    counts, m = PRODUCTS[kernel]
    rng = np.random.default_rng(m)
    G, k, n = len(counts), 64, 40
    off, rows = _sized(kernel, counts, m, 0, 0)
    packed, scales, g = _experts(rng, G, m, k)
    scales[:, 5] = 0x7F
    g[4] = np.inf
    tok = rng.integers(0, n, rows).astype(np.int32)
    bad = rng.random(rows) < 0.3
    tok[bad] = rng.choice([-1, n, 2 ** 31 - 1, -2 ** 31], int(bad.sum()))
    X = _normal(rng, (n, k))
    for dtype in DTYPES.values():
        Y = nvq.nvfp4_gemm_grouped(X, _dev(packed), _dev(scales), _dev(g), _dev(off), tok_idx=_dev(tok), out_dtype=dtype)
        bd = _dev(bad)
        assert (Y[bd] == 0).all() and torch.isnan(Y[~bd][:, 5]).all()
        fine = ~bad
        fine[off[4]:off[5]] = False
        assert torch.isfinite(Y[_dev(fine)][:, torch.arange(m, device=DEV) != 5]).all()


# ---- the product ----------------------------------------------------------------
@pytest.mark.parametrize("kernel", PRODUCTS)
@pytest.mark.parametrize("k", [48, 272, 528, 1040])
def test_product_edges(nvq, kernel, k):
    """Experts that end around every tile height, rows of no expert before the first and behind the last one, tokens outside
    [0, n) everywhere, X and Y in wider buffers, Y's rows at 16-byte places and at their elements' only."""
    counts, m = PRODUCTS[kernel]
    rng = np.random.default_rng([m, k])
    G, n, lead, tail = len(counts), 90, 2, 5
    off, rows = _sized(kernel, counts, m, lead, tail)
    packed, scales, g = _experts(rng, G, m, k)
    W = moe.experts_matrices(packed, scales, g)
    tok = rng.integers(0, n, rows).astype(np.int32)
    bad = rng.random(rows) < 0.05
    bad[off[:-1][np.array(counts) > 2]] = True          # the first and the last row of a tile among them
    bad[off[1:][np.array(counts) > 30] - 1] = True
    tok[bad] = rng.choice([-1, n, 2 ** 31 - 1, -2 ** 31], int(bad.sum()))
    tok[:lead] = tok[rows - tail:] = -2 ** 31           # never looked at
    X = _normal(rng, (n, k + 24))[:, 8:8 + k]
    args = (_dev(packed), _dev(scales), _dev(g), _dev(off))
    ref, mag = _product(_np(X), W, off, tok), _product(np.abs(_np(X)), np.abs(W), off, tok)
    used = slice(lead, rows - tail)
    for dtype in DTYPES.values():
        for first, width in ((8, (m + 23) // 8 * 8), (3, m + 6)):
            Yw = torch.full((rows, width), 7.0, dtype=dtype, device=DEV)
            nvq.nvfp4_gemm_grouped(X, *args, tok_idx=_dev(tok), Y=Yw[:, first:first + m])
            assert (Yw[:lead] == 7).all() and (Yw[rows - tail:] == 7).all()
            assert (Yw[:, :first] == 7).all() and (Yw[:, first + m:] == 7).all()
            Y = Yw[used, first:first + m]
            assert (Y[_dev(bad[used])] == 0).all()
            _close(Y, ref[used], mag[used], k, dtype)


@pytest.mark.parametrize("kernel", PRODUCTS)
def test_product_of_the_rows_themselves(nvq, kernel):
    """Without tok_idx, rows of no expert at both ends."""
    counts, m = PRODUCTS[kernel]
    rng = np.random.default_rng([m, 1])
    G, k, lead, tail = len(counts), 144, 3, 2
    off, rows = _sized(kernel, counts, m, lead, tail)
    packed, scales, g = _experts(rng, G, m, k)
    W = moe.experts_matrices(packed, scales, g)
    X = _normal(rng, (rows, k))
    Y = torch.full((rows, m), 7.0, device=DEV)
    nvq.nvfp4_gemm_grouped(X, _dev(packed), _dev(scales), _dev(g), _dev(off), Y=Y)
    tok, used = np.arange(rows), slice(lead, rows - tail)
    assert (Y[:lead] == 7).all() and (Y[rows - tail:] == 7).all()
    _close(Y[used], _product(_np(X), W, off, tok)[used], _product(np.abs(_np(X)), np.abs(W), off, tok)[used], k, torch.float32)


def _finite_part(got, bad, X, W, off, tok, depth):
    """got where not bad, against the product of the inputs with zeros for all that is not finite."""
    X, W = np.nan_to_num(X, nan=0.0, posinf=0.0, neginf=0.0), np.nan_to_num(W)
    ref, mag = _product(X, W, off, tok), _product(np.abs(X), np.abs(W), off, tok)
    assert np.isfinite(got[~bad]).all()
    assert np.all(np.abs(got - ref)[~bad] <= (mag * ((depth / 16 + 16) * 2.0 ** -23) + 1e-30)[~bad])


@pytest.mark.parametrize("kernel", PRODUCTS)
@pytest.mark.parametrize("k", [256, 656])
def test_product_non_finite(nvq, kernel, k):
    """A row of X with a NaN or an infinity spoils its own rows, a rejected weight row its own channel of its own expert; a
    block's scale may be negative."""
    counts, m = PRODUCTS[kernel]
    rng = np.random.default_rng([m, k, 2])
    G, n = len(counts), 60
    off, rows = _sized(kernel, counts, m, 0, 0)
    packed, scales, g = _experts(rng, G, m, k)
    packed[9, m - 1], scales[9, m - 1] = 0, 0x7F
    packed[4, 5], scales[4, 5, k // 16 - 1] = 0x22, 0x7F            # the last block alone
    scales[:, ::3, 1::2] |= 0x80
    X = _normal(rng, (n, k))
    X[0, 7], X[31, k - 1], X[n - 1, 40] = float("nan"), float("inf"), -float("inf")
    tok = rng.integers(0, n, rows).astype(np.int32)
    tok[::17] = -1                                      # these read nothing of token 0's NaN
    Y = _np(nvq.nvfp4_gemm_grouped(X, _dev(packed), _dev(scales), _dev(g), _dev(off), tok_idx=_dev(tok)))
    bad = np.zeros((rows, m), dtype=bool)
    bad[np.isin(tok, [0, 31, n - 1])] = True
    channel = np.zeros((rows, m), dtype=bool)
    channel[off[9]:off[10], m - 1] = channel[off[4]:off[5], 5] = True
    channel[tok == -1] = False
    assert np.isnan(Y[channel]).all() and not np.isfinite(Y[bad]).any() and np.isnan(Y[tok == 0]).all()
    assert (Y[tok == -1] == 0).all()
    W = moe.experts_matrices(packed, scales & 0x7F, g) * np.where(np.repeat(scales >> 7, 16, axis=2), -1, 1)
    _finite_part(Y, bad | channel, _np(X), W, off, tok, k)


@pytest.mark.parametrize("kernel", PRODUCTS)
def test_product_offsets_out_of_range(nvq, kernel):
    """Offsets are clamped into [0, rows]: whatever they are, nothing outside Y's rows is written."""
    counts, m = PRODUCTS[kernel]
    rng = np.random.default_rng([m, 3])
    G, k = len(counts), 96
    off, rows = _sized(kernel, counts, m, 0, 0)
    packed, scales, g = _experts(rng, G, m, k)
    X = _normal(rng, (rows, k))
    args = (X, _dev(packed), _dev(scales), _dev(g))
    guard = torch.full((rows + 40, m), 7.0, device=DEV)
    clamped = np.clip(off, 0, rows)
    wild = off.copy()
    wild[0], wild[-1] = -2 ** 40, 2 ** 62
    nvq.nvfp4_gemm_grouped(*args, _dev(wild), Y=guard[20:20 + rows])
    assert (guard[:20] == 7).all() and (guard[20 + rows:] == 7).all()
    assert torch.equal(guard[20:20 + rows], nvq.nvfp4_gemm_grouped(*args, _dev(clamped)))


@pytest.mark.parametrize("counts,m", [([5, 0, 9], 40), ([300, 1, 399], 300), ([40, 70, 129], 1000)])
@pytest.mark.parametrize("k", [528, 1040, 1168])
def test_product_of_activations_past_4_gib(nvq, counts, m, k):
    """Rows of X 2^32 bytes and more behind its start, k long enough for every loop over it, tokens outside [0, n)."""
    rng = np.random.default_rng([m, k, 4])
    G, n, ldx = len(counts), 270, 1 << 23
    off, rows = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64), sum(counts) + 3
    packed, scales, g = _experts(rng, G, m, k)
    W = moe.experts_matrices(packed, scales, g)
    X = torch.empty(n, ldx, dtype=torch.bfloat16, device=DEV)[:, :k]
    X.copy_(torch.from_numpy(rng.standard_normal((n, k)).astype(np.float32)))
    assert (n - 1) * ldx * 2 > 2 ** 32
    tok = rng.integers(0, n, rows).astype(np.int32)
    tok[:5], tok[-4] = [n - 1, -1, 257, n, 0], 2 ** 31 - 1
    ref, mag = _product(_np(X), W, off, tok), _product(np.abs(_np(X)), np.abs(W), off, tok)
    for dtype in DTYPES.values():
        Y = torch.full((rows, m), 7.0, dtype=dtype, device=DEV)
        nvq.nvfp4_gemm_grouped(X, _dev(packed), _dev(scales), _dev(g), _dev(off), tok_idx=_dev(tok), Y=Y)
        assert (Y[off[-1]:] == 7).all() and (Y[[1, 3, rows - 4]] == 0).all()
        _close(Y[:off[-1]], ref[:off[-1]], mag[:off[-1]], k, dtype)


# ---- the gradient of the rows -----------------------------------------------------
# Rows of each expert: below 24 on average (64-row tiles) and above (128-row tiles).
GRADIENTS = {64: SMALL + [0] * 5 + [63, 64, 65, 66] + [1] * 15, 128: LARGE}


def _gradient_sized(height, counts, lead, tail):
    off = (lead + np.concatenate([[0], np.cumsum(counts)])).astype(np.int64)
    rows = int(off[-1]) + tail
    assert (128 if rows // min(rows, len(counts)) >= 24 else 64) == height   # nvfp4_gemm_grouped_dx_launch's rule
    return off, rows


def _gradient(dY, W, off):
    dX = np.zeros((len(dY), W.shape[2]))
    for e in range(len(W)):
        r = slice(int(off[e]), int(off[e + 1]))
        dX[r] = moe.grouped_matmul_dx(dY[r], W[e:e + 1], [0, r.stop - r.start])
    return dX


@pytest.mark.parametrize("height", GRADIENTS)
@pytest.mark.parametrize("m,k", [(40, 272), (64, 528), (200, 64), (328, 1040), (1, 16), (71, 304)])
def test_gradient_edges(nvq, height, m, k):
    """dY copied to LDS directly (m and the row stride multiples of 8, 16-byte aligned) and through registers, in wider
    buffers; dX at 16-byte places and at its elements' only; rows of no expert before the first and behind the last one."""
    counts = GRADIENTS[height]
    rng = np.random.default_rng([height, m, k])
    G, lead, tail = len(counts), 3, 6
    off, rows = _gradient_sized(height, counts, lead, tail)
    packed, scales, g = _experts(rng, G, m, k)
    W = moe.experts_matrices(packed, scales, g)
    dYw = _normal(rng, (rows, (m + 31) // 8 * 8))
    args = (_dev(packed), _dev(scales), _dev(g), _dev(off))
    used = slice(lead, rows - tail)
    for at in (8, 5):                                   # at 8 with m % 8 == 0 directly, else through registers
        dY = dYw[:, at:at + m]
        dYw[:lead], dYw[rows - tail:] = float("nan"), float("nan")   # rows that nothing may come from
        ref, mag = _gradient(_np(dY), W, off), _gradient(np.abs(_np(dY)), np.abs(W), off)
        for dtype in DTYPES.values():
            for first, width in ((8, k + 16), (1, k + 7)):
                dXw = torch.full((rows, width), 7.0, dtype=dtype, device=DEV)
                nvq.nvfp4_gemm_grouped_dx(dY, *args, dX=dXw[:, first:first + k])
                assert (dXw[:lead] == 7).all() and (dXw[rows - tail:] == 7).all()
                assert (dXw[:, :first] == 7).all() and (dXw[:, first + k:] == 7).all()
                _close(dXw[used, first:first + k], ref[used], mag[used], m, dtype)


@pytest.mark.parametrize("height", GRADIENTS)
@pytest.mark.parametrize("m", [136, 131])
def test_gradient_non_finite(nvq, height, m):
    """A row of dY with a NaN or an infinity spoils its own row, a rejected weight row all rows of its own expert."""
    counts = GRADIENTS[height]
    rng = np.random.default_rng([height, m])
    G, k = len(counts), 176
    off, rows = _gradient_sized(height, counts, 0, 0)
    packed, scales, g = _experts(rng, G, m, k)
    packed[7, m - 1], scales[7, m - 1] = 0, 0x7F
    scales[:, ::3, 1::2] |= 0x80
    dY = _normal(rng, (rows, m))
    nan, inf = int(off[2]), int(off[9]) - 1
    dY[nan, 3], dY[inf, m - 1], dY[rows - 1, 0] = float("nan"), float("inf"), -float("inf")
    dX = _np(nvq.nvfp4_gemm_grouped_dx(dY, _dev(packed), _dev(scales), _dev(g), _dev(off)))
    bad = np.zeros((rows, k), dtype=bool)
    bad[[nan, inf, rows - 1]] = bad[off[7]:off[8]] = True
    assert np.isnan(dX[nan]).all() and np.isnan(dX[off[7]:off[8]]).all() and not np.isfinite(dX[bad]).any()
    W = moe.experts_matrices(packed, scales & 0x7F, g) * np.where(np.repeat(scales >> 7, 16, axis=2), -1, 1)
    W, D = np.nan_to_num(W), np.nan_to_num(_np(dY), nan=0.0, posinf=0.0, neginf=0.0)
    ref, mag = _gradient(D, W, off), _gradient(np.abs(D), np.abs(W), off)
    assert np.isfinite(dX[~bad]).all()
    assert np.all(np.abs(dX - ref)[~bad] <= (mag * ((m / 16 + 16) * 2.0 ** -23) + 1e-30)[~bad])


@pytest.mark.parametrize("height", GRADIENTS)
@pytest.mark.parametrize("m", [64, 61])
def test_gradient_offsets_out_of_range(nvq, height, m):
    counts = GRADIENTS[height]
    rng = np.random.default_rng([height, m, 5])
    G, k = len(counts), 96
    off, rows = _gradient_sized(height, counts, 0, 0)
    packed, scales, g = _experts(rng, G, m, k)
    args = (_normal(rng, (rows, m)), _dev(packed), _dev(scales), _dev(g))
    guard = torch.full((rows + 40, k), 7.0, device=DEV)
    wild = off.copy()
    wild[0], wild[-1] = -2 ** 40, 2 ** 62
    nvq.nvfp4_gemm_grouped_dx(*args, _dev(wild), dX=guard[20:20 + rows])
    assert (guard[:20] == 7).all() and (guard[20 + rows:] == 7).all()
    assert torch.equal(guard[20:20 + rows], nvq.nvfp4_gemm_grouped_dx(*args, _dev(off)))


@pytest.mark.parametrize("ldd", [(1 << 23) - 8, 1 << 23])
def test_gradient_of_widely_spaced_rows(nvq, ldd):
    """Row strides up to the largest that the direct copies' 32-bit offsets span in a tile of 128, and past it."""
    rng = np.random.default_rng(6)
    rows, m, k = 131, 72, 80
    packed, scales, g = _experts(rng, 1, m, k)
    W = moe.experts_matrices(packed, scales, g)
    dY = torch.empty(rows, ldd, dtype=torch.bfloat16, device=DEV)[:, :m]
    dY.copy_(torch.from_numpy(rng.standard_normal((rows, m)).astype(np.float32)))
    off = np.array([0, rows], dtype=np.int64)
    dX = nvq.nvfp4_gemm_grouped_dx(dY, _dev(packed), _dev(scales), _dev(g), _dev(off))
    _close(dX, _gradient(_np(dY), W, off), _gradient(np.abs(_np(dY)), np.abs(W), off), m, torch.float32)
