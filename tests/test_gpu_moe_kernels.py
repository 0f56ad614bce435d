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
