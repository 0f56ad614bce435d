"""GPU parity of the mixture-of-experts path (router, sort by expert, experts' NVFP4 products, weighted sum, and their
gradients) against the fp64 oracle.

Error bounds, with u = 2^-24 (half a step of fp32) and 2^-8 relative for a bf16 result:
  - weights: the exponent's argument l - max is rounded once, |l - max| <= D, which is D u relative in exp; expf is within
    2 u; numerator and denominator both carry that, the sum of positive terms adds at most 22 additions' u (16 in the lane,
    6 across lanes) and the quotient 2 u: below (2 D + 32) u;
  - router gradient p (d - c): p as above, c = sum dw w within (that + 8 u) sum |dw w|, difference and product 2 u;
  - products: exact per element (8 times 6 bits), k / 16 matrix-core steps and g once: (k / 16 + 16) 2^-23 sum |x w|
    as in the single-matrix product's tests;
  - sums of n fp32 products in any order: n u sum |terms| (fused multiply-adds round once per term).
"""

import numpy as np
import pytest
import torch

from oracle import moe

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
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


def _half(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 0.0


# ---- router -------------------------------------------------------------------
def _logits(rng, T, E, dtype, masked):
    l = torch.from_numpy((rng.standard_normal((T, E)) * 2).astype(np.float32)).to(dtype)
    if masked:
        l[torch.from_numpy(rng.random((T, E)) < 0.5)] = float("-inf")
        l[::5] = float("-inf")
    return l


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K,masked", [(1, 1, 1, False), (1, 256, 8, False), (7, 8, 8, True), (37, 60, 3, True),
                                          (130, 64, 1, False), (65, 65, 6, True), (33, 128, 5, False), (50, 160, 7, True),
                                          (300, 256, 8, True), (9, 1000, 64, True), (5, 1024, 64, False), (4, 513, 16, True)])
def test_topk_and_gradient(nvq, T, E, K, masked, renorm, dtype):
    rng = np.random.default_rng([T, E, K])
    dtype = DTYPES[dtype]
    l = _logits(rng, T, E, dtype, masked)
    ids, w = nvq.moe_topk(l.to(DEV), K, renorm)
    rid, rw = moe.topk(_np(l), K, renorm)
    assert np.array_equal(_np(ids), rid)
    finite = np.where(np.isfinite(_np(l)), _np(l), np.nan)
    D = np.nan_to_num(np.nanmax(finite, 1) - np.nanmin(finite, 1)) if masked else np.ptp(_np(l), axis=1)
    ew = (2 * D + 32)[:, None] * U
    assert np.all(np.abs(_np(w) - rw) <= ew * rw + 1e-37)
    dw = rng.standard_normal((T, K)).astype(np.float32)
    dl = nvq.moe_topk_backward(l.to(DEV), ids, w, _dev(dw), renorm)
    assert dl.dtype == dtype
    ref = moe.topk_backward(_np(l), rid, rw, dw, renorm)
    mag = np.abs(dw * rw).sum(1)[:, None]
    p = np.zeros((T, E))
    if renorm:
        for t in range(T):
            p[t, rid[t][rid[t] >= 0]] = rw[t][rid[t] >= 0]
    else:
        p = np.where(np.isfinite(_np(l)), np.exp(finite - np.nan_to_num(np.nanmax(np.where(np.isnan(finite), -1e30, finite), 1))[:, None]), 0)
        p = np.nan_to_num(p / np.maximum(p.sum(1, keepdims=True), 1e-30))
    bound = np.abs(ref) * (ew + 2 * U + _half(dtype)) + p * mag * (ew + 8 * U) + 1e-37
    assert np.all(np.abs(_np(dl) - ref) <= bound)


def test_topk_ties_strides_and_rejected_rows(nvq):
    # many equal values: every tie goes to the lower index
    rng = np.random.default_rng(3)
    l = torch.from_numpy(rng.integers(0, 4, (64, 200)).astype(np.float32))
    for dtype in DTYPES.values():
        ids, _ = nvq.moe_topk(l.to(DEV, dtype), 12)
        assert np.array_equal(_np(ids), moe.topk(_np(l), 12, True)[0])
    # +0 and -0 are equal
    z = torch.zeros(1, 6)
    z[0, 0] = -0.0
    assert _np(nvq.moe_topk(z.to(DEV), 3)[0]).tolist() == [[0, 1, 2]]
    # a slice of a wider matrix, rows unaligned
    wide = torch.from_numpy(rng.standard_normal((40, 131)).astype(np.float32))
    for dtype in DTYPES.values():
        v = wide.to(DEV, dtype)[:, 1:102]
        ids, w = nvq.moe_topk(v, 5, False)
        rid, rw = moe.topk(_np(v), 5, False)
        assert np.array_equal(_np(ids), rid) and np.allclose(_np(w), rw, rtol=1e-5)
    # NaN and +inf reject their own row only; largest finite values do not overflow
    b = torch.zeros(6, 70)
    b[1, 3], b[2, 69], b[3, 5] = float("nan"), float("inf"), -float("inf")
    b[4, 0], b[4, 1], b[4, 2] = 3e38, -3e38, 3e38
    for renorm in (True, False):
        ids, w = nvq.moe_topk(b.to(DEV), 2, renorm)
        dl = nvq.moe_topk_backward(b.to(DEV), ids, w, torch.ones(6, 2, device=DEV), renorm)
        assert _np(ids)[1:3].tolist() == [[-1, -1], [-1, -1]]
        assert torch.isnan(w[1:3]).all() and torch.isnan(dl[1:3]).all()
        keep = [0, 3, 4, 5]
        assert torch.isfinite(w[keep]).all() and torch.isfinite(dl[keep]).all()
        assert _np(ids)[4].tolist() == [0, 2] and _np(w)[4].tolist() == [0.5, 0.5]
    ids, w = nvq.moe_topk(torch.zeros(0, 5, device=DEV), 2)
    assert ids.shape == w.shape == (0, 2)


def test_topk_gradient_against_differences(nvq):
    # the weights' sum with random factors, differences of the fp64 oracle on the same logits
    rng = np.random.default_rng(4)
    T, E, K = 3, 12, 4
    l = rng.standard_normal((T, E)).astype(np.float32)
    dw = rng.standard_normal((T, K)).astype(np.float32)
    for renorm in (True, False):
        ids, w = nvq.moe_topk(_dev(l), K, renorm)
        dl = _np(nvq.moe_topk_backward(_dev(l), ids, w, _dev(dw), renorm))
        h = 1e-6
        for i in np.ndindex(l.shape):
            a, b = l.astype(np.float64), l.astype(np.float64)
            a[i] += h
            b[i] -= h
            diff = ((moe.topk(a, K, renorm)[1] - moe.topk(b, K, renorm)[1]) * dw).sum() / (2 * h)
            assert abs(diff - dl[i]) <= 1e-5   # fp32 results of order 1, differences to about 1e-9


# ---- sort ---------------------------------------------------------------------
def _sort_ref(ids, E):
    T, K = ids.shape
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    cnt = np.bincount(key, minlength=E + 1)[:E]
    off = np.concatenate([[0], np.cumsum(cnt)])
    n = off[-1]
    tok = np.full(T * K, -1, dtype=np.int32)
    tok[:n] = order[:n] // K
    pos = np.full(T * K, -1, dtype=np.int32)
    pos[order[:n]] = np.arange(n)
    return tok, off, pos.reshape(T, K)


@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (1, 8, 256), (37, 8, 256), (5, 3, 1024), (1000, 7, 60), (2048, 8, 256),
                                   (2049, 8, 256), (16385, 1, 1000), (5461, 3, 1), (70001, 5, 128), (9001, 64, 1024), (1024, 8, 60),
                                   (1025, 8, 256), (131072, 8, 256), (131073, 8, 1000)])
@pytest.mark.parametrize("kind", ["uniform", "skewed", "dropped"])
def test_sort(nvq, T, K, E, kind):
    rng = np.random.default_rng([T, K, E])
    if kind == "skewed":     # almost all to one expert
        ids = np.where(rng.random((T, K)) < 0.95, E - 1, rng.integers(0, E, (T, K)))
    else:
        ids = rng.integers(0, E, (T, K))
    if kind == "dropped":    # no expert, and numbers outside the range
        ids = np.where(rng.random((T, K)) < 0.3, rng.choice([-1, -7, E, E + 1, 2 ** 31 - 1, -2 ** 31], (T, K)), ids)
    ids = ids.astype(np.int32)
    got = [_np(x) for x in nvq.moe_sort(_dev(ids), E)]
    for a, b, name in zip(got, _sort_ref(ids, E), ("tok_idx", "grp_off", "pos")):
        assert np.array_equal(a, b), name
    if T * K <= 300:
        for a, b in zip(got, moe.sort(ids, E)):
            assert np.array_equal(a, b)


def test_sort_nothing_left(nvq):
    for T, K in ((0, 4), (3, 2), (9000, 8)):
        tok, off, pos = nvq.moe_sort(torch.full((T, K), -1, dtype=torch.int32, device=DEV), 17)
        assert not off.any() and (tok == -1).all() and (pos == -1).all()


# ---- experts' products ----------------------------------------------------------
def _experts(rng, G, m, k, big=False):
    packed = rng.integers(0, 256, (G, m, k // 2), dtype=np.uint8)
    scales = rng.integers(0x20 if not big else 0x70, 0x7F, (G, m, k // 16), dtype=np.uint8)
    g = (rng.random(G) + 0.5).astype(np.float32) * np.float32(1e-3)
    return packed, scales, g


def _offsets(rng, G, rows, kind):
    if kind == "one":
        cnt = np.zeros(G, dtype=np.int64)
        cnt[G // 2] = rows
    elif kind == "skewed":
        p = (np.arange(1, G + 1) ** -1.3)[rng.permutation(G)]
        cnt = rng.multinomial(rows, p / p.sum())
    else:
        cnt = rng.multinomial(rows, np.ones(G) / G)
    return np.concatenate([[0], np.cumsum(cnt)]).astype(np.int64)


def _check_product(Y, ref, mag, depth, dtype):
    bound = mag * ((depth / 16 + 16) * 2.0 ** -23) + np.abs(ref) * _half(dtype) + 1e-30
    assert np.all(np.abs(_np(Y) - ref) <= bound)


SHAPES = [  # n tokens, rows, G, m, k
    (1, 1, 1, 1, 16), (1, 8, 256, 64, 128), (3, 5, 7, 33, 48), (1, 8, 16, 100, 4096), (20, 64, 5, 130, 272),
    (64, 512, 40, 96, 512), (100, 300, 24, 203, 1040), (300, 900, 3, 256, 384), (257, 257, 1, 512, 2064),
    (700, 2100, 10, 129, 160), (900, 3600, 6, 320, 544), (1500, 9000, 4, 272, 336), (2048, 8192, 3, 513, 128),
    (50, 70, 1000, 40, 64), (40, 1500, 600, 24, 32), (3000, 9001, 70, 1800, 48), (10, 10, 2, 5, 2320)]


@pytest.mark.parametrize("n,rows,G,m,k", SHAPES)
@pytest.mark.parametrize("kind", ["even", "skewed", "one"])
def test_product(nvq, n, rows, G, m, k, kind):
    rng = np.random.default_rng([n, rows, G, m, k])
    packed, scales, g = _experts(rng, G, m, k)
    W = moe.experts_matrices(packed, scales, g)
    off = _offsets(rng, G, rows, kind)
    tok = rng.integers(0, n, rows).astype(np.int32)
    X = torch.from_numpy(rng.standard_normal((n, k)).astype(np.float32)).to(torch.bfloat16)
    args = (_dev(packed), _dev(scales), _dev(g), _dev(off))
    Xg, ref, mag = _np(X)[tok], np.zeros((rows, m)), np.zeros((rows, m))
    for e in range(G):
        r = slice(off[e], off[e + 1])
        ref[r], mag[r] = Xg[r] @ W[e].T, np.abs(Xg[r]) @ np.abs(W[e]).T
    for dtype in DTYPES.values():
        _check_product(nvq.nvfp4_gemm_grouped(X.to(DEV), *args, tok_idx=_dev(tok), out_dtype=dtype), ref, mag, k, dtype)
    direct = nvq.nvfp4_gemm_grouped(_dev(Xg, torch.bfloat16), *args)   # the rows already in order
    _check_product(direct, ref, mag, k, torch.float32)
    dY = torch.from_numpy(rng.standard_normal((rows, m)).astype(np.float32)).to(torch.bfloat16)
    ref, mag = np.zeros((rows, k)), np.zeros((rows, k))
    for e in range(G):
        r = slice(off[e], off[e + 1])
        ref[r], mag[r] = _np(dY)[r] @ W[e], np.abs(_np(dY)[r]) @ np.abs(W[e])
    for dtype in DTYPES.values():
        _check_product(nvq.nvfp4_gemm_grouped_dx(dY.to(DEV), *args, out_dtype=dtype), ref, mag, m, dtype)


def test_product_of_one_token_per_row_count(nvq):
    # every number of rows around the kernels' tile heights, in one expert of three
    rng = np.random.default_rng(6)
    G, m, k = 3, 72, 256
    packed, scales, g = _experts(rng, G, m, k)
    W = moe.experts_matrices(packed, scales, g)
    args = (_dev(packed), _dev(scales), _dev(g))
    for rows in (1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257):
        X = torch.from_numpy(rng.standard_normal((rows, k)).astype(np.float32)).to(torch.bfloat16)
        off = np.array([0, 0, rows, rows], dtype=np.int64)
        Y = nvq.nvfp4_gemm_grouped(X.to(DEV), *args, _dev(off))
        _check_product(Y, _np(X) @ W[1].T, np.abs(_np(X)) @ np.abs(W[1]).T, k, torch.float32)
        dX = nvq.nvfp4_gemm_grouped_dx(X.to(DEV)[:, :m], *args, _dev(off))
        _check_product(dX, _np(X)[:, :m] @ W[1], np.abs(_np(X)[:, :m]) @ np.abs(W[1]), m, torch.float32)


@pytest.mark.parametrize("rows,m,k", [(6, 40, 128), (40, 64, 256), (500, 136, 160)])
def test_product_strides_tails_and_bad_tokens(nvq, rows, m, k):
    rng = np.random.default_rng([rows, m, k])
    G, n = 5, 30
    packed, scales, g = _experts(rng, G, m, k)
    W = moe.experts_matrices(packed, scales, g)
    used = rows - 3                                     # rows behind the last group
    off = np.array([0, 0, used // 2, used // 2, used, used], dtype=np.int64)
    tok = rng.integers(0, n, rows).astype(np.int32)
    tok[:4] = [-1, n, 2 ** 31 - 1, -2 ** 31]            # not tokens: rows of zeros
    wide = torch.from_numpy(rng.standard_normal((n, k + 24)).astype(np.float32)).to(DEV, torch.bfloat16)
    X = wide[:, 8:8 + k]
    assert X.data_ptr() % 16 == 0
    args = (_dev(packed), _dev(scales), _dev(g), _dev(off))
    ref = moe.grouped_matmul(_np(X), W, off, tok)
    mag = moe.grouped_matmul(np.abs(_np(X)), np.abs(W), off, tok)
    for dtype in DTYPES.values():
        Yw = torch.full((rows, m + 5), 7.0, dtype=dtype, device=DEV)
        nvq.nvfp4_gemm_grouped(X, *args, tok_idx=_dev(tok), Y=Yw[:, 3:3 + m])
        assert (Yw[used:] == 7).all() and (Yw[:, :3] == 7).all() and (Yw[:, 3 + m:] == 7).all()
        assert (Yw[:2, 3:3 + m] == 0).all()
        _check_product(Yw[:used, 3:3 + m], ref[:used], mag[:used], k, dtype)
        dYw = torch.from_numpy(rng.standard_normal((rows, m + 3)).astype(np.float32)).to(DEV, torch.bfloat16)
        dY = dYw[:, 1:1 + m]                            # rows at any 2-byte place
        dXw = torch.full((rows, k + 7), 7.0, dtype=dtype, device=DEV)
        nvq.nvfp4_gemm_grouped_dx(dY, *args, dX=dXw[:, 1:1 + k])
        assert (dXw[used:] == 7).all() and (dXw[:, :1] == 7).all() and (dXw[:, 1 + k:] == 7).all()
        rdx = moe.grouped_matmul_dx(_np(dY), W, off)
        mdx = moe.grouped_matmul_dx(np.abs(_np(dY)), np.abs(W), off)
        _check_product(dXw[:used, 1:1 + k], rdx[:used], mdx[:used], m, dtype)


@pytest.mark.parametrize("rows", [4, 40, 700])
def test_product_non_finite_stays_in_its_row_or_channel(nvq, rows):
    rng = np.random.default_rng(8)
    G, m, k = 2, 70, 256
    packed, scales, g = _experts(rng, G, m, k)
    packed[0, 5], scales[0, 5] = 0, 0x7F                # a weight row that the quantizer rejected
    scales[1, 9, 3] |= 0x80                             # negative block scale, as nvfp4_dequantize takes it
    off = np.array([0, rows // 2, rows], dtype=np.int64)
    X = torch.from_numpy(rng.standard_normal((rows, k)).astype(np.float32)).to(DEV, torch.bfloat16)
    X[1, 7], X[rows - 1, 200] = float("nan"), float("inf")
    args = (_dev(packed), _dev(scales), _dev(g), _dev(off))
    Y = _np(nvq.nvfp4_gemm_grouped(X, *args))
    bad = np.zeros((rows, m), dtype=bool)
    bad[:rows // 2, 5] = bad[1] = bad[rows - 1] = True
    assert np.isfinite(Y[~bad]).all() and np.isnan(Y[1]).all() and np.isnan(Y[:rows // 2, 5]).all()
    assert not np.isfinite(Y[rows - 1]).any()
    W = np.stack([_np(nvq.nvfp4_dequantize(_dev(packed[e]), _dev(scales[e]), _dev(g[e:e + 1]))) for e in range(G)])
    Xn = np.nan_to_num(_np(X), nan=0.0, posinf=0.0)
    Wn = np.nan_to_num(W)
    for e in range(G):
        r = slice(off[e], off[e + 1])
        ref, mag = Xn[r] @ Wn[e].T, np.abs(Xn[r]) @ np.abs(Wn[e]).T
        ok = ~bad[r]
        assert np.all(np.abs(Y[r] - ref)[ok] <= (mag * ((k / 16 + 20) * 2.0 ** -23) + 1e-30)[ok])


def test_product_equals_single_matrix_product_of_each_expert(nvq):
    # the same codes through nvfp4_gemm, expert by expert; codes at 8 modulo 16 bytes (an odd number of 8-byte rows)
    rng = np.random.default_rng(9)
    G, m, k, n = 4, 3, 16, 50
    packed, scales, g = _experts(rng, G + 1, m, k)
    codes = _dev(packed)[1:]
    assert codes.data_ptr() % 16 == 8 and codes.is_contiguous()
    sc, gd = _dev(scales)[1:], _dev(g)[1:]
    off = np.array([0, 10, 10, 30, n], dtype=np.int64)
    X = torch.from_numpy(rng.standard_normal((n, k)).astype(np.float32)).to(DEV, torch.bfloat16)
    Y = nvq.nvfp4_gemm_grouped(X, codes, sc, gd, _dev(off))
    for e in range(G):
        if off[e] == off[e + 1]:
            continue
        one = nvq.nvfp4_gemm(X[off[e]:off[e + 1]].clone(), codes[e].clone(), sc[e].clone(), gd[e:e + 1].clone())
        mag = np.abs(_np(X)[off[e]:off[e + 1]]) @ np.abs(moe.experts_matrices(packed[e + 1:e + 2], scales[e + 1:e + 2], g[e + 1:e + 2])[0]).T
        assert np.all(np.abs(_np(Y[off[e]:off[e + 1]]) - _np(one)) <= 2 * mag * (17 * 2.0 ** -23))


def test_product_wide_weights_and_offsets_out_of_range(nvq):
    # experts behind 2^31 weight bytes, and offsets that the call clamps into [0, rows] (in bounds; the rows are undefined)
    G, m, k = 40, 7168, 16384
    codes = torch.zeros(G, m, k // 2, dtype=torch.uint8, device=DEV)
    scales = torch.full((G, m, k // 16), 0x38, dtype=torch.uint8, device=DEV)   # 1.0
    g = torch.ones(G, device=DEV)
    codes[G - 1].fill_(0x22)                                                    # all 1.0
    codes[G - 1, 11] = 0xAA                                                     # all -1.0
    off = torch.zeros(G + 1, dtype=torch.int64, device=DEV)
    off[G] = 9
    X = torch.ones(9, k, dtype=torch.bfloat16, device=DEV)
    Y = nvq.nvfp4_gemm_grouped(X, codes, scales, g, off)
    assert (Y[:, 11] == -k).all() and (Y[:, :11] == k).all() and (Y[:, 12:] == k).all()
    dX = nvq.nvfp4_gemm_grouped_dx(torch.ones(9, m, dtype=torch.bfloat16, device=DEV), codes, scales, g, off)
    assert (dX == m - 2).all()
    guard = torch.full((11, m), 7.0, device=DEV)
    off[G], off[3] = 1 << 40, -5
    nvq.nvfp4_gemm_grouped(X, codes, scales, g, off, Y=guard[1:10])
    assert (guard[0] == 7).all() and (guard[10] == 7).all()


@pytest.mark.parametrize("rows,m", [(5, 40), (300, 70), (700, 300)])
def test_product_activations_past_4_gib(nvq, rows, m):
    # rows of X that lie 2^32 bytes and more behind its start (a wide row stride)
    rng = np.random.default_rng(rows)
    G, n, k, ldx = 3, 270, 272, 1 << 23
    packed, scales, g = _experts(rng, G, m, k)
    W = moe.experts_matrices(packed, scales, g)
    X = torch.empty(n, ldx, dtype=torch.bfloat16, device=DEV)[:, :k]
    X.copy_(torch.from_numpy(rng.standard_normal((n, k)).astype(np.float32)))
    assert (n - 1) * ldx * 2 > 2 ** 32
    off = np.array([0, rows // 3, rows - 1, rows], dtype=np.int64)
    tok = rng.integers(0, n, rows).astype(np.int32)
    tok[-1], tok[0] = n - 1, 257
    Y = nvq.nvfp4_gemm_grouped(X, _dev(packed), _dev(scales), _dev(g), _dev(off), tok_idx=_dev(tok))
    _check_product(Y, moe.grouped_matmul(_np(X), W, off, tok), moe.grouped_matmul(np.abs(_np(X)), np.abs(W), off, tok), k,
                   torch.float32)


# ---- weighted sum -----------------------------------------------------------------
def _positions(rng, T, K, rows, dropped):
    pos = rng.permutation(max(rows, T * K))[:T * K].reshape(T, K).astype(np.int32)   # distinct; those >= rows name no row
    if dropped:
        pos[rng.random((T, K)) < 0.3] = -1
        pos[-1] = -1
    return pos


@pytest.mark.parametrize("yt", ["f32", "bf16"])
@pytest.mark.parametrize("ot", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,d", [(1, 1, 1), (1, 8, 4096), (37, 8, 512), (5, 3, 7), (100, 6, 2056), (64, 2, 1001),
                                   (9, 64, 40), (1030, 1, 136)])
def test_combine_and_gradient(nvq, T, K, d, yt, ot):
    rng = np.random.default_rng([T, K, d])
    yt, ot = DTYPES[yt], DTYPES[ot]
    for dropped in (False, True):
        rows = T * K + 3 if not dropped else max(1, T * K - 2)
        pos = _positions(rng, T, K, rows, dropped)
        Y = torch.from_numpy(rng.standard_normal((rows, d)).astype(np.float32)).to(yt)
        w = rng.standard_normal((T, K)).astype(np.float32)
        for weights in (w, None):
            wd = None if weights is None else _dev(weights)
            out = nvq.moe_combine(Y.to(DEV), _dev(pos), wd, out_dtype=ot)
            ref = moe.combine(_np(Y), pos, weights)
            mag = moe.combine(np.abs(_np(Y)), pos, None if weights is None else np.abs(weights))
            assert np.all(np.abs(_np(out) - ref) <= K * U * mag + np.abs(ref) * _half(ot) + 1e-37)
            dout = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(ot)
            dY0 = torch.full((rows, d), 7.0, dtype=yt, device=DEV)
            dY, dw = nvq.moe_combine_backward(dout.to(DEV), Y.to(DEV), _dev(pos), wd, dY=dY0)
            rdY, rdw = moe.combine_backward(_np(dout), _np(Y), pos, weights)
            named = np.zeros(rows, dtype=bool)
            named[pos[(pos >= 0) & (pos < rows)]] = True
            assert (_np(dY)[~named] == 7).all()
            assert np.all(np.abs(_np(dY) - rdY)[named] <= (np.abs(rdY) * (U + _half(yt)))[named] + 1e-37)
            amag = moe.combine_backward(np.abs(_np(dout)), np.abs(_np(Y)), pos, weights)[1]
            assert np.all(np.abs(_np(dw) - rdw) <= d * U * amag + 1e-37)


def test_combine_strides_and_non_finite(nvq):
    rng = np.random.default_rng(11)
    T, K, d = 20, 4, 100
    wide = torch.from_numpy(rng.standard_normal((T * K, d + 9)).astype(np.float32)).to(DEV)
    pos = _dev(rng.permutation(T * K).reshape(T, K).astype(np.int32))
    w = torch.rand(T, K, device=DEV)
    for dtype in DTYPES.values():
        Y = wide.to(dtype)[:, 3:3 + d]
        ow = torch.full((T, d + 5), 7.0, device=DEV, dtype=dtype)
        nvq.moe_combine(Y, pos, w, out=ow[:, 1:1 + d])
        assert (ow[:, 0] == 7).all() and (ow[:, 1 + d:] == 7).all()
        assert torch.equal(ow[:, 1:1 + d], nvq.moe_combine(Y.contiguous(), pos, w))
        dout = ow[:, 1:1 + d]
        dYw = torch.full((T * K, d + 3), 7.0, device=DEV, dtype=dtype)
        _, dw = nvq.moe_combine_backward(dout, Y, pos, w, dY=dYw[:, 1:1 + d])
        dY2, dw2 = nvq.moe_combine_backward(dout.contiguous(), Y.contiguous(), pos, w)
        assert (dYw[:, 0] == 7).all() and (dYw[:, 1 + d:] == 7).all() and torch.equal(dYw[:, 1:1 + d], dY2)
        assert np.all(np.abs(_np(dw) - _np(dw2)) <= 2 * d * U * _np((dout.abs().float()[:, None] * Y.abs().float()[pos.long()]).sum(2)))
    # a NaN weight (a token whose router row was rejected) makes that token NaN, also where no row is named
    w[2] = float("nan")
    p2 = pos.clone()
    p2[2] = -1
    for p in (pos, p2):
        out = nvq.moe_combine(wide[:, :d].contiguous(), p, w)
        assert torch.isnan(out[2]).all() and torch.isfinite(out[[0, 1, 3, 19]]).all()
    empty = nvq.moe_combine(torch.zeros(0, 5, device=DEV), torch.full((3, 2), -1, dtype=torch.int32, device=DEV))
    assert (empty == 0).all()
    assert nvq.moe_combine(torch.zeros(4, 5, device=DEV), torch.zeros(0, 2, dtype=torch.int32, device=DEV)).shape == (0, 5)


# ---- the operators together -----------------------------------------------------
def _layer(nvq, X, logits, ex, K, renorm=True, dtype=torch.float32):
    ids, w = nvq.moe_topk(logits, K, renorm)
    tok, off, pos = nvq.moe_sort(ids, logits.shape[1])
    Y = nvq.nvfp4_gemm_grouped(X, *ex, off, tok_idx=tok, out_dtype=dtype)
    return nvq.moe_combine(Y, pos, w), (ids, w, tok, off, pos, Y)


def test_quantized_experts_end_to_end(nvq):
    """The router's sort feeds the grouped Hessians, the experts are quantized by the library, and the routed layer runs on
    them: tokens with a masked expert, padded tokens with none, and the layer's output and gradients against the oracle."""
    rng = np.random.default_rng(12)
    T, E, K, m, k = 1200, 6, 2, 48, 256
    X = torch.from_numpy((rng.standard_normal((T, k)) * np.exp(0.5 * rng.standard_normal(k))).astype(np.float32)).to(torch.bfloat16)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[:, 4] = -np.inf                              # an expert switched off
    logits[100:110] = -np.inf                           # padded tokens
    W = torch.from_numpy((0.02 * rng.standard_normal((E, m, k))).astype(np.float32)).to(DEV, torch.bfloat16)
    Xd, ld = X.to(DEV), _dev(logits)
    ids, w = nvq.moe_topk(ld, K)
    tok, off, pos = nvq.moe_sort(ids, E)
    H = nvq.hessian_accumulate_grouped(Xd, tok, off.tolist())
    V, _, info = nvq.factor_chol_batched(H + 1e-3 * torch.eye(k, device=DEV))
    g = torch.cat([nvq.nvfp4_global_scale(W[e]) for e in range(E)])
    q = nvq.gptq_nvfp4_quantize_batched(W, V, H, g, 8, nvq.FLAG_CHOL_FACTOR)
    ex = (q["codes"], q["scales"], g)
    out, (ids, w, tok, off, pos, Y) = _layer(nvq, Xd, ld, ex, K)
    rid, rw = moe.topk(logits, K, True)
    assert np.array_equal(_np(ids), rid)
    rtok, roff, rpos = moe.sort(rid, E)
    assert np.array_equal(_np(pos), rpos) and np.array_equal(_np(off), roff) and np.array_equal(_np(tok), rtok)
    Wq = moe.experts_matrices(q["codes"].cpu().numpy(), q["scales"].cpu().numpy(), _np(g))
    rY = moe.grouped_matmul(_np(X), Wq, roff, rtok)
    ref = moe.combine(rY, rpos, rw)
    mag = moe.combine(moe.grouped_matmul(np.abs(_np(X)), np.abs(Wq), roff, rtok), rpos, rw)
    ew = (2 * 10 + 32) * U
    assert np.all(np.abs(_np(out) - ref) <= mag * ((k / 16 + 16) * 2.0 ** -23 + K * U + ew) + 1e-30)
    assert (out[100:110] == 0).all()
    # the gradients, each against its oracle on the same inputs
    dout = torch.from_numpy(rng.standard_normal((T, m)).astype(np.float32)).to(DEV)
    dY, dw = nvq.moe_combine_backward(dout, Y, pos, w)
    n = int(off[-1])
    dYb = torch.zeros(T * K, m, dtype=torch.bfloat16, device=DEV)
    dYb[:n] = dY[:n].to(torch.bfloat16)
    dX = nvq.moe_combine(nvq.nvfp4_gemm_grouped_dx(dYb, *ex, off), torch.where(pos >= 0, pos, -1))
    dl = nvq.moe_topk_backward(ld, ids, w, dw)
    rdX = moe.combine(moe.grouped_matmul_dx(_np(dYb), Wq, roff), rpos)
    mdX = moe.combine(moe.grouped_matmul_dx(np.abs(_np(dYb)), np.abs(Wq), roff), rpos)
    assert np.all(np.abs(_np(dX) - rdX) <= mdX * ((m / 16 + 16) * 2.0 ** -23 + K * U) + 1e-30)
    rdY, rdw = moe.combine_backward(_np(dout), rY, rpos, rw)
    rdl = moe.topk_backward(logits, rid, rw, rdw, True)
    edw = moe.combine_backward(np.abs(_np(dout)), moe.grouped_matmul(np.abs(_np(X)), np.abs(Wq), roff, rtok), rpos)[1]
    edw = (edw * ((k / 16 + 16) * 2.0 ** -23 + m * U)).sum(1, keepdims=True)   # of the products, then of the dot products
    assert np.all(np.abs(_np(dl) - rdl) <= 2 * edw + (ew + 16 * U) * (np.abs(rdw * rw).sum(1, keepdims=True) + np.abs(rdw).max(1, keepdims=True)) + 1e-30)
    assert np.all(_np(dl)[100:110] == 0) and np.all(_np(dl)[:, 4] == 0)


@pytest.mark.parametrize("T,E,K,m,k", [(1, 64, 8, 256, 512), (33, 16, 4, 200, 256), (3000, 8, 6, 130, 272)])
def test_layer_captured_and_replayed(nvq, T, E, K, m, k):
    """The forward and the gradients in one graph, replayed on new inputs between eager runs of the same shapes."""
    rng = np.random.default_rng([T, E])
    packed, scales, g = _experts(rng, E, m, k)
    ex = (_dev(packed), _dev(scales), _dev(g))
    X = torch.zeros(T, k, dtype=torch.bfloat16, device=DEV)
    logits = torch.zeros(T, E, device=DEV)
    dout = torch.zeros(T, m, device=DEV)

    def step():
        out, (ids, w, tok, off, pos, Y) = _layer(nvq, X, logits, ex, K)
        dY, dw = nvq.moe_combine_backward(dout, Y, pos, w)
        dX = nvq.moe_combine(nvq.nvfp4_gemm_grouped_dx(dY.to(torch.bfloat16), *ex, off), pos)
        return out, ids, tok, off, pos, dX, nvq.moe_topk_backward(logits, ids, w, dw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(4):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        X.copy_(torch.randn(T, k, generator=gen, device=DEV))
        logits.copy_(torch.randn(T, E, generator=gen, device=DEV))
        dout.copy_(torch.randn(T, m, generator=gen, device=DEV))
        graph.replay()
        got = [x.clone() for x in captured]
        eager = step()
        torch.cuda.synchronize()
        for a, b in zip(got, eager):
            assert torch.equal(a, b)   # every sum has a fixed order


def test_two_streams_at_once(nvq):
    """The same calls on two streams with different inputs give what each gives alone."""
    rng = np.random.default_rng(13)
    T, E, K, m, k = 5000, 32, 4, 256, 256
    packed, scales, g = _experts(rng, E, m, k)
    ex = (_dev(packed), _dev(scales), _dev(g))
    ins = [(torch.randn(T, k, device=DEV).to(torch.bfloat16), torch.randn(T, E, device=DEV)) for _ in range(2)]
    alone = [_layer(nvq, *i, ex, K)[0] for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    outs = [[], []]
    for _ in range(3):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[j].append(_layer(nvq, *ins[j], ex, K)[0])
    torch.cuda.synchronize()
    for j in range(2):
        for o in outs[j]:
            assert torch.equal(o, alone[j])


def test_python_functions_refuse_wrong_tensors(nvq):
    f = torch.zeros(4, 32, device=DEV)
    b = f.to(torch.bfloat16)
    ids = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    codes = torch.zeros(3, 8, 16, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(3, 8, 2, dtype=torch.uint8, device=DEV)
    g = torch.ones(3, device=DEV)
    off = torch.zeros(4, dtype=torch.int64, device=DEV)
    bad = [
        (TypeError, lambda: nvq.moe_topk(f.double(), 2)), (ValueError, lambda: nvq.moe_topk(f.t(), 2)),
        (ValueError, lambda: nvq.moe_topk(f[0], 2)), (nvq.NvqError, lambda: nvq.moe_topk(f, 33)),
        (nvq.NvqError, lambda: nvq.moe_topk(f, 0)), (nvq.NvqError, lambda: nvq.moe_topk(f, -1)),
        (TypeError, lambda: nvq.moe_sort(ids.long(), 4)), (ValueError, lambda: nvq.moe_sort(ids[:, :1], 4)),
        (nvq.NvqError, lambda: nvq.moe_sort(ids, 0)), (nvq.NvqError, lambda: nvq.moe_sort(ids, -3)),
        (nvq.NvqError, lambda: nvq.moe_sort(ids, 1025)), (nvq.NvqError, lambda: nvq.moe_sort(ids[:, :0].contiguous(), 4)),
        (ValueError, lambda: nvq.moe_topk_backward(f, ids, f[:, :2], f[:, :2])),
        (ValueError, lambda: nvq.moe_topk_backward(f, ids, f[:3, :2].contiguous(), f[:, :2].contiguous())),
        (TypeError, lambda: nvq.nvfp4_gemm_grouped(f, codes, scales, g, off)),
        (ValueError, lambda: nvq.nvfp4_gemm_grouped(b[:, :16], codes, scales, g, off)),
        (ValueError, lambda: nvq.nvfp4_gemm_grouped(b, codes, scales[:2], g, off)),
        (ValueError, lambda: nvq.nvfp4_gemm_grouped(b, codes, scales, g, off[:3])),
        (TypeError, lambda: nvq.nvfp4_gemm_grouped(b, codes, scales, g, off.int())),
        (TypeError, lambda: nvq.nvfp4_gemm_grouped(b, codes, scales, g, off, tok_idx=off)),
        (ValueError, lambda: nvq.nvfp4_gemm_grouped(b, codes, scales, g, off, Y=torch.zeros(5, 8, device=DEV))),
        (ValueError, lambda: nvq.nvfp4_gemm_grouped(b, codes, scales, g.cpu(), off)),
        (ValueError, lambda: nvq.nvfp4_gemm_grouped(b, codes[:, ::2], scales[:, ::2], g, off)),
        (nvq.NvqError, lambda: nvq.nvfp4_gemm_grouped(torch.zeros(4, 36, device=DEV).to(torch.bfloat16)[:, :32], codes, scales, g, off)),
        (TypeError, lambda: nvq.nvfp4_gemm_grouped_dx(f[:, :8], codes, scales, g, off)),
        (ValueError, lambda: nvq.nvfp4_gemm_grouped_dx(b, codes, scales, g, off)),
        (ValueError, lambda: nvq.moe_combine(f.t(), ids)), (TypeError, lambda: nvq.moe_combine(f, ids.long())),
        (ValueError, lambda: nvq.moe_combine(f, ids, f[:3, :2].contiguous())),
        (ValueError, lambda: nvq.moe_combine(f, ids, out=f[:, :30])),
        (ValueError, lambda: nvq.moe_combine(f[:1].expand(4, 32), ids)),
        (ValueError, lambda: nvq.moe_combine_backward(f, f[:, :16], ids)),
        (TypeError, lambda: nvq.moe_combine_backward(f, f, ids, dY=b)),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            print("accepted", i)


# ---- calls at the edges of what is documented -------------------------------------
@pytest.mark.parametrize("T,E,K", [(5, 6, 4), (9000, 60, 8)])
@pytest.mark.parametrize("renorm", [True, False])
def test_topk_gradient_of_an_expert_named_twice(nvq, T, E, K, renorm):
    """The slots of one expert add up (at most K = 8 terms: 8 u of their absolute sum on top of the bound above)."""
    rng = np.random.default_rng([T, E])
    l = _dev((rng.standard_normal((T, E))).astype(np.float32))
    ids = rng.integers(0, 3, (T, K)).astype(np.int32)
    w = rng.random((T, K)).astype(np.float32)
    dw = rng.standard_normal((T, K)).astype(np.float32)
    got = _np(nvq.moe_topk_backward(l, _dev(ids), _dev(w), _dev(dw), renorm=renorm))
    ref = moe.topk_backward(_np(l), ids, w.astype(np.float64), dw, renorm)
    D = float((l.max(dim=1).values - l.min(dim=1).values).max())
    size = np.abs(dw).sum(axis=1, keepdims=True) * (1 + np.abs(w).max() * K)   # above every |term| sum
    assert np.all(np.abs(got - ref) <= (2 * D + 64 + 2 * K) * U * size)


def test_more_tokens_than_one_launch_takes(nvq):
    """A launch holds fewer than 2^32 threads: 2^28 tokens of the router, 2^26 of the weighted sum (one column)."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    T = 2 ** 28 + 70
    l = torch.randint(-8, 8, (T, 2), generator=gen, device=DEV, dtype=torch.int8).to(torch.bfloat16)
    ids, w = nvq.moe_topk(l, 1, renorm=False)
    assert torch.equal(ids[:, 0], (l[:, 1] > l[:, 0]).int())
    dl = nvq.moe_topk_backward(l, ids, w, w, renorm=False)
    del l, ids
    # the two experts' gradients cancel, up to a bf16 rounding of each and 8 fp32 roundings of terms below 1
    assert bool(((w > 0.49) & (w <= 1)).all())
    assert bool(((dl[:, 0].float() + dl[:, 1].float()).abs() <= 2 * 2.0 ** -8 * dl[:, 0].float().abs() + 8 * U).all())
    del w, dl
    T = 2 ** 26 + 70
    pos = torch.arange(T - 1, -1, -1, device=DEV, dtype=torch.int32)[:, None]
    y = torch.randint(-99, 99, (T, 1), generator=gen, device=DEV, dtype=torch.int32).float()
    w = torch.randint(-9, 9, (T, 1), generator=gen, device=DEV, dtype=torch.int32).float()
    assert torch.equal(nvq.moe_combine(y, pos, w), y.flip(0) * w)
    dy, dw = nvq.moe_combine_backward(y, y, pos, w)
    assert torch.equal(dy, (y * w).flip(0)) and torch.equal(dw, y * y.flip(0))


def test_sort_of_the_most_slots(nvq):
    """3 times 715827882 slots, the largest multiple of 3 below 2^31."""
    T, K, E = (2 ** 31 - 1) // 3, 3, 5
    gen = torch.Generator(device=DEV).manual_seed(6)
    ids = torch.randint(-1, E, (T, K), generator=gen, device=DEV, dtype=torch.int32)
    tok, off, pos = nvq.moe_sort(ids, E)
    total, step, where = int(off[E]), 2 ** 22, 0
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        assert hi - lo == sum(int((ids[a:a + 2 ** 27] == e).sum()) for a in range(0, T, 2 ** 27))
        for a in range(lo, hi - 1, 2 ** 28):   # the tokens of an expert in order
            assert bool((tok[a + 1:min(a + 2 ** 28 + 1, hi)] >= tok[a:min(a + 2 ** 28, hi - 1)]).all())
    for a in list(range(0, T, T // 8)) + [T - step]:
        b = min(a + step, T)
        i, p = ids[a:b], pos[a:b].long()
        has = i >= 0
        assert torch.equal(p >= 0, has)
        t = torch.arange(a, b, device=DEV)[:, None].expand(b - a, K)[has]
        assert torch.equal(tok[p[has]].long(), t)
        assert bool(((off[i[has].long()] <= p[has]) & (p[has] < off[i[has].long() + 1])).all())
    for a in range(0, T, 2 ** 26):
        p = pos[a:a + 2 ** 26].reshape(-1)
        where += int(p[p >= 0].long().sum())
    assert where == total * (total - 1) // 2
    assert bool((tok[total:] == -1).all())


@pytest.mark.parametrize("T,E", [(5000, e) for e in (1, 3, 16, 17, 60, 128, 200, 256)] +
                         [(70, e) for e in (2, 64, 65, 200, 512, 1000, 1024)])
@pytest.mark.parametrize("K", [1, 2, 8, 9, 16])
def test_topk_choice_for_every_row_length(nvq, T, E, K):
    """Ids and order against a stable sort, with many equal values and some experts masked."""
    K = min(K, E)
    rng = np.random.default_rng([T, E, K])
    for dtype in DTYPES.values():
        l = torch.from_numpy(rng.integers(-20, 20, (T, E)).astype(np.float32)).to(dtype)
        l[:, E // 2:] += torch.from_numpy(rng.standard_normal((T, E - E // 2)).astype(np.float32)).to(dtype)
        l[torch.from_numpy(rng.random((T, E)) < 0.3)] = float("-inf")
        v, i = torch.sort(l, dim=1, descending=True, stable=True)
        ref = torch.where(v[:, :K] == float("-inf"), -1, i[:, :K])
        ids, _ = nvq.moe_topk(l.to(DEV), K)
        assert torch.equal(ids.cpu().long(), ref)


@pytest.mark.parametrize("T,E,K", [(20, 60, 3), (20, 300, 12), (5000, 60, 3), (5000, 60, 12)])
def test_topk_rejects_every_nan_and_infinity(nvq, T, E, K):
    """NaNs of both signs, quiet and signalling, and +inf, anywhere in the row; the largest finite values are kept."""
    bits = {torch.float32: (torch.int32, [0x7FC00000, 0x7F800001, 0x7FFFFFFF, -0x400000, -0x7FFFFF, -1, 0x7F800000]),
            torch.bfloat16: (torch.int16, [0x7FC0, 0x7F81, 0x7FFF, -0x40, -0x7F, -1, 0x7F80])}
    rng = np.random.default_rng([T, E, K])
    for dtype, (as_int, values) in bits.items():
        l = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(dtype)
        bad = torch.zeros(T, dtype=torch.bool)
        for j, b in enumerate(values):
            for t in (2 * j, T - 1 - 2 * j if T > 100 else 2 * j):
                l.view(as_int)[t, int(rng.integers(E))] = b
                bad[t] = True
        l[1, 3], l[3, 5] = torch.finfo(dtype).max, torch.finfo(dtype).min
        ids, w = nvq.moe_topk(l.to(DEV), K)
        assert torch.equal((ids == -1).all(1).cpu(), bad) and torch.equal(torch.isnan(w).all(1).cpu(), bad)
        assert not torch.isnan(w[~bad.to(DEV)]).any() and int(ids[1, 0]) == 3


@pytest.mark.parametrize("k", [128, 384, 496, 512, 528, 640, 656, 768, 784, 896, 1040, 1168])
@pytest.mark.parametrize("n,rows,G,m", [(900, 5000, 30, 1800), (60, 200, 30, 1800), (3, 9, 30, 64)])
def test_product_for_every_end_of_k(nvq, n, rows, G, m, k):
    """Each tile size (128 x 256, 64 x 128, few rows) with k ending in every part of its steps."""
    test_product(nvq, n, rows, G, m, k, "skewed")
