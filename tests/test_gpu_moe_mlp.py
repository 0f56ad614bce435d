"""GPU parity of the whole mixture-of-experts MLP for a few tokens against the fp64 oracle.

Error bounds, with u = 2^-24.  A sum over n of bf16-exact products on the matrix cores, in parts joined by fp32 additions:
(n / 16 + 16) 2^-23 sum |terms|, as in the experts' products' tests; g once, u.  gate and up carry eg and eu of that; silu's
slope is below 1.1 and silu itself is within 10 u, so the activation w silu(gate) up carries |w| (1.1 eg |up| + |silu| eu +
1.1 eg eu) + 16 u of itself, and K u for the weight's sum over slots.  It is held as hi + lo, each bf16: 2^-16.  These errors
pass through |D|; the second sum has 2 K h terms, and joining K experts and 8 waves adds K + 16 roundings.  A bf16 result adds 2^-8.
"""

import numpy as np
import pytest
import torch

from oracle import codec, mlp, moe

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


def _np(t):
    return t.double().cpu().numpy() if t.dtype.is_floating_point else t.cpu().numpy()


def _experts(rng, E, m, k, size):
    """(device tensors, dequantized fp64 [E, m, k])."""
    codes = rng.integers(0, 16, (E, m, k), dtype=np.uint8)
    scales = rng.integers(0x20, 0x60, (E, m, k // 16), dtype=np.uint8)
    g = ((rng.random(E) + 0.5) * size / 32).astype(np.float32)
    packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
    s = np.array([codec.e4m3_decode(b) for b in range(0x7F)])[scales]
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    w = np.where(codes & 8, -1.0, 1.0) * grid[codes & 7] * np.repeat(s, 16, axis=2) * g.astype(np.float64)[:, None, None]
    return tuple(torch.from_numpy(a).to(DEV) for a in (packed, scales, g)), w


def _layer(rng, E, d, h, m):
    gu, wgu = _experts(rng, E, 2 * h, d, 0.5 / np.sqrt(d))
    dn, wdn = _experts(rng, E, m, h, 0.5 / np.sqrt(h))
    return gu, dn, wgu, wdn


def _bound(X, wgu, wdn, ids, w, ref, dtype):
    T, K = ids.shape
    h, d = wdn.shape[2], X.shape[1]
    out = np.zeros_like(ref)
    for t in range(T):
        for e in np.unique(ids[t]):
            if not 0 <= e < wdn.shape[0]:
                continue
            we = np.abs(w[t][ids[t] == e]).sum()
            y = wgu[e] @ X[t]
            err = ((d / 16 + 16) * 2.0 ** -23 + U) * (np.abs(wgu[e]) @ np.abs(X[t])) + U * np.abs(y)
            gate, up, eg, eu = y[:h], y[h:], err[:h], err[h:]
            silu = gate * mlp.sigmoid(gate)
            act = we * np.abs(silu * up)
            ea = we * (1.1 * eg * np.abs(up) + np.abs(silu) * eu + 1.1 * eg * eu) + act * ((16 + K) * U + 2.0 ** -16)
            D = np.abs(wdn[e])
            out[t] += D @ (ea + (act + ea) * ((2 * K * h / 16 + 16 + K + 16) * 2.0 ** -23))
    return out + (2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 0) + 1e-30


def _check_out(out, X, wgu, wdn, ids, w, dtype):
    ref = mlp.moe_mlp(X, wgu, wdn, ids, w)
    assert np.all(np.abs(_np(out) - ref) <= _bound(X, wgu, wdn, ids, w, ref, dtype))


def _inputs(rng, T, d, E, gap=0):
    X = torch.from_numpy(rng.standard_normal((T, d + gap)).astype(np.float32)).to(torch.bfloat16).to(DEV)[:, :d]
    return X, torch.from_numpy((rng.standard_normal((T, E)) * 2).astype(np.float32)).to(DEV)


SIZES = [(1, 1, 1, 32, 48, 1), (1, 2, 1, 48, 32, 3), (3, 4, 2, 512, 1024, 20), (2, 8, 8, 4112, 1040, 33), (64, 4, 2, 528, 496, 18), (20, 64, 4, 4096, 512, 48), (1, 8, 2, 256, 256, 64), (1, 64, 8, 512, 128, 96), (2, 3, 3, 48, 80, 17), (5, 16, 4, 272, 304, 33),
         (15, 8, 2, 2064, 48, 16), (16, 32, 6, 256, 272, 40), (17, 8, 1, 528, 64, 100), (31, 60, 8, 128, 160, 31), (33, 1, 1, 256, 512, 48),
         (48, 24, 3, 80, 32, 257), (63, 200, 5, 64, 48, 20), (64, 16, 8, 288, 544, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K,d,h,m", SIZES)
def test_routed(nvq, T, E, K, d, h, m, renorm, dtype):
    rng = np.random.default_rng([T, E, d])
    gu, dn, wgu, wdn = _layer(rng, E, d, h, m)
    X, logits = _inputs(rng, T, d, E, gap=8 if T % 2 else 0)
    logits = logits.to(DTYPES[dtype])
    out, ids, w = nvq.nvfp4_moe_mlp(X, gu, dn, logits=logits, top_k=K, renorm=renorm, out_dtype=DTYPES[dtype])
    assert out.dtype == DTYPES[dtype] and out.shape == (T, m)
    rid, rw = moe.topk(_np(logits), K, renorm)
    assert np.array_equal(_np(ids), rid)
    D = np.ptp(_np(logits), axis=1)[:, None]
    assert np.all(np.abs(_np(w) - rw) <= (2 * D + 32) * U * rw + 1e-37)      # the router's own bound
    _check_out(out, _np(X), wgu, wdn, rid, _np(w), DTYPES[dtype])
    # the same layer with the routing given: the same bits
    again, ids2, w2 = nvq.nvfp4_moe_mlp(X, gu, dn, ids=ids, weights=w, out_dtype=DTYPES[dtype])
    assert ids2 is ids and w2 is w and torch.equal(again, out)


@pytest.mark.parametrize("T,E,K", [(2, 300, 40), (40, 1024, 64), (64, 1000, 20)])
def test_many_experts(nvq, T, E, K):
    rng = np.random.default_rng([T, E])
    gu, dn, wgu, wdn = _layer(rng, E, 32, 32, 24)
    X, logits = _inputs(rng, T, 32, E)
    out, ids, w = nvq.nvfp4_moe_mlp(X, gu, dn, logits=logits, top_k=K, out_dtype=torch.float32)
    rid, _ = moe.topk(_np(logits), K, True)
    assert np.array_equal(_np(ids), rid)
    _check_out(out, _np(X), wgu, wdn, rid, _np(w), torch.float32)


@pytest.mark.parametrize("T", [3, 20, 50])
def test_masked_and_rejected_tokens(nvq, T):
    """Fewer experts left than slots, none at all (zeros), and logits with a NaN or +inf (NaN)."""
    rng = np.random.default_rng(T)
    E, K, d, h, m = 12, 4, 96, 48, 40
    gu, dn, wgu, wdn = _layer(rng, E, d, h, m)
    X, logits = _inputs(rng, T, d, E)
    logits[0] = float("-inf")
    logits[1, 2:] = float("-inf")
    logits[T - 1, 5] = float("nan")
    if T > 10:
        logits[7, 3] = float("inf")
    out, ids, w = nvq.nvfp4_moe_mlp(X, gu, dn, logits=logits, top_k=K, out_dtype=torch.float32)
    o, i = _np(out), _np(ids)
    assert (i[0] == -1).all() and (o[0] == 0).all() and sorted(i[1]) == [-1, -1, 0, 1]
    bad = [T - 1] + ([7] if T > 10 else [])
    good = [t for t in range(T) if t not in bad]
    assert np.isnan(o[bad]).all() and (i[bad] == -1).all() and np.isnan(_np(w)[bad]).all()
    _check_out(out[good], _np(X)[good], wgu, wdn, i[good], _np(w)[good], torch.float32)


@pytest.mark.parametrize("T", [4, 30, 64])
def test_given_routing_edges(nvq, T):
    """Ids outside the experts, experts named twice, negative and zero weights, one expert for all, no expert for any."""
    rng = np.random.default_rng([T, 1])
    E, K, d, h, m = 9, 5, 112, 272, 35
    gu, dn, wgu, wdn = _layer(rng, E, d, h, m)
    X, _ = _inputs(rng, T, d, E)
    ids = rng.integers(-2, E + 2, (T, K)).astype(np.int32)
    ids[1] = 3
    ids[2] = [4, 4, 7, 4, -5]
    ids[3] = [2 ** 31 - 1, -2 ** 31, E, -1, E + 1]
    w = rng.standard_normal((T, K)).astype(np.float32)
    w[0, 1] = 0
    for i in (ids, np.full_like(ids, 8), np.full_like(ids, -1)):
        out, _, _ = nvq.nvfp4_moe_mlp(X, gu, dn, ids=torch.from_numpy(i).to(DEV), weights=torch.from_numpy(w).to(DEV), out_dtype=torch.float32)
        _check_out(out, _np(X), wgu, wdn, i, w.astype(np.float64), torch.float32)
    assert not _np(out).any()


@pytest.mark.parametrize("T", [2, 24, 64])
def test_non_finite_values_stay_with_their_tokens(nvq, T):
    """NaN in one token's X, a NaN weight of an empty slot, a rejected weight row of one expert: only who uses it sees it."""
    rng = np.random.default_rng([T, 2])
    E, K, d, h, m = 6, 2, 64, 32, 24
    gu, dn, wgu, wdn = _layer(rng, E, d, h, m)
    X, _ = _inputs(rng, T, d, E)
    ids = np.stack([np.arange(T) % 3, 3 + np.arange(T) % 2], 1).astype(np.int32)      # experts 0-2 and 3-4
    w = (rng.random((T, K)) + 0.5).astype(np.float32)
    idt, wt = torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV)
    clean = _np(nvq.nvfp4_moe_mlp(X, gu, dn, ids=idt, weights=wt, out_dtype=torch.float32)[0])

    def run(X=X, gu=gu, dn=dn, ids=idt, weights=wt):
        return _np(nvq.nvfp4_moe_mlp(X, gu, dn, ids=ids, weights=weights, out_dtype=torch.float32)[0])

    bad = X.clone()
    bad[T - 1, 5] = float("nan")
    o = run(X=bad)
    assert np.isnan(o[T - 1]).all() and np.array_equal(o[:T - 1], clean[:T - 1])
    s = dn[1].clone()
    s[1, 10] = 0x7F                                   # expert 1's output channel 10
    o = run(dn=(dn[0], s, dn[2]))
    users = (ids == 1).any(1)
    assert np.isnan(o[users, 10]).all() and np.array_equal(o[~users], clean[~users])
    assert np.array_equal(np.delete(o, 10, 1), np.delete(clean, 10, 1))
    s = gu[1].clone()
    s[4, 7] = 0x7F                                    # a gate row of expert 4
    o = run(gu=(gu[0], s, gu[2]))
    users = (ids == 4).any(1)
    assert np.isnan(o[users]).all() and np.array_equal(o[~users], clean[~users])
    s = dn[1].clone()
    s[5] = 0x7F                                       # an expert that nobody uses
    assert np.array_equal(run(dn=(dn[0], s, dn[2])), clean)
    i2, w2 = idt.clone(), wt.clone()
    i2[0, 1] = -1
    w2[0, 1] = float("nan")
    o = run(ids=i2, weights=w2)
    assert np.isnan(o[0]).all() and np.array_equal(o[1:], clean[1:])


def test_infinite_activation_stays_infinite(nvq):
    """A gate and an up value whose product passes fp32's range: infinities, no NaN out of the split into two parts."""
    d = h = 32
    one = torch.full((1, 2 * h, d // 2), 0x22, dtype=torch.uint8, device=DEV)        # all weights 1
    sc = torch.full((1, 2 * h, 2), 0x38, dtype=torch.uint8, device=DEV)
    g = torch.ones(1, device=DEV)
    X = torch.full((1, d), 3e30, dtype=torch.bfloat16, device=DEV)
    out, _, _ = nvq.nvfp4_moe_mlp(X, (one, sc, g), (one[:, :h].contiguous(), sc[:, :h].contiguous(), g), logits=torch.zeros(1, 1, device=DEV),
                                  top_k=1, out_dtype=torch.float32)
    assert bool(torch.isposinf(out).all())


def test_output_rows_apart_and_empty(nvq):
    rng = np.random.default_rng(8)
    E, K, d, h, m, T = 4, 2, 64, 64, 19, 10
    gu, dn, wgu, wdn = _layer(rng, E, d, h, m)
    X, logits = _inputs(rng, T, d, E)
    wide = torch.cat((logits, logits), 1)[:, 2:2 + E]                 # rows apart, at an odd element
    for dt in DTYPES.values():
        buf = torch.full((T + 2, m + 6), 7.0, dtype=dt, device=DEV)
        out = buf[1:T + 1, 3:3 + m]
        got, ids, w = nvq.nvfp4_moe_mlp(X, gu, dn, logits=wide, top_k=K, out=out)
        assert got is out
        _check_out(out, _np(X), wgu, wdn, _np(ids), _np(w), dt)
        out.fill_(7.0)
        assert bool((buf == 7.0).all())
    out, ids, w = nvq.nvfp4_moe_mlp(X[:0], gu, dn, logits=logits[:0], top_k=K)
    assert out.shape == (0, m) and ids.shape == (0, K)


# ---- the operators together -----------------------------------------------------------
def test_as_the_grouped_path(nvq):
    """The layer in two kernels against the same layer in six, which tokens past 64 take."""
    rng = np.random.default_rng(9)
    E, K, d, h, m, T = 16, 4, 256, 128, 96, 40
    gu, dn, wgu, wdn = _layer(rng, E, d, h, m)
    X, logits = _inputs(rng, T, d, E)
    out, ids, w = nvq.nvfp4_moe_mlp(X, gu, dn, logits=logits, top_k=K, out_dtype=torch.float32)
    ids6, w6 = nvq.moe_topk(logits, K)
    tok, off, pos = nvq.moe_sort(ids6, E)
    act = nvq.swiglu(nvq.nvfp4_gemm_grouped(X, *gu, off, tok_idx=tok), out_dtype=torch.bfloat16)
    out6 = nvq.moe_combine(nvq.nvfp4_gemm_grouped(act, *dn, off), pos, w6)
    assert torch.equal(ids, ids6)
    ref = mlp.moe_mlp(_np(X), wgu, wdn, _np(ids), _np(w))
    size = np.zeros_like(ref)
    for t in range(T):
        for e, we in zip(_np(ids)[t], _np(w)[t]):
            size[t] += we * (np.abs(wdn[e]) @ np.abs(mlp.swiglu((wgu[e] @ _np(X)[t])[None])[0]))
    tight = _bound(_np(X), wgu, wdn, _np(ids), _np(w), ref, torch.float32)
    assert np.all(np.abs(_np(out) - ref) <= tight)
    assert np.all(np.abs(_np(out6) - ref) <= 2 * tight + (2.0 ** -8 + 2.0 ** -16) * size)     # its activations are one bf16


def test_grouped_mlp_gradients(nvq):
    """Training through frozen experts: dX of product -> swiglu -> product -> weighted sum, against the formulas."""
    rng = np.random.default_rng(10)
    E, K, d, h, m, T = 5, 2, 64, 48, 64, 70
    gu, dn, wgu, wdn = _layer(rng, E, d, h, m)
    X, logits = _inputs(rng, T, d, E)
    ids, w = nvq.moe_topk(logits, K)
    tok, off, pos = nvq.moe_sort(ids, E)
    hid = nvq.nvfp4_gemm_grouped(X, *gu, off, tok_idx=tok, out_dtype=torch.bfloat16)
    act = nvq.swiglu(hid)
    Y = nvq.nvfp4_gemm_grouped(act, *dn, off, out_dtype=torch.bfloat16)
    dout = torch.from_numpy(rng.standard_normal((T, m)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    dY, _ = nvq.moe_combine_backward(dout, Y, pos, w, need_dweights=False)
    dact = nvq.nvfp4_gemm_grouped_dx(dY, *dn, off, out_dtype=torch.bfloat16)
    dhid = nvq.swiglu_backward(dact, hid)
    dX = nvq.moe_combine(nvq.nvfp4_gemm_grouped_dx(dhid, *gu, off), pos)
    ref, mag = np.zeros((T, d)), np.zeros((T, d))
    Xn, wn, idn, don = _np(X), _np(w), _np(ids), _np(dout)
    for t in range(T):
        for e, we in zip(idn[t], wn[t]):
            hidden = (wgu[e] @ Xn[t])[None]
            da = (we * don[t]) @ wdn[e]
            ref[t] += mlp.swiglu_backward(da[None], hidden)[0] @ wgu[e]
            gate, up = np.split(np.abs(hidden[0]), 2)
            size = np.concatenate((up * (1 + gate), gate)) * np.tile(np.abs(we * don[t]) @ np.abs(wdn[e]), 2)
            mag[t] += size @ np.abs(wgu[e])
    # six values on the way are rounded to bf16 (2^-8 each of what they pass on), |silu'| below 1.1 and |silu''| below 1
    assert np.all(np.abs(_np(dX) - ref) <= 8 * 2.0 ** -8 * 1.1 * mag)


def test_dense_mxfp4_mlp(nvq):
    """A dense MLP on 4-bit operands and its gradient: quantize once for gate and up, product, swiglu, product."""
    from oracle import mxfp4
    rng = np.random.default_rng(11)
    n, d, h = 150, 128, 96
    X = torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    W1 = nvq.mxfp4_quantize(torch.from_numpy((rng.standard_normal((2 * h, d)) * 0.1).astype(np.float32)).to(DEV))
    W2 = nvq.mxfp4_quantize(torch.from_numpy((rng.standard_normal((d, h)) * 0.1).astype(np.float32)).to(DEV))
    w1, w2 = (mxfp4.values(mxfp4.unpack(_np(c)), _np(s)) for c, s in (W1, W2))
    xc, xs = nvq.mxfp4_quantize(X)
    hid = nvq.mxfp4_gemm(xc, *W1, x_scales=xs, out_dtype=torch.bfloat16)
    parts = [nvq.mxfp4_gemm(xc, W1[0][i * h:(i + 1) * h], W1[1][i * h:(i + 1) * h], x_scales=xs, out_dtype=torch.bfloat16) for i in (0, 1)]
    x = mxfp4.values(mxfp4.unpack(_np(xc)), _np(xs))
    bound = (d / 32 + 16) * 2.0 ** -23 * (np.abs(x) @ np.abs(w1).T) + 2.0 ** -8 * np.abs(x @ w1.T)
    assert np.all(np.abs(_np(hid) - x @ w1.T) <= bound)
    assert np.all(np.abs(_np(torch.cat(parts, 1)) - x @ w1.T) <= bound)
    act = nvq.swiglu(hid)
    ref = mlp.swiglu(_np(hid))
    assert np.all(np.abs(_np(act) - ref) <= (10 * U + 2.0 ** -8) * np.abs(ref) + 2.0 ** -120)
    Y = nvq.mxfp4_gemm(act, *W2)
    a = mxfp4.values(*mxfp4.quantize(_np(act)))
    assert np.all(np.abs(_np(Y) - a @ w2.T) <= (h / 32 + 16) * 2.0 ** -23 * (np.abs(a) @ np.abs(w2).T) + 1e-37)
    dY = torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    dact = nvq.mxfp4_gemm_dx(dY, *W2, out_dtype=torch.bfloat16)
    dX = nvq.mxfp4_gemm_dx(nvq.swiglu_backward(dact, hid), *W1)
    da = _np(dY) @ w2
    rdh = mlp.swiglu_backward(da, _np(hid))
    gate, up = np.split(np.abs(_np(hid)), 2, axis=1)
    size = np.concatenate((up * (1 + gate), gate), 1) * np.tile(np.abs(_np(dY)) @ np.abs(w2), 2)
    assert np.all(np.abs(_np(dX) - rdh @ w1) <= 4 * 2.0 ** -8 * 1.1 * (size @ np.abs(w1)))
