"""Forms of the mixture-of-experts gradients that the layer's own chain does not take: either gradient of the weighted sum
alone, the router's gradient between wider buffers.  Bounds: a sum of n fp32 products in any order is within n u sum |terms|,
u = 2^-24; a bf16 result within 2^-8 of itself."""

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


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _np(t):
    return t.double().cpu().numpy() if t.dtype.is_floating_point else t.cpu().numpy()


@pytest.mark.parametrize("yt", DTYPES)
@pytest.mark.parametrize("T,K,d", [(1, 8, 4096), (37, 3, 7), (100, 6, 520), (20, 11, 2056), (600, 2, 136)])
@pytest.mark.parametrize("weighted", [True, False])
def test_either_gradient_of_the_weighted_sum_alone(nvq, T, K, d, yt, weighted):
    """As both together give it, bit for bit; without dweights Y is not read, and without dY nothing but dweights is written."""
    rng = np.random.default_rng([T, K, d])
    rows = T * K - K // 2
    pos = rng.permutation(T * K).reshape(T, K).astype(np.int32)      # those >= rows name no row
    pos[rng.random((T, K)) < 0.2] = -1
    pos = _dev(pos)
    Y = _dev(rng.standard_normal((rows, d)).astype(np.float32)).to(DTYPES[yt])
    dout = _dev(rng.standard_normal((T, d)).astype(np.float32))
    w = _dev(rng.standard_normal((T, K)).astype(np.float32)) if weighted else None
    dY, dw = nvq.moe_combine_backward(dout, Y, pos, w, dY=torch.full_like(Y, 7.0))
    # the library's own call, with NULL for what is left out
    code = nvq.NVQ_DTYPE_BF16 if yt == "bf16" else nvq.NVQ_DTYPE_F32
    stream = torch.cuda.current_stream().cuda_stream
    wp = w.data_ptr() if weighted else None
    one = torch.full_like(Y, 7.0)
    assert nvq.lib.moe_combine_backward(dout.data_ptr(), nvq.NVQ_DTYPE_F32, T, d, d, None, code, rows, 0, pos.data_ptr(), wp, K,
                                        one.data_ptr(), d, None, stream) == 0
    assert torch.equal(one, dY)
    two = torch.full_like(dw, 7.0)
    assert nvq.lib.moe_combine_backward(dout.data_ptr(), nvq.NVQ_DTYPE_F32, T, d, d, Y.data_ptr(), code, rows, d, pos.data_ptr(), wp,
                                        K, None, 0, two.data_ptr(), stream) == 0
    assert torch.equal(two, dw)
    # and the Python function
    nans = torch.full_like(Y, float("nan"))
    got = nvq.moe_combine_backward(dout, nans, pos, w, dY=torch.full_like(Y, 7.0), need_dweights=False)
    assert got[1] is None and torch.equal(got[0], dY)
    got = nvq.moe_combine_backward(dout, None, pos, w, dY=torch.full_like(Y, 7.0), need_dweights=False)
    assert got[1] is None and torch.equal(got[0], dY)
    got = nvq.moe_combine_backward(dout, Y, pos, w, need_dY=False)
    assert got[0] is None and torch.equal(got[1], dw)
    # both against the oracle
    rdY, rdw = moe.combine_backward(_np(dout), _np(Y), _np(pos), None if w is None else _np(w))
    amag = moe.combine_backward(np.abs(_np(dout)), np.abs(_np(Y)), _np(pos), None)[1]
    named = np.zeros(rows, dtype=bool)
    p = _np(pos)
    named[p[(p >= 0) & (p < rows)]] = True
    half = 2.0 ** -8 if yt == "bf16" else 0.0
    assert np.all(np.abs(_np(one) - rdY)[named] <= (np.abs(rdY) * (U + half))[named] + 1e-37) and (_np(one)[~named] == 7).all()
    assert np.all(np.abs(_np(two) - rdw) <= d * U * amag + 1e-37)


def test_gradients_of_the_weighted_sum_refused(nvq):
    f = torch.zeros(4, 32, device=DEV)
    pos = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    for kind, call in [(nvq.NvqError, lambda: nvq.moe_combine_backward(f, f, pos, need_dY=False, need_dweights=False)),
                       (ValueError, lambda: nvq.moe_combine_backward(f, None, pos)),
                       (ValueError, lambda: nvq.moe_combine_backward(f, None, pos, need_dweights=False)),
                       (ValueError, lambda: nvq.moe_combine_backward(f, None, pos, dY=torch.zeros_like(f))),
                       (ValueError, lambda: nvq.moe_combine_backward(f, f, pos, dY=torch.zeros_like(f), need_dY=False))]:
        with pytest.raises(kind):
            call()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K", [(5, 7, 3), (4100, 100, 8), (33, 300, 20), (5000, 256, 6)])
def test_router_gradient_between_wider_buffers(nvq, T, E, K, dtype, renorm):
    """Logits and their gradient as column slices at any element's place: what contiguous ones give, and no other column."""
    rng = np.random.default_rng([T, E, K])
    dtype = DTYPES[dtype]
    wide = _dev(rng.standard_normal((T, E + 10)).astype(np.float32)).to(dtype)
    dw = _dev(rng.standard_normal((T, K)).astype(np.float32))
    for at, left in ((3, 1), (8, 5)):
        logits = wide[:, at:at + E]
        ids, w = nvq.moe_topk(logits, K, renorm)
        ref = nvq.moe_topk_backward(logits.contiguous(), ids, w, dw, renorm)
        assert torch.equal(nvq.moe_topk_backward(logits, ids, w, dw, renorm), ref)
        out = torch.full((T, E + left + 4), 7.0, dtype=dtype, device=DEV)
        code = nvq.NVQ_DTYPE_BF16 if dtype == torch.bfloat16 else nvq.NVQ_DTYPE_F32
        assert nvq.lib.moe_topk_backward(logits.data_ptr(), code, T, E, logits.stride(0), ids.data_ptr(), w.data_ptr(), dw.data_ptr(), K,
                                         int(renorm), out[:, left:].data_ptr(), out.stride(0),
                                         torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(out[:, left:left + E], ref)
        assert (out[:, :left] == 7).all() and (out[:, left + E:] == 7).all()


def test_the_chain_in_bf16(nvq):
    """Products in bf16 hand moe_combine_backward a Y whose gradient nvfp4_gemm_grouped_dx takes as it is."""
    rng = np.random.default_rng(21)
    T, E, K, m, k = 50, 6, 2, 48, 64
    codes = _dev(rng.integers(0, 256, (E, m, k // 2), dtype=np.uint8))
    scales = _dev(rng.integers(0x20, 0x7F, (E, m, k // 16), dtype=np.uint8))
    g = _dev((rng.random(E) * 1e-3 + 1e-3).astype(np.float32))
    X = _dev(rng.standard_normal((T, k)).astype(np.float32)).to(torch.bfloat16)
    logits = _dev(rng.standard_normal((T, E)).astype(np.float32))
    ids, w = nvq.moe_topk(logits, K)
    tok, off, pos = nvq.moe_sort(ids, E)
    Y = nvq.nvfp4_gemm_grouped(X, codes, scales, g, off, tok, out_dtype=torch.bfloat16)
    out = nvq.moe_combine(Y, pos, w)
    dout = torch.randn(T, m, device=DEV).to(torch.bfloat16)
    dY, dw = nvq.moe_combine_backward(dout, Y, pos, w)
    dX = nvq.moe_combine(nvq.nvfp4_gemm_grouped_dx(dY, codes, scales, g, off), pos)
    assert out.dtype == dY.dtype == torch.bfloat16 and dX.shape == X.shape
    W = moe.experts_matrices(codes.cpu().numpy(), scales.cpu().numpy(), _np(g))
    ref = moe.combine(moe.grouped_matmul_dx(_np(dY), W, _np(off)), _np(pos))
    mag = moe.combine(moe.grouped_matmul_dx(np.abs(_np(dY)), np.abs(W), _np(off)), _np(pos))
    assert np.all(np.abs(_np(dX) - ref) <= mag * ((m / 16 + 16) * 2.0 ** -23 + K * U) + 1e-30)


@pytest.mark.parametrize("T", [2, 65])
def test_weighted_sum_of_rows_of_2_28_columns(nvq, T):
    """Where one launch holds fewer than 64 tokens, 65 take two.  Small whole numbers: every product and sum is exact."""
    d = 2 ** 28 + 5
    y = (torch.arange(d, device=DEV, dtype=torch.int32) % 7 - 3).float()[None]
    pos = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    w = (torch.arange(T, device=DEV) % 5 - 2).float()[:, None]
    out = nvq.moe_combine(y, pos, w, out_dtype=torch.bfloat16)
    for t in range(T):
        assert torch.equal(out[t], (y[0] * float(t % 5 - 2)).to(torch.bfloat16))
