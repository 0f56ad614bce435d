"""The MXFP4, gated-activation and mixture-of-experts MLP oracles against independent forms."""

import numpy as np
import pytest
import torch

from oracle import mlp, mxfp4


def test_grid_is_e2m1():
    vals = [(m * 0.5 if e == 0 else 2.0 ** (e - 1) * (1 + m / 2)) for e in range(4) for m in range(2)]
    assert np.array_equal(vals, mxfp4.GRID)


def test_quantize_known_block():
    x = np.zeros((1, 32))
    x[0, :10] = [7.9, -6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.2]      # largest in [4, 8): scale 1, ties to even
    codes, scales = mxfp4.quantize(x)
    assert scales[0, 0] == 127
    assert np.array_equal(mxfp4.values(codes, scales)[0, :10], [6, -6, 4, 4, 2, 2, 1, 1, 0, 0])


@pytest.mark.parametrize("e", [-149, -130, -126, -100, 0, 100, 127])
def test_quantize_scale_range(e):
    x = np.zeros((1, 32))
    x[0, 3] = np.ldexp(1.0, e)
    codes, scales = mxfp4.quantize(x)
    assert scales[0, 0] == max(e - 2, -127) + 127
    v = mxfp4.values(codes, scales)[0, 3]
    assert v == (x[0, 3] if e >= -128 else 0.0)      # half of 2^-127 is the smallest value


def test_quantize_is_nearest_and_idempotent():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 96)) * np.exp(rng.standard_normal((5, 96)))
    codes, scales = mxfp4.quantize(x)
    v = mxfp4.values(codes, scales)
    step = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=1)
    assert np.all(np.abs(v - x) <= np.where(np.abs(x) <= 6 * step, step, 2 * step))
    c2, s2 = mxfp4.quantize(v)
    assert np.array_equal(mxfp4.values(c2, s2), v)
    assert np.array_equal(mxfp4.unpack(mxfp4.pack(codes)), codes)


def test_quantize_non_finite_block():
    x = np.ones((1, 64))
    x[0, 40] = np.inf
    codes, scales = mxfp4.quantize(x)
    assert list(scales[0]) == [125, 255] and not codes[0, 32:].any()
    assert np.isnan(mxfp4.values(codes, scales)[0, 32:]).all()


def test_swiglu_and_gradient_against_autograd():
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((7, 10)) * 4).requires_grad_()
    d = torch.from_numpy(rng.standard_normal((7, 5)))
    y = torch.nn.functional.silu(x[:, :5]) * x[:, 5:]
    y.backward(d)
    assert np.allclose(mlp.swiglu(x.detach().numpy()), y.detach().numpy(), rtol=1e-14, atol=0)
    assert np.allclose(mlp.swiglu_backward(d.numpy(), x.detach().numpy()), x.grad.numpy(), rtol=1e-13, atol=1e-16)


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(2)
    x, d, eps = rng.standard_normal((3, 8)) * 3, rng.standard_normal((3, 4)), 1e-5
    g = mlp.swiglu_backward(d, x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        assert abs(((mlp.swiglu(a) - mlp.swiglu(b)) * d).sum() / (2 * eps) - g[i]) < 1e-8


def test_moe_mlp_is_the_sum_over_experts():
    rng = np.random.default_rng(3)
    E, d, h, m, T = 3, 6, 4, 5, 4
    gu, dn = rng.standard_normal((E, 2 * h, d)), rng.standard_normal((E, m, h))
    X = rng.standard_normal((T, d))
    ids, w = np.array([[0, 1], [2, -1], [1, 1], [-1, 3]]), rng.random((T, 2))
    out = mlp.moe_mlp(X, gu, dn, ids, w)
    for e in range(E):                                                # each expert alone, by its tokens' total weight
        share = (w * (ids == e)).sum(1)
        out -= share[:, None] * (mlp.swiglu(X @ gu[e].T) @ dn[e].T)
    assert np.abs(out).max() < 1e-12
