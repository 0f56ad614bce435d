"""GPU parity of the gated activation and its gradient against the fp64 oracle.

Errors with u = 2^-24: z = exp(-|g|) within 2 u; 1 + z, 1 / (1 + z) and their product one u (three for the quotient) each, so
s and 1 - s within 8 u; two products more for the forward pass: 10 u |out|.  The gradient's 1 + g (1 - s) may cancel: its
error is below (8 u + 2 u) (1 + |g (1 - s)|), so dgate is within 20 u |dout up s| (1 + |g (1 - s)|); dup as the forward pass.
Below fp32's normal range (2^-126) an absolute 2^-126 is allowed times the other factors.  bf16 results add 2^-8.
"""

import numpy as np
import pytest
import torch

from oracle import mlp

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
    return t.double().cpu().numpy()


def _half(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


SHAPES = [(1, 1, 0), (1, 8, 0), (3, 7, 1), (5, 9, 2), (64, 16, 0), (33, 100, 4), (2, 2060, 0), (17, 1027, 3), (300, 64, 8), (9, 5000, 0)]


@pytest.mark.parametrize("xtype", ["f32", "bf16"])
@pytest.mark.parametrize("otype", ["f32", "bf16"])
@pytest.mark.parametrize("n,h,gap", SHAPES)
def test_swiglu(nvq, n, h, gap, xtype, otype):
    rng = np.random.default_rng([n, h])
    X = torch.from_numpy((rng.standard_normal((n, 2 * h + gap)) * 6).astype(np.float32)).to(DTYPES[xtype]).to(DEV)[:, gap // 2:gap // 2 + 2 * h]
    dt = DTYPES[otype]
    out = nvq.swiglu(X, out_dtype=dt)
    ref = mlp.swiglu(_np(X))
    assert np.all(np.abs(_np(out) - ref) <= (10 * U + _half(dt)) * np.abs(ref) + 2.0 ** -120)
    buf = torch.full((n + 1, h + 5), 3.0, dtype=dt, device=DEV)
    nvq.swiglu(X, out=buf[:n, 2:2 + h])
    assert torch.equal(buf[:n, 2:2 + h], out)
    buf[:n, 2:2 + h] = 3.0
    assert bool((buf == 3.0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,h,gap", SHAPES)
def test_swiglu_backward(nvq, n, h, gap, dtype):
    rng = np.random.default_rng([n, h, 1])
    dt = DTYPES[dtype]
    X = torch.from_numpy((rng.standard_normal((n, 2 * h + gap)) * 4).astype(np.float32)).to(dt).to(DEV)[:, gap // 2:gap // 2 + 2 * h]
    d = torch.from_numpy(rng.standard_normal((n, h + gap)).astype(np.float32)).to(dt).to(DEV)[:, :h]
    dX = nvq.swiglu_backward(d, X)
    x, dd = _np(X), _np(d)
    ref = mlp.swiglu_backward(dd, x)
    g, up = np.split(x, 2, axis=1)
    s, rest = mlp.sigmoid(g), mlp.sigmoid(-g)
    mag = np.concatenate((20 * U * np.abs(dd * up * s) * (1 + np.abs(g * rest)), 10 * U * np.abs(ref[:, h:])), axis=1)
    assert np.all(np.abs(_np(dX) - ref) <= mag + _half(dt) * np.abs(ref) + 2.0 ** -120)
    buf = torch.full((n + 1, 2 * h + 3), 3.0, dtype=dt, device=DEV)
    nvq.swiglu_backward(d, X, dX=buf[:n, 1:1 + 2 * h])
    assert torch.equal(buf[:n, 1:1 + 2 * h], dX)
    buf[:n, 1:1 + 2 * h] = 3.0
    assert bool((buf == 3.0).all())


def test_swiglu_large_gates(nvq):
    """Gates far on either side: no overflow, nothing but the formula's own limits."""
    g = torch.tensor([-1e30, -200.0, -90.0, -88.0, -30.0, 0.0, -0.0, 30.0, 88.0, 200.0, 1e30, float("inf"), float("nan")])
    X = torch.stack((g, torch.full_like(g, 2.0)), 1).reshape(-1, 2).to(DEV)
    out = _np(nvq.swiglu(X))[:, 0]
    with np.errstate(invalid="ignore"):
        ref = mlp.swiglu(_np(X))[:, 0]
    assert np.isnan(out[-1]) and np.isposinf(out[-2])
    assert np.all(np.abs(out[:-2] - ref[:-2]) <= 11 * U * np.abs(ref[:-2]) + 2.0 ** -120)
    dX = _np(nvq.swiglu_backward(torch.ones(len(g), 1, device=DEV), X))
    ref = mlp.swiglu_backward(np.ones((11, 1)), _np(X)[:11])
    assert np.all(np.abs(dX[:11] - ref) <= 40 * U * np.maximum(np.abs(ref), 1e-3) + 2.0 ** -120)
    assert np.isnan(dX[-1]).all()


def test_swiglu_backward_against_differences(nvq):
    rng = np.random.default_rng(9)
    X = torch.from_numpy((rng.standard_normal((4, 12)) * 2).astype(np.float32)).to(DEV)
    d = torch.from_numpy(rng.standard_normal((4, 6)).astype(np.float32)).to(DEV)
    g, eps = _np(nvq.swiglu_backward(d, X)), 2.0 ** -6
    for i in ((0, 0), (1, 5), (2, 6), (3, 11)):
        a, b = X.clone(), X.clone()
        a[i] += eps
        b[i] -= eps
        diff = ((_np(nvq.swiglu(a)) - _np(nvq.swiglu(b))) * _np(d)).sum() / float(a[i] - b[i])
        # third derivative of silu(x) u below 1 |u| (eps^2 / 6 of it), and the outputs' rounding over 2 eps
        assert abs(diff - g[i]) <= 8 * eps ** 2 + 1e-4


def test_swiglu_empty(nvq):
    assert nvq.swiglu(torch.zeros(0, 8, device=DEV)).shape == (0, 4)
    assert nvq.swiglu_backward(torch.zeros(0, 4, device=DEV), torch.zeros(0, 8, device=DEV)).shape == (0, 8)
