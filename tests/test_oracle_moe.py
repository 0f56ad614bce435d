"""Pins of the mixture-of-experts oracle: closed forms, invariances and gradients against differences."""

import numpy as np
import pytest

from oracle import moe


def _layer(rng, T, E, K, m, k):
    X = rng.standard_normal((T, k))
    W = rng.standard_normal((E, m, k))
    return X, W, rng.standard_normal((T, E))


def _forward(X, W, logits, K, renorm):
    ids, w = moe.topk(logits, K, renorm)
    tok, off, pos = moe.sort(ids, len(W))
    Y = moe.grouped_matmul(X, W, off, tok)
    return moe.combine(Y, pos, w), (ids, w, tok, off, pos, Y)


@pytest.mark.parametrize("renorm", [True, False])
def test_layer_equals_dense_sum_over_chosen_experts(renorm):
    rng = np.random.default_rng(1)
    T, E, K, m, k = 9, 7, 3, 5, 6
    X, W, logits = _layer(rng, T, E, K, m, k)
    out, (ids, w, *_) = _forward(X, W, logits, K, renorm)
    for t in range(T):
        chosen = np.argsort(-logits[t])[:K]
        assert list(ids[t]) == list(chosen)
        p = np.exp(logits[t])
        q = p[chosen] / (p[chosen].sum() if renorm else p.sum())
        assert np.allclose(out[t], sum(q[i] * (W[e] @ X[t]) for i, e in enumerate(chosen)), rtol=1e-12)


def test_ties_masks_and_rejected_rows():
    inf, nan = np.inf, np.nan
    ids, w = moe.topk([[1, 2, 2, 0], [-inf, 3, -inf, -inf], [-inf] * 4, [0, nan, 0, 0], [0, inf, 0, 0]], 2, True)
    assert ids.tolist() == [[1, 2], [1, -1], [-1, -1], [-1, -1], [-1, -1]]
    assert w[0].tolist() == [0.5, 0.5] and w[1].tolist() == [1, 0] and w[2].tolist() == [0, 0]
    assert np.isnan(w[3:]).all()
    tok, off, pos = moe.sort([[2, -1], [0, 2], [5, 2]], 3)
    assert off.tolist() == [0, 1, 1, 4]
    assert tok.tolist() == [1, 0, 1, 2, -1, -1]
    assert pos.tolist() == [[1, -1], [0, 2], [-1, 3]]


@pytest.mark.parametrize("renorm", [True, False])
def test_gradients_against_differences(renorm):
    rng = np.random.default_rng(2)
    T, E, K, m, k = 4, 5, 2, 3, 4
    X, W, logits = _layer(rng, T, E, K, m, k)
    G = rng.standard_normal((T, m))
    out, (ids, w, tok, off, pos, Y) = _forward(X, W, logits, K, renorm)
    dY, dw = moe.combine_backward(G, Y, pos, w)
    dl = moe.topk_backward(logits, ids, w, dw, renorm)
    dX = moe.combine(moe.grouped_matmul_dx(dY, W, off), pos)
    h = 1e-6
    for A, d in ((logits, dl), (X, dX)):
        for i in np.ndindex(A.shape):
            keep = A[i]
            A[i] = keep + h
            up = (_forward(X, W, logits, K, renorm)[0] * G).sum()
            A[i] = keep - h
            down = (_forward(X, W, logits, K, renorm)[0] * G).sum()
            A[i] = keep
            assert abs((up - down) / (2 * h) - d[i]) < 1e-6 * (1 + abs(d[i]))


def test_router_gradient_of_an_expert_named_twice():
    """Slots of one expert add up: the gradient of sum_s dw_s softmax(l[ids])_s, by differences."""
    rng = np.random.default_rng(11)
    l, ids, dw = rng.standard_normal((1, 6)), np.array([[2, 4, 2, 2]], dtype=np.int32), rng.standard_normal((1, 4))

    def weights(x, renorm):
        over = x[0, ids[0]] if renorm else x[0]
        return np.exp(x[0, ids[0]])[None] / np.exp(over).sum()

    for renorm in (True, False):
        got = moe.topk_backward(l, ids, weights(l, renorm), dw, renorm)
        for j in range(6):
            h = np.zeros((1, 6))
            h[0, j] = 1e-5
            d = (dw * (weights(l + h, renorm) - weights(l - h, renorm))).sum() / 2e-5
            assert abs(d - got[0, j]) < 1e-8
