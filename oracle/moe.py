"""Mixture-of-experts path around the quantized experts (oracle; test infrastructure only).

Source: the layer's definition.  A router scores E experts per token, the
top_k largest are chosen and weighted by a softmax, each expert multiplies its
tokens with its own NVFP4 weights, and a token's result is the weighted sum of
its experts' rows.  Everything is NumPy in fp64, one formula per function.
"""

import numpy as np

from . import codec


def topk(logits, top_k, renorm):
    """(ids [T, K], weights [T, K]): largest logits first, ties to the lower index; -inf is never chosen (id -1, weight 0);
    a row with a NaN or +inf has ids -1 and NaN weights.  Softmax over the chosen logits (renorm) or over all."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    ids = np.full((T, top_k), -1, dtype=np.int32)
    weights = np.zeros((T, top_k))
    for t in range(T):
        row = logits[t]
        if not np.all(row < np.inf):
            weights[t] = np.nan
            continue
        order = sorted((e for e in range(E) if row[e] > -np.inf), key=lambda e: (-row[e], e))[:top_k]
        if not order:
            continue
        ex = np.exp(row - row[order[0]])
        total = ex[order].sum() if renorm else ex.sum()
        ids[t, :len(order)] = order
        weights[t, :len(order)] = ex[order] / total
    return ids, weights


def topk_backward(logits, ids, weights, dweights, renorm):
    """Gradient of the weights with respect to the logits: the softmax's, d l_j = p_j (d_j - sum_s dw_s w_s)."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        if np.any(np.isnan(weights[t])):
            out[t] = np.nan
            continue
        s = np.flatnonzero(ids[t] >= 0)
        if len(s) == 0:
            continue
        e = ids[t][s]
        dw = np.asarray(dweights[t], dtype=np.float64)[s]
        w = np.asarray(weights[t], dtype=np.float64)[s]
        c = float(np.dot(dw, w))
        if renorm:
            np.add.at(out[t], e, w * (dw - c))
        else:
            d = np.zeros(E)
            np.add.at(d, e, dw)
            ex = np.exp(logits[t] - logits[t].max())
            out[t] = ex / ex.sum() * (d - c)
    return out


def sort(ids, n_experts):
    """(tok_idx [T*K], grp_off [E+1], pos [T, K]): slots by expert, token, slot; ids outside [0, E) have no row."""
    ids = np.asarray(ids)
    T, K = ids.shape
    rows = sorted((int(ids[t, s]), t, s) for t in range(T) for s in range(K) if 0 <= ids[t, s] < n_experts)
    tok_idx = np.full(T * K, -1, dtype=np.int32)
    pos = np.full((T, K), -1, dtype=np.int32)
    off = np.zeros(n_experts + 1, dtype=np.int64)
    for r, (e, t, s) in enumerate(rows):
        tok_idx[r] = t
        pos[t, s] = r
        off[e + 1:] += 1
    return tok_idx, off, pos


def experts_matrices(packed, scales, g):
    """Dequantized experts [G, m, k] in fp64 (the exact products)."""
    return np.stack([codec.dequant_exact(codec.unpack_codes(packed[e]), np.repeat(scales[e], 16, axis=1), np.float32(g[e]))
                     for e in range(len(packed))])


def grouped_matmul(X, W, grp_off, tok_idx=None):
    """Rows r of expert e: X[tok_idx[r]] W_e^T (a token outside X: zeros, whatever the weights).  Rows no expert has stay 0."""
    X = np.asarray(X, dtype=np.float64)
    rows = len(X) if tok_idx is None else len(tok_idx)
    Y = np.zeros((rows, W.shape[1]))
    for e in range(len(W)):
        for r in range(int(grp_off[e]), int(grp_off[e + 1])):
            t = r if tok_idx is None else int(tok_idx[r])
            if 0 <= t < len(X):
                Y[r] = W[e] @ X[t]
    return Y


def grouped_matmul_dx(dY, W, grp_off):
    """Gradient of grouped_matmul with respect to the gathered rows: dY_r W_e."""
    dY = np.asarray(dY, dtype=np.float64)
    dX = np.zeros((len(dY), W.shape[2]))
    for e in range(len(W)):
        r = slice(int(grp_off[e]), int(grp_off[e + 1]))
        dX[r] = dY[r] @ W[e]
    return dX


def combine(Y, pos, weights=None):
    """out[t] = sum_s weights[t, s] Y[pos[t, s]]; a position outside Y counts as zeros."""
    Y = np.asarray(Y, dtype=np.float64)
    T, K = pos.shape
    out = np.zeros((T, Y.shape[1]))
    for t in range(T):
        for s in range(K):
            row = Y[pos[t, s]] if 0 <= pos[t, s] < len(Y) else np.zeros(Y.shape[1])
            out[t] = out[t] + (1.0 if weights is None else float(weights[t, s])) * row
    return out


def combine_backward(dout, Y, pos, weights=None):
    """(dY, dweights) of combine; rows of dY that no position names stay 0."""
    dout, Y = np.asarray(dout, dtype=np.float64), np.asarray(Y, dtype=np.float64)
    T, K = pos.shape
    dY, dw = np.zeros_like(Y), np.zeros((T, K))
    for t in range(T):
        for s in range(K):
            p = pos[t, s]
            if 0 <= p < len(Y):
                dY[p] = (1.0 if weights is None else float(weights[t, s])) * dout[t]
                dw[t, s] = dout[t] @ Y[p]
    return dY, dw
