"""The gated activation of an MLP, its gradient, and a whole mixture-of-experts MLP, plainly in fp64 (oracle; test
infrastructure only)."""

import numpy as np


def sigmoid(x):
    x = np.asarray(x, dtype=np.float64)
    z = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, z) / (1.0 + z)


def swiglu(x):
    x = np.asarray(x, dtype=np.float64)
    g, u = np.split(x, 2, axis=1)
    return g * sigmoid(g) * u


def swiglu_backward(dout, x):
    x = np.asarray(x, dtype=np.float64)
    g, u = np.split(x, 2, axis=1)
    s, rest = sigmoid(g), sigmoid(-g)
    d = np.asarray(dout, dtype=np.float64)
    return np.concatenate((d * u * s * (1 + g * rest), d * g * s), axis=1)


def moe_mlp(X, gate_up, down, ids, weights):
    """out[t] = sum_s weights[t, s] D_e (silu(G_e x_t) * (U_e x_t)), e = ids[t, s]; gate_up [E, 2h, d] holds G then U, down
    [E, m, h].  A slot whose id is outside [0, E) counts as zeros under its weight."""
    X = np.asarray(X, dtype=np.float64)
    out = np.zeros((X.shape[0], down.shape[1]))
    for t in range(X.shape[0]):
        for e, w in zip(ids[t], weights[t]):
            y = np.zeros(down.shape[1])
            if 0 <= e < down.shape[0]:
                y = down[e] @ swiglu((gate_up[e] @ X[t])[None])[0]
            out[t] += w * y
    return out
