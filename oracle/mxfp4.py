"""MXFP4 quantization, plainly in fp64 (oracle; test infrastructure only).

32 consecutive E2M1 elements of a row under one power of two 2^(byte - 127) (byte 255: NaN).
"""

import numpy as np

BLOCK = 32
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def quantize(x):
    """(4-bit codes [n, k], scale bytes [n, k/32]) of x [n, k] (any float type, taken exactly)."""
    x = np.asarray(x, dtype=np.float64)
    n, k = x.shape
    codes = np.zeros((n, k), dtype=np.uint8)
    scales = np.zeros((n, k // BLOCK), dtype=np.uint8)
    for r in range(n):
        for b in range(k // BLOCK):
            v = x[r, b * BLOCK:(b + 1) * BLOCK]
            if not np.all(np.isfinite(v)):
                scales[r, b] = 255
                continue
            top = np.abs(v).max()
            e = -127
            if top > 0:
                e = min(max(int(np.frexp(top)[1]) - 1 - 2, -127), 127)
            scales[r, b] = e + 127
            y = np.ldexp(np.abs(v), -e)
            dist = np.abs(y[:, None] - GRID)
            best = dist.min(1)
            for i in range(BLOCK):
                near = np.flatnonzero(dist[i] == best[i])           # two on a tie: the even code
                idx = int(near[0]) if len(near) == 1 else int(near[near % 2 == 0][0])
                codes[r, b * BLOCK + i] = idx | (8 if np.signbit(v[i]) else 0)
    return codes, scales


def values(codes, scales):
    """The values [n, k] of 4-bit codes [n, k] under scale bytes [n, k/32]."""
    codes = np.asarray(codes)
    v = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]
    s = np.where(np.asarray(scales) == 255, np.nan, np.ldexp(1.0, np.asarray(scales, dtype=np.int64) - 127))
    return v * np.repeat(s, BLOCK, axis=1)


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty((packed.shape[0], 2 * packed.shape[1]), dtype=np.uint8)
    out[:, 0::2] = packed & 15
    out[:, 1::2] = packed >> 4
    return out
