"""The activation between the two products of the few-token expert MLP keeps fp32's bits where the result is fp32.

Every sum has one term: a token has one input, a row of the second layer one weight, each global scale is a power of two and
there is one expert per token.  So with u = 2^-24, gate and up are exact; silu is within 10 u, times up and the weight 2 u
more.  The activation's three parts add nothing; their products are exact, and an instruction that adds one has at most two roundings of
2^-23 = 2 u each, 12 u; the rest of the sums are zeros.  32 u cover it with the bound's own roundings.  A bf16 result keeps
two parts: the first leaves up to 2^-8 of the value, of which the second's half step is up to 2^-17, 128 u; then 32 u + 2^-8.
"""

import numpy as np
import pytest
import torch

from oracle import codec, mlp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


@pytest.fixture(scope="module")
def nvq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import post_nvfp4_weight_amd as m
    return m


def _layer(codes, scales, g):
    """(device tensors, values in fp64) of codes [E, m, k], scales [E, m, k / 16], g [E]."""
    packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
    s = np.array([codec.e4m3_decode(b) for b in range(0x7F)])[scales]
    w = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7] * np.repeat(s, 16, axis=2) * g.astype(np.float64)[:, None, None]
    return tuple(torch.from_numpy(a).to(DEV) for a in (packed, scales, g)), w


# tokens and experts: entries of 4 tokens and of 8;  h: whole chunks, and one that ends inside (in the middle of a piece too)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E", [(1, 3), (11, 4), (64, 4), (64, 40)])
@pytest.mark.parametrize("d,h", [(512, 512), (96, 560), (1024, 1056)])
def test_single_terms(nvq, d, h, T, E, dtype):
    rng = np.random.default_rng(T * h + E)
    gu, wgu = _layer(rng.integers(1, 16, (E, 2 * h, d), dtype=np.uint8), rng.integers(0x30, 0x40, (E, 2 * h, d // 16), dtype=np.uint8),
                     2.0 ** rng.integers(-3, 1, E).astype(np.float32))
    codes = np.zeros((E, h, h), dtype=np.uint8)
    codes[:, np.arange(h), np.arange(h)[::-1]] = rng.choice([1, 2, 3, 4, 5, 6, 7, 9, 13, 15], (E, h)).astype(np.uint8)
    dn, wdn = _layer(codes, rng.integers(0x20, 0x60, (E, h, h // 16), dtype=np.uint8), 2.0 ** rng.integers(-3, 3, E).astype(np.float32))
    X = torch.zeros(T, d, dtype=torch.bfloat16)
    X[torch.arange(T), torch.from_numpy(rng.integers(0, d, T))] = torch.from_numpy(rng.standard_normal(T).astype(np.float32)).to(torch.bfloat16)
    ids = rng.integers(0, E, (T, 1)).astype(np.int32)
    w = (rng.random((T, 1)) + 0.01).astype(np.float32)
    out, _, _ = nvq.nvfp4_moe_mlp(X.to(DEV), gu, dn, ids=torch.from_numpy(ids).to(DEV), weights=torch.from_numpy(w).to(DEV), out_dtype=dtype)
    ref = mlp.moe_mlp(X.double().numpy(), wgu, wdn, ids, w.astype(np.float64))
    off = np.abs(out.double().cpu().numpy() - ref) / np.maximum(np.abs(ref), 1e-30)
    bound = 32 * U if dtype == torch.float32 else 160 * U + 2.0 ** -8
    assert off.max() <= bound, (off.max() / U, np.unravel_index(off.argmax(), off.shape))
