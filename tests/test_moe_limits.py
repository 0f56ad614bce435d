"""The mixture-of-experts calls refuse sizes past what one launch holds on the host, before any GPU work."""

import ctypes

import pytest

P = ctypes.c_void_p
SHAPE = -2
a, b, c = P(4096), P(8192), P(12288)   # never dereferenced


@pytest.fixture(scope="module")
def nvq():
    import post_nvfp4_weight_amd as m
    return m


def test_combine_columns(nvq):
    d = (1 << 33) + 1
    assert nvq.lib.moe_combine(a, 0, 8, d, d, b, b, 4, 2, c, 0, d, None) == SHAPE


@pytest.mark.parametrize("rows,G,wide", [((1 << 31) - 1, 4, 4000000), ((1 << 31) - 1, 1, 16), (1 << 22, 1 << 22, 1040)])
def test_products_of_too_many_tiles(nvq, rows, G, wide):
    assert nvq.lib.nvfp4_gemm_grouped(a, 1, 10, 32, 32, b, rows, b, G, b, b, b, wide, c, 1, wide, None) == SHAPE
    assert b"tiles" in nvq.lib.nvq_last_error()
    assert nvq.lib.nvfp4_gemm_grouped_dx(a, 1, rows, 16, 16, b, G, b, b, b, wide, c, 1, wide, None) == SHAPE
    assert b"tiles" in nvq.lib.nvq_last_error()
