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
