"""Pins of the mixture-of-experts oracle where two of its rules meet."""

import numpy as np

from oracle import moe


def test_a_row_without_a_token_is_zeros_whatever_its_expert_holds():
    W = np.ones((2, 3, 4))
    W[0, 1] = np.nan                    # a rejected weight row
    W[1, 2] = np.inf
    X = np.ones((2, 4))
    Y = moe.grouped_matmul(X, W, [0, 3, 5], [0, -1, 2, 1, 7])
    assert np.array_equal(Y[[1, 2, 4]], np.zeros((3, 3)))
    assert np.isnan(Y[0, 1]) and Y[0, 0] == Y[0, 2] == 4 and Y[3].tolist() == [4, 4, np.inf]
