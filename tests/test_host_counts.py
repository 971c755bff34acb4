"""Counts given as arrays (n_draft, n_new) reach the library as they are, or are refused: no
fraction is cut off, no large value wraps around."""
import ctypes

import numpy as np
import pytest
import torch

from layer_wise_mixed_b200 import kvq


@pytest.mark.parametrize("bad", [[1.7, 2.0], [2 ** 32 + 1, 1], [-2 ** 31 - 1, 1], [True, False]])
def test_arrays_that_int32_does_not_hold(bad):
    with pytest.raises(ValueError):
        kvq._host_i32(np.array(bad))


@pytest.mark.parametrize("bad", [[1.7, 2.0], [2 ** 32 + 1, 1]])
def test_lists_that_int32_does_not_hold(bad):
    with pytest.raises((TypeError, OverflowError)):
        kvq._host_i32(bad)


@pytest.mark.parametrize("make", [list, tuple, np.array, lambda v: np.array(v, np.int64)[::1], torch.tensor,
                                  lambda v: np.array(v, np.uint8)])
def test_counts_arrive(make):
    for v in ([3, 0, 7], [5]):
        at, keep = kvq._host_i32(make(v))
        assert list((ctypes.c_int32 * len(v)).from_address(at)) == v
    assert kvq._host_i32(None) == (None, None)
