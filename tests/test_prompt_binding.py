"""The binding of the operators of a layer over packed prompts, without a GPU."""
import numpy as np
import pytest
import torch

import packed_varlen_gb300 as pv


def _widths(values):
    arr, n, at = pv._host_ints(values)
    assert len(arr) == n and at
    return list(arr)


def test_axis_widths_are_whole_numbers_whatever_was_asked_before():
    assert _widths([16, 56, 56]) == [16, 56, 56]
    assert _widths(np.array([16, 56, 56])) == [16, 56, 56]
    for floats in ([16.0, 56.0, 56.0], (16, 56.0, 56), np.array([16.0, 56.0, 56.0])):
        with pytest.raises(TypeError):
            pv._host_ints(floats)


def test_axis_widths_are_those_of_the_call():
    """Tensors that stand for numbers, changed between two calls."""
    dims = [torch.tensor(24), torch.tensor(40)]
    assert _widths(dims) == [24, 40]
    dims[0].fill_(40)
    dims[1].fill_(24)
    assert _widths(dims) == [40, 24]
    both = torch.tensor([8, 56])
    assert _widths(both) == [8, 56]
    both += 2
    assert _widths(both) == [10, 58]
