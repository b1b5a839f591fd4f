"""The table of turns for positions on several axes from numpy arrays, whose integers are not Python's (CPU)."""
import numpy as np
import pytest
import torch

from tests.test_abi_rope import binding, clib  # noqa: F401

FREQ = 10000.0 ** (-np.arange(0, 64, 2) / 64)


@pytest.mark.parametrize("dtype", [np.int64, np.int32, np.uint8])
def test_axes_as_an_array(binding, dtype):  # noqa: F811
    axis = [0] * 8 + [1] * 12 + [2] * 12
    got = binding.rope_turns_axes(FREQ, np.array(axis, dtype=dtype))
    assert got.shape == (3, 32) and torch.equal(got, binding.rope_turns_axes(FREQ.tolist(), axis))


@pytest.mark.parametrize("axis", [np.full(32, 4), np.full(32, -1), np.zeros(32), np.zeros(32, dtype=bool), np.zeros(31, dtype=int)])
def test_arrays_that_name_no_axis(binding, axis):  # noqa: F811
    with pytest.raises(ValueError):
        binding.rope_turns_axes(FREQ, axis)
