"""The plans of cross attention (CPU: host arithmetic for GPUs of 148 and 152 SMs): the sizes by which GPU tests mean a
form take it, the limits of the forms without tiles, shares that hold keys, and sizes that the calls refuse."""
import pytest

from tests import test_gpu_cross_by_tiles as by_tiles
from tests.test_abi_rope import binding, clib  # noqa: F401

SMS = (148, 152)


@pytest.mark.parametrize("sms", SMS)
def test_sizes_by_which_tests_mean_a_form(binding, sms):  # noqa: F811
    for size, want, ragged in by_tiles.PLANNED:
        form, shares = binding.testing_cross_plan(*size, ragged, sms)
        assert form == want[0], (size, ragged, form, shares)
        assert shares == want[1] if len(want) > 1 and want[1] else shares > 1, (size, ragged, shares)


@pytest.mark.parametrize("sms", SMS)
def test_limits_of_the_forms_without_tiles(binding, sms):  # noqa: F811
    for B, H, Sk in ((1, 1, 1), (64, 32, 1500), (1, 16, 32768), (200, 128, 77)):
        for ragged in (False, True):
            assert all(binding.testing_cross_plan(B, H, Sq, Sk, ragged, sms)[0] == 0 for Sq in (1, 2, 8))
    assert binding.testing_cross_plan(64, 32, 9, 1500, False, sms)[0] == by_tiles.ONE
    assert binding.testing_cross_plan(2, 64, 4096, 6404, False, sms) == (by_tiles.TWO, 1)
    for Sq, Sk in ((16, 512), (32, 256), (64, 32)):
        assert binding.testing_cross_backward_plan(4, 8, Sq, Sk, sms)[:2] == (0, 1)
        assert binding.testing_cross_backward_plan(4, 8, Sq + 1, Sk, sms)[0] == 1
        assert binding.testing_cross_backward_plan(4, 8, Sq, Sk + 1, sms)[0] == 1


@pytest.mark.parametrize("sms", SMS)
def test_shares_hold_keys(binding, sms):  # noqa: F811
    for H, Sq, Sk in ((1, 1, 1), (1, 1, 100000), (3, 8, 129), (2, 130, 5000), (1, 4096, 100), (1, 300, 128)):
        for ragged in (False, True):
            assert 1 <= binding.testing_cross_plan(1, H, Sq, Sk, ragged, sms)[1] <= -(-Sk // 128)
        _, q, k = binding.testing_cross_backward_plan(1, H, Sq, Sk, sms)
        assert 1 <= q <= -(-Sq // 128) and 1 <= k <= -(-Sk // 64)


def test_refused_sizes_have_no_plan(binding):  # noqa: F811
    for size in ((0, 1, 1, 1), (1, 1, 1, 0), (65536, 1, 1, 1), (1, 1, 2 ** 31 - 1, 1), (1, 1, 1, 2 ** 31 - 1)):
        assert binding.testing_cross_plan(*size, False, 152)[0] == -1
        assert binding.testing_cross_backward_plan(*size, 152)[0] == -1
