"""Cross attention with heads enough that every call takes its tiles (small ones do without): row blocks of one kind and
of both, odd counts of rows and keys, key lengths around the tiles, shares, few rows past eight.  Bounds as in
test_gpu_cross.py."""
import pytest
import torch

from tests.test_gpu_cross import Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,Sq,Sk", [
    (1, 80, 9, 500), (2, 40, 31, 333), (1, 40, 127, 256), (1, 40, 128, 257), (1, 40, 129, 300), (2, 16, 256, 511),
    (1, 60, 257, 130), (1, 9, 300, 1025), (3, 9, 385, 64), (1, 1100, 513, 1), (40, 80, 25, 64), (2, 80, 100, 65)])
def test_shapes(lib, B, H, Sq, Sk):
    p = Problem(B, H, Sq, Sk)
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)
    assert all(torch.equal(a, b) for a, b in zip(got, p.run(lib)))


@pytest.mark.parametrize("Sq", [20, 128, 200, 300])
@pytest.mark.parametrize("Sk,lens", [
    (300, [300, 0, 1, 127, 128, 129, 255, 256, 257]), (128, [0, 128, 1, 64]), (700, [-3, 701, 2 ** 31 - 1, -2 ** 31, 699, 513])])
def test_key_lengths_with_nan_behind_them(lib, Sq, Sk, lens):
    p = Problem(len(lens), 1 + 80000 * 8 // (len(lens) * Sq * Sk), Sq, Sk, lens=lens)
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)


@pytest.mark.parametrize("B,H,Sq,Sk,lens", [(1, 2, 130, 5000, None), (1, 3, 40, 9097, None), (2, 1, 300, 3000, [3000, 1])])
def test_keys_split_over_the_gpu(lib, B, H, Sq, Sk, lens):
    assert lib.cross_attention_workspace_size(B, H, Sq, Sk) > 0
    p = Problem(B, H, Sq, Sk, lens=lens)
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)


@pytest.mark.parametrize("mag,scale", [(0.0, 0.07), (1e-20, 0.07), (30.0, 0.07), (1.0, 1e-6), (1.0, 3.0)])
def test_magnitudes_and_scales(lib, mag, scale):
    p = Problem(2, 14, 70, 333, lens=[333, 200], mag=mag, scale=scale)
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)


def test_rising_maxima(lib):
    p = Problem(1, 4, 200, 900, mag=0.3)
    ramp = 1 + torch.arange(900, device="cuda") // 128 * 8
    p.qn[..., 0] = 4.0
    p.kn[..., 0] = ramp[:, None].bfloat16()
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)


def test_small_calls_in_blocks_of_eight_rows(lib):
    # without tiles: a block's rows, keys and shares at every edge
    for B, H, Sq, Sk, lens in ((2, 2, 9, 300, None), (1, 3, 16, 700, None), (1, 1, 100, 4000, None), (3, 2, 63, 130, [130, 0, 17]),
                               (1, 1, 4096, 40, None), (50, 30, 24, 64, None), (50, 30, 17, 33, None)):
        p = Problem(B, H, Sq, Sk, lens=lens)
        got = p.run(lib)
        lib.check_device_error()
        p.check(*got)
