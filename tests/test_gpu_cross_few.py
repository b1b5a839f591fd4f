"""Cross attention of one to nine queries a sequence (up to eight take a form without tiles): every count, key lengths
around the steps of 16 and 128 keys and the shares, NaN and infinity behind the last key and before it, rows of
unlike maxima.  Bounds as in test_gpu_cross.py."""
import pytest
import torch

from tests.test_gpu_cross import Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Sq", range(1, 10))
@pytest.mark.parametrize("B,H,Sk,lens", [
    (12, 3, 300, [0, 1, 2, 3, 4, 7, 15, 16, 17, 127, 129, 300]), (2, 1, 16, None), (3, 2, 2100, [2100, 129, 0]),
    (40, 16, 140, None), (1, 1, 40000, None)])
def test_counts_and_lengths(lib, Sq, B, H, Sk, lens):
    p = Problem(B, H, Sq, Sk, lens=lens)
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)
    assert all(torch.equal(a, b) for a, b in zip(got, p.run(lib)))


@pytest.mark.parametrize("Sq", [1, 2, 7, 8])
def test_rising_and_falling_maxima(lib, Sq):
    p = Problem(1, 2, Sq, 1500, mag=0.3)
    ramp = torch.arange(1500, device="cuda") // 16 * 0.5
    p.qn[..., 0] = torch.tensor([4.0, -4.0] * 4, device="cuda")[:Sq, None].bfloat16()
    p.kn[..., 0] = ramp[:, None].bfloat16()
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)


@pytest.mark.parametrize("Sq", [1, 3, 8])
def test_infinite_and_nan_values(lib, Sq):
    p = Problem(3, 2, Sq, 700, lens=[700, 650, 300])
    clean = p.run(lib)
    p.kn[0, 650, 1, 0] = float("-inf")  # scores of -inf or +inf by the sign of the query's column
    p.qn[0, :, 1, 0] = 1.0
    p.v[1, 649, 0, 5] = float("nan")
    p.kn[2, 299, 1] = float("nan")
    p.v[2, 300:] = float("inf")
    out, lse = p.run(lib)
    lib.check_device_error()
    # a key with a score of -inf has no weight
    assert bool(torch.isfinite(out[0].float()).all()) and bool(torch.isfinite(lse[0]).all())
    assert torch.equal(out[0, :, 0], clean[0][0, :, 0])
    assert bool(torch.isnan(out[1, :, 0, 5]).all()) and torch.equal(out[1, :, 0, 6:], clean[0][1, :, 0, 6:])
    assert torch.equal(out[1, :, 1], clean[0][1, :, 1]) and torch.equal(lse[1], clean[1][1])
    assert bool(torch.isnan(out[2, :, 1].float()).all()) and torch.equal(out[2, :, 0], clean[0][2, :, 0])


@pytest.mark.parametrize("Sq", [1, 5])
def test_keys_that_no_query_sees(lib, Sq):
    # all scores -inf: no weight anywhere, as without keys
    p = Problem(1, 2, Sq, 200)
    p.qn[..., 0] = 1.0
    p.kn[:, :, 1, 0] = float("-inf")
    out, lse = p.run(lib)
    lib.check_device_error()
    assert not bool(out[:, :, 1].any()) and bool(torch.isneginf(lse[:, 1]).all())
    assert bool(torch.isfinite(lse[:, 0]).all())


@pytest.mark.parametrize("Sq", [1, 6])
@pytest.mark.parametrize("mag,scale", [(0.0, 0.07), (1e-20, 0.07), (30.0, 0.07), (1.0, 1e-6), (1.0, 3.0)])
def test_magnitudes_and_scales(lib, Sq, mag, scale):
    p = Problem(2, 2, Sq, 333, lens=[333, 200], mag=mag, scale=scale)
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)


@pytest.mark.parametrize("Sq", [1, 8])
def test_offsets_past_32_bits(lib, Sq):
    # 128 heads x 140000 keys: the heads at the ends, over all keys
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    p = Problem(1, 1, Sq, 8)
    x = rnd(1, Sq, 128, 128), rnd(1, Sq, 128, 64), rnd(1, 140000, 128, 128), rnd(1, 140000, 64), rnd(1, 140000, 128, 128)
    out, lse = lib.mla_cross_attention(*x, softmax_scale=p.scale)
    lib.check_device_error()
    for h in (0, 127):
        p.qn, p.qr, p.kn, p.kr, p.v = (t[:, :, h:h + 1] if t.dim() == 4 else t for t in x)
        p.Sk = 140000
        p.check(out[:, :, h:h + 1], lse[:, h:h + 1])
