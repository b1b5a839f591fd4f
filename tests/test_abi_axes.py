"""Positions on several axes without a GPU: refusals of the entry points in the C ABI and the binding,
the table of turns, and the oracle's form of the rotation."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import norm_rope_ref as ref
from tests.test_abi_rope import (APPEND, APPEND0, BACKWARD, BACKWARD0, FORWARD, FORWARD0, I, binding, call,  # noqa: F401
                                 clib, cpu)

FREQ = 10000.0 ** (-np.arange(0, 64, 2) / 64)


def with_axes(spec, after="turns"):
    at = [n for n, _ in spec].index(after) + 1
    return spec[:at] + [("axes", I)] + spec[at:]


APPEND_AXES, FORWARD_AXES = with_axes(APPEND), with_axes(FORWARD)
BACKWARD_AXES = with_axes(with_axes(BACKWARD), "ukr")
BACKWARD_AXES[4] = ("ukrt", I)
AXES = [(1, dict(axes=0)), (1, dict(axes=-1)), (2, dict(axes=5)), (2, dict(axes=2 ** 31 - 1)), (1, dict(pos=None)),
        (1, dict(turns=None)), (1, dict(pos=18)), (1, dict(turns=24))]


@pytest.mark.parametrize("want,kw", AXES + [(1, dict(stride=568)), (2, dict(dl=256)), (1, dict(dt=1)), (1, dict(B=0))])
def test_append_refuses(clib, want, kw):
    assert call(clib.mla_rope_append_axes, APPEND_AXES, dict(APPEND0, axes=3), **kw) == want
    assert b"mla_rope_append_axes" in clib.mla_last_error()


@pytest.mark.parametrize("want,kw", AXES + [(1, dict(oqr=None)), (2, dict(dr=128)), (1, dict(qs=385)), (1, dict(R=0))])
def test_norm_refuses(clib, want, kw):
    assert call(clib.mla_qk_norm_rope_axes, FORWARD_AXES, dict(FORWARD0, axes=3), **kw) == want
    assert b"mla_qk_norm_rope_axes" in clib.mla_last_error()


@pytest.mark.parametrize("want,kw", AXES + [(2, dict(ukrt=1)), (2, dict(ukrt=7)), (1, dict(dq=None)), (1, dict(qh=0)),
                                            (1, dict(ukr=24, ukrt=0))])
def test_norm_backward_refuses(clib, want, kw):
    assert call(clib.mla_qk_norm_rope_axes_backward, BACKWARD_AXES, dict(BACKWARD0, axes=3, ukrt=2), **kw) == want
    assert b"mla_qk_norm_rope_axes_backward" in clib.mla_last_error()


def test_binding_refuses(binding):
    turns = binding.rope_turns_axes(FREQ, [0] * 16 + [1] * 16)
    pos = cpu(1, 2, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="one of q"):
        binding.mla_qk_norm_rope_axes(positions=pos, rope_turns=turns)
    with pytest.raises(ValueError, match="CUDA"):
        binding.mla_qk_norm_rope_axes(cpu(1, 2, 3, 192), positions=pos, rope_turns=turns)
    with pytest.raises(ValueError, match="2 dimensions"):  # the table of one axis
        binding.mla_qk_norm_rope_axes(cpu(1, 2, 3, 192), positions=pos, rope_turns=turns[0])
    with pytest.raises(ValueError, match="1 dimensions"):
        binding.mla_qk_norm_rope(cpu(1, 2, 3, 192), positions=pos, rope_turns=turns)
    with pytest.raises(ValueError, match="CUDA"):
        binding.mla_rope_append_axes(cpu(1, 2, 576), cpu(2, 64, 576), cpu(1, 1, dtype=torch.int32),
                                     cpu(1, dtype=torch.int32), rope_turns=turns, positions=pos)
    with pytest.raises(TypeError):
        binding.mla_rope_append_axes(cpu(1, 2, 576), cpu(2, 64, 576), cpu(1, 1, dtype=torch.int32),
                                     cpu(1, dtype=torch.int32), rope_turns=turns)


def test_turns_of_axes(binding):
    one = binding.rope_turns(FREQ)
    axis = [i % 3 for i in range(32)]
    table = binding.rope_turns_axes(FREQ, axis)
    assert table.shape == (3, 32) and table.dtype == torch.int64 and table.is_contiguous()
    for i, a in enumerate(axis):
        assert table[a, i] == one[i] and int(table[:, i].abs().sum()) == abs(int(one[i]))
    assert torch.equal(binding.rope_turns_axes(torch.tensor(FREQ), torch.tensor(axis)), table)
    assert torch.equal(binding.rope_turns_axes(FREQ, [0] * 32)[0], one)
    for bad in ([0] * 31, [0] * 31 + [4], [0] * 31 + [-1], [0.5] * 32, []):
        with pytest.raises(ValueError):
            binding.rope_turns_axes(FREQ, bad)
    with pytest.raises(ValueError, match="finite"):
        binding.rope_turns_axes([float("nan")] * 32, [0] * 32)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_turns_each_pair_by_its_axis(interleaved):
    rng = np.random.default_rng(5)
    axis = rng.permutation([0] * 8 + [1] * 12 + [2] * 12)
    table = np.where(axis == np.arange(3)[:, None], FREQ, 0.0)
    x, pos = rng.standard_normal((2, 3, 4, 64)), rng.integers(-50, 9000, (2, 3, 3))
    got = ref.rotate(x, pos[:, :, None], table, interleaved)
    for a in range(3):
        alone = ref.rotate(x, pos[:, :, None, a], FREQ, interleaved)
        pick = np.repeat(axis == a, 2) if interleaved else np.tile(axis == a, 2)
        assert np.abs(got - alone)[..., pick].max() < 1e-12
    # positions that agree on all axes are one axis (text among images)
    same = np.repeat(pos[..., :1], 3, -1)
    assert np.abs(ref.rotate(x, same[:, :, None], table, interleaved) -
                  ref.rotate(x, pos[:, :, None, 0], FREQ, interleaved)).max() < 1e-12


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_backward_of_axes_against_differences(interleaved):
    rng = np.random.default_rng(6)
    freq = rng.random((2, 3))  # general tables: pairs that both axes turn
    q, kn, kr = rng.standard_normal((1, 2, 2, 10)), rng.standard_normal((1, 2, 2, 4)), rng.standard_normal((1, 2, 6))
    pos, w = rng.integers(0, 9, (1, 2, 2)), [rng.standard_normal(d) for d in (4, 6, 4, 6)]
    up = [rng.standard_normal(s) for s in ((1, 2, 2, 4), (1, 2, 2, 6), (1, 2, 2, 4), (1, 2, 6))]

    def loss():
        return sum((a * b).sum() for a, b in zip(ref.qk_norm_rope(q, kn, kr, pos, freq, w, 1e-3, interleaved), up))

    grads = ref.qk_norm_rope_backward(*up, q, kn, kr, pos, freq, w, 1e-3, interleaved)
    for x, g in zip([q, kn, kr] + w, grads):
        for at in np.ndindex(x.shape):
            keep, d = x[at], []
            for h in (1e-5, -1e-5):
                x[at] = keep + h
                d.append(loss())
            x[at] = keep
            assert abs((d[0] - d[1]) / 2e-5 - g[at]) < 1e-7
