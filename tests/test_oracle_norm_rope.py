"""Pins of the head-norm, rotation, rotated-append and drafted-tree oracles, and of the host-side
helpers that make the operators' plans (CPU only)."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from gen import make_decode
from oracle import norm_rope_ref as ref

THETA = 10000.0


def inv_freq(n=64):
    return THETA ** (-np.arange(0, n, 2) / n)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_multiplication_by_a_unit_complex_number(interleaved):
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((3, 5, 64)), rng.integers(-100, 100000, (3, 5))
    z = x[..., 0::2] + 1j * x[..., 1::2] if interleaved else x[..., :32] + 1j * x[..., 32:]
    want = z * np.exp(1j * pos[..., None] * inv_freq())
    y = ref.rotate(x, pos, inv_freq(), interleaved)
    got = y[..., 0::2] + 1j * y[..., 1::2] if interleaved else y[..., :32] + 1j * y[..., 32:]
    assert np.abs(got - want).max() < 1e-12
    # scores of rotated pairs depend on the distance of their positions only
    a = (ref.rotate(x, pos, inv_freq(), interleaved) * ref.rotate(x, pos + 7, inv_freq(), interleaved)).sum(-1)
    b = (x * ref.rotate(x, np.full_like(pos, 7), inv_freq(), interleaved)).sum(-1)
    assert np.abs(a - b).max() < 1e-9


def test_rms_against_closed_forms():
    x = np.array([[3.0, -4.0, 0.0, 0.0]])
    assert np.allclose(ref.rms(x, np.ones(4), 0.0), x / 2.5, atol=0, rtol=1e-15)
    assert (ref.rms(np.zeros((2, 4)), np.ones(4), 1e-6) == 0).all()
    assert ref.rms(x, None, 1e-6) is x or np.array_equal(ref.rms(x, None, 1e-6), x)
    t = torch.randn(3, 8, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    w = torch.randn(8, dtype=torch.float64, generator=torch.Generator().manual_seed(2))
    want = torch.nn.functional.rms_norm(t, (8,), w, 1e-3).numpy()
    assert np.abs(ref.rms(t.numpy(), w.numpy(), 1e-3) - want).max() < 1e-14


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_backward_against_differences_and_autograd(interleaved, norm):
    rng = np.random.default_rng(3)
    B, S, H, dn, dr, eps = 1, 2, 2, 4, 6, 1e-3
    freq = inv_freq(dr)
    x = {"q": rng.standard_normal((B, S, H, dn + dr)), "kn": rng.standard_normal((B, S, H, dn)),
         "kr": rng.standard_normal((B, S, dr))}
    w = [rng.standard_normal(d) if norm else None for d in (dn, dr, dn, dr)]
    pos = rng.integers(0, 50, (B, S))
    up = [rng.standard_normal(s) for s in ((B, S, H, dn), (B, S, H, dr), (B, S, H, dn), (B, S, dr))]

    def loss():
        y = ref.qk_norm_rope(x["q"], x["kn"], x["kr"], pos, freq, w, eps, interleaved)
        return sum(float((a * b).sum()) for a, b in zip(y, up))

    got = ref.qk_norm_rope_backward(*up, x["q"], x["kn"], x["kr"], pos, freq, w, eps, interleaved)
    leaves = [x["q"], x["kn"], x["kr"]] + w
    for leaf, g in zip(leaves, got):
        if leaf is None:
            assert g is None
            continue
        for idx in np.ndindex(*leaf.shape):
            keep, h = leaf[idx], 1e-5
            leaf[idx] = keep + h
            a = loss()
            leaf[idx] = keep - h
            b = loss()
            leaf[idx] = keep
            # central differences: h^2 truncation (~1e-9) and 2^-52 |loss| / h rounding (~1e-10)
            assert abs((a - b) / (2 * h) - g[idx]) < 1e-7
    # autograd through torch's own norm and complex product
    t = [None if v is None else torch.tensor(v, requires_grad=True) for v in leaves]
    ang = torch.tensor(pos)[..., None] * torch.tensor(freq)

    def turned(v, a):
        z = torch.view_as_complex(v.unflatten(-1, (-1, 2)).contiguous()) if interleaved else \
            torch.complex(*v.chunk(2, -1))
        z = z * torch.polar(torch.ones_like(a), a)
        return torch.view_as_real(z).flatten(-2) if interleaved else torch.cat((z.real, z.imag), -1)

    def normed(v, wt):
        return v if wt is None else torch.nn.functional.rms_norm(v, (v.shape[-1],), wt, eps)

    y = (normed(t[0][..., :dn], t[3]), turned(normed(t[0][..., dn:], t[4]), ang[:, :, None]),
         normed(t[1], t[5]), turned(normed(t[2], t[6]), ang))
    sum((a * torch.tensor(b)).sum() for a, b in zip(y, up)).backward()
    for leaf, g in zip(t, got):
        if leaf is not None:
            assert np.abs(leaf.grad.numpy() - g).max() < 1e-12


def test_append_places():
    p = ref.append_places([5, 2, 9, 4, 1], [3, 3, 0, 4, 2], 3)
    assert p.tolist() == [[2, 3, 4], [-1, 0, 1], [-1, -1, -1], [-1, -1, -1], [-1, 0, -1]]


# ----------------------------------------------------------------------------- drafted trees

def chain(B, T):
    return np.broadcast_to(np.tril(np.ones((T, T), bool)), (B, T, T))


@pytest.mark.parametrize("fp8", [False, True])
def test_a_chain_is_the_causal_decode(fp8):
    inp = make_decode(4, 2, 3, [0, 2, 3, 70], fp8=fp8, seed=3, extra_pages=1)
    O, L = oracle.mla_decode(inp)
    O2, L2 = oracle.mla_decode_tree(inp, chain(4, 3))
    assert np.abs(O - O2).max() < 1e-12
    assert np.array_equal(np.isneginf(L), np.isneginf(L2))
    fin = np.isfinite(L)
    assert np.abs(L[fin] - L2[fin]).max() < 1e-12


def test_tree_against_each_branch_decoded_alone():
    # every root-to-node path decoded as a chain over a cache holding only that path
    parents = [-1, 0, 0, 1, -1, 4, 3]
    T = len(parents)
    inp = make_decode(1, 2, T, [90], seed=5)
    C = oracle.decode_gather(inp, 0)
    sees = np.zeros((1, T, T), bool)
    for t in range(T):
        j = t
        while j >= 0:
            sees[0, t, j] = True
            j = parents[j]
    O, L = oracle.mla_decode_tree(inp, sees)
    for t in range(T):
        path = [j for j in range(T) if sees[0, t, j]]
        rows = np.concatenate([C[:90 - T], C[90 - T:][path]])
        q = np.concatenate([oracle.bf16_to_f64(inp.q_latent[0, t]), oracle.bf16_to_f64(inp.q_rope[0, t])], 1)
        s = inp.softmax_scale * q @ rows.T
        p = np.exp(s - s.max(1, keepdims=True))
        assert np.abs((p / p.sum(1, keepdims=True)) @ rows[:, :512] - O[0, t]).max() < 1e-12
        assert np.abs(np.log(p.sum(1)) + s.max(1) - L[0, :, t]).max() < 1e-12


def test_padding_and_unseen_drafts_do_not_matter():
    inp = make_decode(2, 2, 4, [66, 3], seed=9)
    sees = chain(2, 4).copy()
    sees[0, 1] = False
    O, L = oracle.mla_decode_tree(inp, sees, [2, 0])
    assert np.isneginf(L[:, :, 2:]).all() and (O[:, 2:] == 0).all()
    assert np.isneginf(L[1]).all() and (O[1] == 0).all()
    # row 1 of sequence 0 sees the 64 keys of the prefix only
    C = oracle.decode_gather(inp, 0)[:64]
    q = np.concatenate([oracle.bf16_to_f64(inp.q_latent[0, 1]), oracle.bf16_to_f64(inp.q_rope[0, 1])], 1)
    s = inp.softmax_scale * q @ C.T
    assert np.abs(np.log(np.exp(s - s.max(1, keepdims=True)).sum(1)) + s.max(1) - L[0, :, 1]).max() < 1e-12


# ---------------------------------------------------------------------------- host-side plans

@pytest.fixture(scope="module")
def binding():
    import os

    from mla_flash_attention_gb300 import build

    if not (os.path.exists(build.LIB) and os.path.exists(build.MARSHAL)):
        build.build()
    from mla_flash_attention_gb300 import binding

    return binding


def test_rope_turns_keep_far_angles(binding):
    f = inv_freq()
    turns = binding.rope_turns(torch.from_numpy(f))
    assert turns.dtype == torch.int64 and turns.shape == (32,)
    for i, t in enumerate(turns.tolist()):
        for pos in (0, 1, 12345, 2 ** 31 - 1, -(2 ** 31)):
            phase = Fraction((pos * t) % 2 ** 64, 2 ** 64)
            exact = Fraction(pos) * Fraction(float(f[i])) / Fraction(2 * math.pi)
            off = (phase - exact) % 1
            off = min(off, 1 - off)
            # half a unit of 2^-64 a position, and the 2^-53 of f / (2 pi) in fp64
            assert off <= abs(pos) * (Fraction(1, 2 ** 64) + Fraction(float(f[i])) * Fraction(1, 2 ** 53))
    assert binding.rope_turns([0.0, 2 * math.pi]).tolist() == [0, 0]  # whole turns fall off
    with pytest.raises(ValueError):
        binding.rope_turns([float("nan")])


@pytest.mark.parametrize("T", [1, 2, 7, 32, 33, 64, 130])
def test_tree_masks_from_parents(binding, T):
    rng = np.random.default_rng(T)
    parents = np.stack([[int(rng.integers(-1, t)) if t else -1 for t in range(T)],
                        np.arange(T) - 1])  # a random tree and a chain
    mask, depth = binding.tree_mask_from_parents(torch.from_numpy(parents))
    words = (T + 31) // 32
    assert mask.shape == (2, T, words) and mask.dtype == torch.int32 and depth.dtype == torch.int32
    for b in range(2):
        for t in range(T):
            want, j, d = set(), t, -1
            while j >= 0:
                want.add(j)
                j = parents[b, j]
                d += 1
            got = {j for j in range(words * 32) if int(mask[b, t, j // 32]) >> (j % 32) & 1}
            assert got == want and int(depth[b, t]) == d
    one, _ = binding.tree_mask_from_parents(parents[0].tolist())
    assert torch.equal(one, mask[0])


@pytest.mark.parametrize("bad", [[0], [-2], [-1, 1], [], [0.5], [[[-1]]]])
def test_tree_mask_refuses(binding, bad):
    with pytest.raises(ValueError):
        binding.tree_mask_from_parents(bad)
