"""Pins of the cross attention oracle (CPU only): torch's attention in float64, closed forms, differences."""
import math

import pytest
import torch

from oracle import cross_ref as ref

SCALE = 0.3


def problem(B=2, H=2, Sq=3, Sk=5, dn=4, dr=2, dv=3, seed=0):
    g = torch.Generator().manual_seed(seed)
    shapes = ((B, Sq, H, dn), (B, Sq, H, dr), (B, Sk, H, dn), (B, Sk, dr), (B, Sk, H, dv))
    return [torch.randn(s, generator=g, dtype=torch.float64) for s in shapes]


@pytest.mark.parametrize("lens", [None, [5, 2], [0, 7], [-1, 1]])
def test_forward_is_torchs_attention_over_the_keys_that_exist(lens):
    qn, qr, kn, kr, v = problem()
    o, lse, a, e = ref.forward(qn, qr, kn, kr, v, lens, SCALE)
    for b, n in enumerate(ref.counts(kn, lens)):
        if n == 0:
            assert not bool(o[b].any()) and bool(torch.isneginf(lse[b]).all())
            continue
        q = torch.cat((qn[b], qr[b]), -1).transpose(0, 1)
        k = torch.cat((kn[b, :n], kr[b, :n, None].expand(-1, 2, -1)), -1).transpose(0, 1)
        want = torch.nn.functional.scaled_dot_product_attention(q, k, v[b, :n].transpose(0, 1), scale=SCALE)
        assert (o[b].transpose(0, 1) - want).abs().max() < 1e-14
        assert (lse[b] - torch.logsumexp(SCALE * q @ k.transpose(1, 2), -1)).abs().max() < 1e-14
        assert bool((a[b] >= o[b].abs() - 1e-14).all()) and bool((e[b] > 0).all())


def test_equal_scores_give_the_mean_of_the_values_that_exist():
    qn, qr, kn, kr, v = problem()
    o, lse, _, _ = ref.forward(0 * qn, 0 * qr, kn, kr, v, [3, 5], SCALE)
    assert (o[0] - v[0, :3].mean(0)).abs().max() < 1e-14 and (lse[0] - math.log(3)).abs().max() < 1e-14
    assert (o[1] - v[1].mean(0)).abs().max() < 1e-14


def test_keys_behind_the_last_do_not_matter():
    qn, qr, kn, kr, v = problem()
    a = ref.forward(qn, qr, kn, kr, v, [3, 4], SCALE)
    kn[0, 3:], kr[0, 3:], v[0, 3:], v[1, 4:] = float("nan"), float("nan"), float("inf"), float("nan")
    assert all(torch.equal(x, y) for x, y in zip(a, ref.forward(qn, qr, kn, kr, v, [3, 4], SCALE)))


@pytest.mark.parametrize("lens", [None, [4, 1], [0, 5]])
def test_backward_against_differences_of_the_forward(lens):
    x = problem()
    d_out = torch.randn(2, 3, 2, 3, generator=torch.Generator().manual_seed(9), dtype=torch.float64)
    o, lse, _, _ = ref.forward(*x, lens, SCALE)
    grads, bounds = ref.backward(*x, lens, SCALE, o, lse, d_out)
    for t, g, w in zip(x, grads, bounds):
        assert g.shape == t.shape == w.shape and bool((w >= 0).all())
        flat = t.view(-1)
        for i in range(flat.numel()):
            keep, d = float(flat[i]), []
            for h in (1e-5, -1e-5):
                flat[i] = keep + h
                d.append(float((ref.forward(*x, lens, SCALE)[0] * d_out).sum()))
            flat[i] = keep
            assert abs((d[0] - d[1]) / 2e-5 - float(g.view(-1)[i])) < 1e-8


def test_shares_join_by_their_log_sums():
    qn, qr, kn, kr, v = problem(Sk=6)
    whole, lse, _, _ = ref.forward(qn, qr, kn, kr, v, None, SCALE)
    parts = [ref.forward(qn, qr, kn[:, c], kr[:, c], v[:, c], None, SCALE)[:2] for c in (slice(0, 2), slice(2, 6))]
    joined = torch.logaddexp(parts[0][1], parts[1][1])
    o = sum(torch.exp(l - joined).transpose(1, 2)[..., None] * p for p, l in parts)
    assert (joined - lse).abs().max() < 1e-14 and (o - whole).abs().max() < 1e-14
