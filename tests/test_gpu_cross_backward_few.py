"""Gradients of cross attention of few queries and keys, which take a form without tiles (up to 16 queries and 512 keys, 32
and 256, or 64 and 32), and of the sizes next to it: strips of 16, steps of 64 keys, runs of several CTAs, sequences without
keys, NaN behind the last key, repeated bit for bit.  Bounds as in test_gpu_cross_backward.py."""
import pytest
import torch

from oracle import cross_ref as ref
from tests.test_gpu_cross_backward import NAMES, Grad

pytestmark = pytest.mark.gpu


def lengths(B, Sk):
    g = torch.Generator().manual_seed(Sk)
    lens = torch.randint(0, Sk + 1, (B,), generator=g)
    lens[0], lens[-1] = Sk, 0
    return lens.tolist()


@pytest.mark.parametrize("Sq", [1, 2, 15, 16, 17, 31, 32, 33, 50, 64, 65])
@pytest.mark.parametrize("Sk", [1, 15, 16, 17, 32, 33, 63, 64, 65, 128, 129, 200, 256, 257])
def test_counts(lib, Sq, Sk):
    for lens in (None, lengths(5, Sk)):
        p = Grad(lib, 5, 3, Sq, Sk, lens=lens)
        grads = p.backward(lib)
        lib.check_device_error()
        p.check_grads(grads)


@pytest.mark.parametrize("B,H,Sq,Sk,lens", [
    (1, 1, 16, 512, None), (2, 2, 9, 511, [511, 65]), (1, 1, 16, 513, None), (3, 1, 30, 250, [250, 129, 0]), (40, 17, 12, 130, None),
    (130, 5, 7, 90, "any"), (60, 40, 3, 20, "any"), (60, 40, 60, 20, "any"), (40, 30, 47, 128, "any")])
def test_runs_and_many_heads_repeat_exactly(lib, B, H, Sq, Sk, lens):
    p = Grad(lib, B, H, Sq, Sk, lens=lengths(B, Sk) if lens == "any" else lens)
    grads = p.backward(lib)
    lib.check_device_error()
    p.check_grads(grads)
    assert all(torch.equal(a, b) for _ in range(3) for a, b in zip(grads, p.backward(lib)))


@pytest.mark.parametrize("Sq", [5, 29])
@pytest.mark.parametrize("mag,scale", [(0.0, 0.07), (1e-20, 0.07), (30.0, 0.07), (1.0, 3.0)])
def test_magnitudes_and_scales(lib, Sq, mag, scale):
    # Weights of peaked rows pass below the normal numbers: a P or dS under 2^-126 is 0, which the bounds leave out.  With
    # |dP - D| <= 2 * 128 max|dO| max|V| and n terms, dV is off by 2^-126 n max|dO| more, dK and dQ by scale n max|Q or K|
    # times 2^-126 (|dP - D| + 1).
    p = Grad(lib, 2, 2, Sq, 133, lens=[133, 70], mag=mag, scale=scale)
    grads = p.backward(lib)
    lib.check_device_error()
    top = lambda *ts: max(t.float().nan_to_num(0.0).abs().max().item() for t in ts)  # noqa: E731
    n, do = 2 * 133, top(p.d_out)
    tiny = 2.0 ** -126 * n * max(do, scale * top(p.qn, p.qr, p.kn, p.kr) * (2 * 128 * do * top(p.v) + 1))
    assert tiny < 1e-29
    want, bounds = ref.backward(*p.args(), p.scale, p.out, p.lse, p.d_out)
    for name, g, x, w in zip(NAMES, grads, want, bounds):
        assert bool(((g.double() - x).abs() <= 2.0 ** -8 * x.abs() + 1.02 * w + tiny).all()), name


def test_non_finite_values_stay_in_their_sequence_and_head(lib):
    p = Grad(lib, 2, 3, 20, 130)
    clean = p.backward(lib)
    p.v[1, 5, 2, 7] = float("nan")
    grads = p.backward(lib)
    lib.check_device_error()
    for i, (g, c) in enumerate(zip(grads, clean)):
        assert torch.equal(g[0], c[0])
        assert i == 3 or torch.equal(g[1, :, :2], c[1, :, :2])
    assert not bool(torch.isfinite(grads[0][1, :, 2].float()).all())


def test_writes_only_its_outputs_and_workspace(lib):
    from tests.test_gpu_canaries import Guarded

    for B, H, Sq, Sk in ((2, 3, 16, 200), (1, 1, 11, 500), (1, 1, 32, 256), (3, 5, 1, 3), (2, 3, 61, 33), (2, 3, 64, 128)):
        p = Grad(lib, B, H, Sq, Sk)
        grads = [Guarded(t.shape, torch.bfloat16) for t in p.args()[:5]]
        ws = Guarded((lib.cross_attention_backward_workspace_size(B, H, Sq, Sk),), torch.uint8)
        p.backward(lib, grads=[g.t for g in grads], workspace=ws.t)
        lib.check_device_error()
        assert all(g.intact() for g in grads) and ws.intact()
        p.check_grads([g.t for g in grads])
