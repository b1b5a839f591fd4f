"""GPU parity of mla_cross_attention_backward (through the C ABI) against the float64 definition on the
forward's own out and lse.

Tolerances, element by element: the rounding of the gradient, 2^-8 of itself, and 1.02 times
oracle.cross_ref's bound (P and dS rounded to bf16, fp32 sums; 1.02 for second orders), which is pinned
nowhere but in its arithmetic: a weight off by 2^-8 is 2^-8 |dO| in dV, dS off by 2^-8 is 2^-8 scale |K| in dQ.
"""
import pytest
import torch

from oracle import cross_ref as ref
from tests.test_gpu_cross import DV, SCALE, Problem, randn

pytestmark = pytest.mark.gpu

NAMES = ("dq_nope", "dq_rope", "dk_nope", "dk_rope", "dv")


class Grad(Problem):
    def __init__(self, lib, B, H, Sq, Sk, **kw):
        super().__init__(B, H, Sq, Sk, **kw)
        self.d_out = randn(torch.Generator(device="cuda").manual_seed(B + Sq), B, Sq, H, DV)
        self.out, self.lse = self.run(lib)

    def backward(self, lib, **kw):
        return lib.mla_cross_attention_backward(*self.args()[:5], self.out, self.lse, self.d_out, self.lens,
                                                softmax_scale=self.scale, **kw)

    def check_grads(self, grads):
        want, bounds = ref.backward(*self.args(), self.scale, self.out, self.lse, self.d_out)
        for name, g, x, w in zip(NAMES, grads, want, bounds):
            assert g.dtype == torch.bfloat16 and g.shape == x.shape, name
            err, tol = (g.double() - x).abs(), 2.0 ** -8 * x.abs() + 1.02 * w
            assert bool((err <= tol).all()), (name, (err - tol).max().item())
        for b, n in enumerate(self.counts()):  # written in full
            assert not any(bool(g[b, n:].any()) for g in grads[2:])
            assert n > 0 or not any(bool(g[b].any()) for g in grads[:2])


@pytest.mark.parametrize("B,H,Sq,Sk", [
    (1, 1, 1, 1), (1, 8, 1, 77), (2, 3, 5, 129), (1, 2, 127, 256), (1, 2, 128, 128), (1, 2, 129, 300), (2, 2, 256, 511),
    (1, 3, 257, 130), (3, 5, 385, 64), (1, 1, 513, 1), (2, 1, 2, 640)])
def test_shapes(lib, B, H, Sq, Sk):
    p = Grad(lib, B, H, Sq, Sk)
    grads = p.backward(lib)
    lib.check_device_error()
    p.check_grads(grads)


@pytest.mark.parametrize("Sq", [1, 128, 200])
@pytest.mark.parametrize("Sk,lens", [(300, [300, 0, 1, 127, 128, 129, 255, 256, 257]), (128, [0, 128, 1, 64]), (1, [0, 1]),
                                     (700, [-3, 701, 2 ** 31 - 1, 699, 513])])
def test_key_lengths_with_nan_behind_them(lib, Sq, Sk, lens):
    p = Grad(lib, len(lens), 2, Sq, Sk, lens=lens)
    grads = p.backward(lib)
    lib.check_device_error()
    p.check_grads(grads)


@pytest.mark.parametrize("B,H,Sq,Sk,lens", [
    (1, 1, 40, 6000, None), (1, 2, 3000, 100, None), (1, 1, 1500, 1700, None), (2, 1, 130, 3000, [3000, 0]),
    (3, 1, 5, 2500, [2500, 129, 1300]), (2, 1, 2000, 300, [257, 130])])
def test_streamed_tiles_cut_in_shares(lib, B, H, Sq, Sk, lens):
    p = Grad(lib, B, H, Sq, Sk, lens=lens)
    grads = p.backward(lib)
    lib.check_device_error()
    p.check_grads(grads)


def test_many_heads_repeat_exactly(lib):
    p = Grad(lib, 2, 40, 150, 400, lens=[400, 333])
    grads = p.backward(lib)
    lib.check_device_error()
    p.check_grads(grads)
    assert all(torch.equal(a, b) for _ in range(3) for a, b in zip(grads, p.backward(lib)))


@pytest.mark.parametrize("mag,scale", [(0.0, SCALE), (1e-20, SCALE), (30.0, SCALE), (1.0, 3.0)])
def test_magnitudes_and_scales(lib, mag, scale):
    p = Grad(lib, 2, 2, 70, 333, lens=[333, 200], mag=mag, scale=scale)
    grads = p.backward(lib)
    lib.check_device_error()
    p.check_grads(grads)


def test_gradient_against_differences_of_the_definition(lib):
    p = Grad(lib, 1, 2, 3, 150, lens=[140])
    grads = [g.double() for g in p.backward(lib)]
    x = [t.double() for t in p.args()[:5]]
    g = torch.Generator().manual_seed(4)
    for k, (t, grad) in enumerate(zip(x, grads)):
        for _ in range(12):
            at = tuple(int(torch.randint(0, 140 if d == 1 and k >= 2 else n, (), generator=g)) for d, n in enumerate(t.shape))
            keep, d = t[at].item(), []
            for h in (1e-4, -1e-4):
                t[at] = keep + h
                d.append(float((ref.forward(*x, [140], SCALE)[0] * p.d_out.double()).sum()))
            t[at] = keep
            d = (d[0] - d[1]) / 2e-4
            # the rounding of the gradient and of out (in D), P and dS: sums of 1e-3 of terms of order 1 here
            assert abs(d - float(grad[at])) <= 2.0 ** -8 * abs(d) + 0.02, NAMES[k]


def test_non_finite_values_stay_in_their_sequence_and_head(lib):
    p = Grad(lib, 2, 3, 150, 280)
    clean = p.backward(lib)
    p.v[1, 5, 2, 7] = float("nan")
    grads = p.backward(lib)
    lib.check_device_error()
    for i, (g, c) in enumerate(zip(grads, clean)):
        assert torch.equal(g[0], c[0])
        assert i == 3 or torch.equal(g[1, :, :2], c[1, :, :2])
    assert not bool(torch.isfinite(grads[0][1, :, 2].float()).all())


def test_captured_replayed_and_on_side_streams(lib):
    shapes = [(2, 3, 150, 600, [600, 17]), (1, 1, 1400, 700, [650])]
    ps, new = [[Grad(lib, *s[:4], lens=s[4], seed=k) for s in shapes] for k in (1, 2)]
    ws = [torch.empty(lib.cross_attention_backward_workspace_size(*s[:4]), dtype=torch.uint8, device="cuda") for s in shapes]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in shapes]
    got = [[p.backward(lib, workspace=w, stream=s) for _ in range(3)][-1] for p, w, s in zip(ps, ws, sides)]
    for p, g, s in zip(ps, got, sides):
        s.synchronize()
        p.check_grads(g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [p.backward(lib, workspace=w) for p, w in zip(ps, ws)]
    for p, q in zip(ps, new):
        for a, b in zip(p.args() + (p.out, p.lse, p.d_out), q.args() + (q.out, q.lse, q.d_out)):
            a.copy_(b)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    lib.check_device_error()
    for q, g in zip(new, got):
        q.check_grads(g)


def test_writes_only_its_outputs_and_workspace(lib):
    from tests.test_gpu_canaries import Guarded

    for B, H, Sq, Sk in ((2, 3, 131, 200), (1, 1, 60, 3000), (1, 1, 2500, 140)):
        p = Grad(lib, B, H, Sq, Sk)
        grads = [Guarded(t.shape, torch.bfloat16) for t in p.args()[:5]]
        ws = Guarded((lib.cross_attention_backward_workspace_size(B, H, Sq, Sk),), torch.uint8)
        p.backward(lib, grads=[g.t for g in grads], workspace=ws.t)
        lib.check_device_error()
        assert all(g.intact() for g in grads) and ws.intact()
        p.check_grads([g.t for g in grads])


def test_refusals_on_the_device(lib):
    p = Grad(lib, 2, 2, 4, 300)
    size = lib.cross_attention_backward_workspace_size(2, 2, 4, 300)
    with pytest.raises(lib.MLAError, match="WORKSPACE"):
        p.backward(lib, workspace=torch.empty(size - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="grads"):
        p.backward(lib, grads=[torch.empty_like(t) for t in p.args()[:4]])
    with pytest.raises(TypeError, match="grads"):
        p.backward(lib, grads=[torch.empty_like(t, dtype=torch.float32) for t in p.args()[:5]])
    with pytest.raises(ValueError, match="lse"):
        lib.mla_cross_attention_backward(*p.args()[:5], p.out, p.lse.transpose(1, 2), p.d_out, softmax_scale=SCALE)
