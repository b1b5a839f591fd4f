"""GPU parity of mla_cross_attention (through the C ABI) against a plain float64 form.

Tolerances, element by element.  A softmax weight enters the product with V rounded to bf16, off by at
most 2^-8 of itself, and O is normalised by the sum of the rounded weights: with A = sum_j p_j |v_j| the
error is at most 2^-8 (A + |O|) (1 + 2^-7 for the second order), and storing O rounds it by 2^-8 |O|.  A score
is an fp32 sum of 192 exact products: off by at most 192 * 2^-24 of scale * sum |q k|, below 2^-16 of it
with the two roundings of its exponent's argument; with e the largest of these in the row, weights are off
by 2 e, so O by 4 e A more, and the LSE by e and 2^-20 (1 + |LSE|) for exponentials, sums and logarithm.  A join of
shares adds fp32 roundings that the 2^-7 of the second order covers.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DN, DR, DV = 128, 64, 128
SCALE = 192 ** -0.5


def randn(gen, *shape, mag=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * mag).to(dtype)


class Problem:
    def __init__(self, B, H, Sq, Sk, lens=None, seed=0, mag=1.0, scale=SCALE, poison=True):
        g = torch.Generator(device="cuda").manual_seed(seed + 1000003 * Sq + Sk)
        self.B, self.H, self.Sq, self.Sk, self.scale = B, H, Sq, Sk, scale
        self.qn, self.qr = randn(g, B, Sq, H, DN, mag=mag), randn(g, B, Sq, H, DR, mag=mag)
        self.kn, self.kr, self.v = randn(g, B, Sk, H, DN), randn(g, B, Sk, DR), randn(g, B, Sk, H, DV)
        self.lens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        for b, n in enumerate(self.counts()):
            if poison:  # what stands behind the last key does not matter
                self.kn[b, n:] = self.kr[b, n:] = self.v[b, n:] = float("nan")

    def counts(self):
        return [self.Sk] * self.B if self.lens is None else [min(max(n, 0), self.Sk) for n in self.lens.tolist()]

    def args(self):
        return self.qn, self.qr, self.kn, self.kr, self.v, self.lens

    def run(self, lib, **kw):
        return lib.mla_cross_attention(*self.args(), softmax_scale=self.scale, **kw)

    def reference(self):
        """(O, LSE, A, e): float64 results and the bounds' parts."""
        B, H, Sq = self.B, self.H, self.Sq
        o = torch.zeros(B, Sq, H, DV, dtype=torch.float64, device="cuda")
        a, lse = o.clone(), torch.full((B, H, Sq), -math.inf, dtype=torch.float64, device="cuda")
        e = torch.zeros(B, H, Sq, dtype=torch.float64, device="cuda")
        for b, n in enumerate(self.counts()):
            for h in range(H if n else 0):
                q = torch.cat((self.qn[b, :, h], self.qr[b, :, h]), -1).double()
                k = torch.cat((self.kn[b, :n, h], self.kr[b, :n]), -1).double()
                v = self.v[b, :n, h].double()
                s = (q @ k.T) * self.scale
                lse[b, h] = torch.logsumexp(s, -1)
                p = torch.exp(s - lse[b, h][:, None])
                o[b, :, h], a[b, :, h] = p @ v, p @ v.abs()
                e[b, h] = 2.0 ** -16 * ((q.abs() @ k.abs().T) * self.scale).amax(-1)
        return o, lse, a, e

    def check(self, out, lse):
        o, want, a, e = self.reference()
        assert out.dtype == torch.bfloat16 and lse.dtype == torch.float32
        assert bool(torch.isfinite(out.float()).all())
        tol = 2.0 ** -8 * (o.abs() + (1 + 2.0 ** -7) * (a + o.abs())) + 4 * e.transpose(1, 2)[..., None] * a
        err = (out.double() - o).abs()
        assert bool((err <= tol).all()), (err - tol).max().item()
        none = torch.isneginf(want)
        assert torch.equal(torch.isneginf(lse), none)
        got, want, e = lse.double()[~none], want[~none], e[~none]
        assert bool(((got - want).abs() <= e + 2.0 ** -20 * (1 + want.abs())).all()), (got - want).abs().max().item()


@pytest.mark.parametrize("B,H,Sq,Sk", [
    (1, 1, 1, 1), (1, 8, 1, 77), (2, 3, 1, 128), (2, 3, 5, 129), (1, 2, 31, 33), (1, 2, 127, 256), (1, 2, 128, 257),
    (1, 2, 129, 300), (2, 2, 256, 511), (1, 3, 257, 130), (1, 1, 300, 1025), (3, 5, 385, 64), (1, 1, 513, 1),
    (2, 1, 2, 640)])
def test_shapes(lib, B, H, Sq, Sk):
    p = Problem(B, H, Sq, Sk)
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)


@pytest.mark.parametrize("Sq", [1, 40, 128, 200, 300])
@pytest.mark.parametrize("Sk,lens", [
    (300, [300, 0, 1, 127, 128, 129, 255, 256, 257]), (128, [0, 128, 1, 64]), (1, [0, 1]),
    (700, [-3, 701, 2 ** 31 - 1, -2 ** 31, 699, 513])])
def test_key_lengths_with_nan_behind_them(lib, Sq, Sk, lens):
    p = Problem(len(lens), 2, Sq, Sk, lens=lens)
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)


def test_all_sequences_without_keys(lib):
    for Sq in (1, 129):
        p = Problem(3, 2, Sq, 500, lens=[0, 0, -1])
        out, lse = p.run(lib)
        lib.check_device_error()
        assert not bool(out.any()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("B,H,Sq,Sk,lens", [
    (1, 1, 1, 20000, None), (1, 2, 130, 5000, None), (1, 3, 7, 4097, None), (2, 1, 300, 3000, [3000, 1]),
    (3, 2, 1, 9000, [9000, 0, 130])])
def test_keys_split_over_the_gpu(lib, B, H, Sq, Sk, lens):
    assert lib.cross_attention_workspace_size(B, H, Sq, Sk) > 0
    p = Problem(B, H, Sq, Sk, lens=lens)
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)


@pytest.mark.parametrize("B,H,Sq,Sk", [(7, 64, 1, 300), (9, 61, 3, 700), (5, 70, 300, 200), (3, 80, 400, 260)])
def test_several_units_a_cta_of_unlike_lengths(lib, B, H, Sq, Sk):
    # more units than SMs: every CTA's rings and barriers run on from one to the next, some without keys
    lens = [(b * 7919 + 1) * 131 % (Sk + 1) for b in range(B)]
    lens[0], lens[-1] = 0, Sk
    p = Problem(B, H, Sq, Sk, lens=lens)
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)
    again = p.run(lib)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("Sq", [2, 200])
def test_rising_maxima(lib, Sq):
    # each key tile's scores above the ones before by far more than the 2^8 that is let pass
    p = Problem(1, 2, Sq, 900, mag=0.3)
    ramp = 1 + torch.arange(900, device="cuda") // 128 * 8
    p.qn[..., 0] = 4.0
    p.kn[..., 0] = ramp[:, None].bfloat16()
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)


@pytest.mark.parametrize("mag,scale", [(0.0, SCALE), (1e-20, SCALE), (30.0, SCALE), (1.0, 1e-6), (1.0, 3.0)])
def test_magnitudes_and_scales(lib, mag, scale):
    p = Problem(2, 2, 70, 333, lens=[333, 200], mag=mag, scale=scale)
    got = p.run(lib)
    lib.check_device_error()
    p.check(*got)


def test_non_finite_values_stay_in_their_head_and_sequence(lib):
    p = Problem(2, 3, 150, 280)
    clean = p.run(lib)
    p.v[0, 5, 1, 7] = float("nan")
    p.kn[1, 200, 2, 3] = float("inf")
    p.qn[1, 9, 0, 0] = float("nan")
    out, lse = p.run(lib)
    lib.check_device_error()
    assert bool(torch.isnan(out[0, :, 1, 7]).all()) and not bool(torch.isfinite(out[1, :, 2].float()).all())
    assert bool(torch.isnan(out[1, 9, 0]).all()) and bool(torch.isnan(lse[1, 0, 9]))
    keep = torch.ones(2, 150, 3, dtype=torch.bool, device="cuda")
    keep[0, :, 1] = keep[1, :, 2] = keep[1, 9, 0] = False
    assert torch.equal(out[keep], clean[0][keep])
    keep = keep.transpose(1, 2)
    assert torch.equal(lse[keep], clean[1][keep])
    assert torch.equal(out[0, :, 1, 8:], clean[0][0, :, 1, 8:]) and torch.equal(lse[0], clean[1][0])


def test_square_without_mask_is_the_prefill(lib):
    p = Problem(1, 3, 300, 300)
    out, lse = lib.mla_prefill(*p.args()[:5], softmax_scale=SCALE, causal=False)
    p.check(out, lse)
    p.check(*p.run(lib))


def test_prefix_joined_with_the_causal_rest_is_the_whole(lib):
    # a prompt in two chunks: the second one's queries see the first chunk's keys, then causally their own
    S, C = 400, 260
    p = Problem(1, 2, S, S)
    whole, whole_lse = lib.mla_prefill(*p.args()[:5], softmax_scale=SCALE, causal=True)
    tail = [t[:, C:].contiguous() for t in p.args()[:5]]
    head = [t[:, :C].contiguous() for t in p.args()[2:5]]
    a, la = lib.mla_cross_attention(tail[0], tail[1], *head, softmax_scale=SCALE)
    b, lb = lib.mla_prefill(*tail, softmax_scale=SCALE, causal=True)
    lse = torch.logaddexp(la, lb)
    w = [torch.exp(x - lse).transpose(1, 2)[..., None] for x in (la, lb)]
    got = w[0] * a.float() + w[1] * b.float()
    assert (lse - whole_lse[:, :, C:]).abs().max() < 1e-5
    # three results of 2^-8 (A + 2 |O|) each, with A and |O| below 4 here
    assert (got - whole[:, C:].float()).abs().max() < 0.03


def test_captured_replayed_and_on_side_streams(lib):
    shapes = [(2, 4, 1, 3000, [3000, 17]), (1, 2, 300, 700, [650])]
    ps = [Problem(*s[:4], lens=s[4], seed=1) for s in shapes]
    new = [Problem(*s[:4], lens=[s[4][0] - 5] + s[4][1:], seed=2) for s in shapes]
    ws = [torch.empty(max(16, lib.cross_attention_workspace_size(*s[:4])), dtype=torch.uint8, device="cuda") for s in shapes]
    sides = [torch.cuda.Stream() for _ in shapes]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [[p.run(lib, workspace=w, stream=s) for _ in range(3)][-1] for p, w, s in zip(ps, ws, sides)]  # both at once
    for p, g, s in zip(ps, got, sides):
        s.synchronize()
        p.check(*g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [p.run(lib, workspace=w) for p, w in zip(ps, ws)]
    for p, q in zip(ps, new):
        for a, b in zip(p.args(), q.args()):
            a.copy_(b)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    lib.check_device_error()
    for q, g in zip(new, got):
        q.check(*g)


def test_writes_only_its_outputs_and_workspace(lib):
    from tests.test_gpu_canaries import Guarded

    for B, H, Sq, Sk in ((1, 2, 3, 4000), (2, 3, 131, 200), (1, 2, 300, 2000)):
        p = Problem(B, H, Sq, Sk)
        out, lse = Guarded((B, Sq, H, DV), torch.bfloat16), Guarded((B, H, Sq), torch.float32)
        ws = Guarded((max(16, lib.cross_attention_workspace_size(B, H, Sq, Sk)),), torch.uint8)
        p.run(lib, out=out.t, lse=lse.t, workspace=ws.t)
        lib.check_device_error()
        assert out.intact() and lse.intact() and ws.intact()
        p.check(out.t, lse.t)


def test_offsets_past_32_bits(lib):
    # 2.3e9 elements of keys and of values; only the first and the last keys have weight
    H, Sk = 128, 140000
    g = torch.Generator(device="cuda").manual_seed(3)
    kn = torch.zeros(1, Sk, H, DN, device="cuda", dtype=torch.bfloat16)
    v, kr = torch.zeros_like(kn), torch.zeros(1, Sk, DR, device="cuda", dtype=torch.bfloat16)
    qn, qr = torch.ones(1, 2, H, DN, device="cuda").bfloat16(), torch.zeros(1, 2, H, DR, device="cuda").bfloat16()
    at = torch.tensor([0, 1, Sk - 2, Sk - 1], device="cuda")
    kn[:, at] = 4.0 + randn(g, 1, 4, H, DN)
    v[:, at] = randn(g, 1, 4, H, DV)
    out, lse = lib.mla_cross_attention(qn, qr, kn, kr, v, softmax_scale=SCALE)
    small, small_lse = lib.mla_cross_attention(qn, qr, kn[:, at].contiguous(), kr[:, at].contiguous(),
                                               v[:, at].contiguous(), softmax_scale=SCALE)
    lib.check_device_error()
    assert (out.float() - small.float()).abs().max() < 0.06 and (lse - small_lse).abs().max() < 1e-4
    assert small.float().abs().max() > 0.5


def test_refusals_on_the_device(lib):
    p = Problem(2, 2, 4, 3000)
    size = lib.cross_attention_workspace_size(2, 2, 4, 3000)
    assert size > 0
    with pytest.raises(lib.MLAError, match="WORKSPACE"):
        p.run(lib, workspace=torch.empty(size - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        lib.mla_cross_attention(p.qn.transpose(1, 2).contiguous().transpose(1, 2), *p.args()[1:], softmax_scale=SCALE)
    with pytest.raises(ValueError, match="key_lens"):
        lib.mla_cross_attention(*p.args()[:5], torch.zeros(3, dtype=torch.int32, device="cuda"), softmax_scale=SCALE)
    with pytest.raises(TypeError, match="key_lens"):
        lib.mla_cross_attention(*p.args()[:5], torch.zeros(2, dtype=torch.int64, device="cuda"), softmax_scale=SCALE)
    with pytest.raises(ValueError, match="k_rope"):
        lib.mla_cross_attention(p.qn, p.qr, p.kn, p.kr[:, 1:].contiguous(), p.v, softmax_scale=SCALE)
    with pytest.raises(lib.MLAError, match="INVALID_ARG"):
        lib.mla_cross_attention(*p.args(), softmax_scale=0.0)
