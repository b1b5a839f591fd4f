"""GPU parity of mla_qk_norm_rope and its backward (through the C ABI) against the fp64 oracle.

Tolerances, element by element, from the arithmetic (fp32 inside, one rounding at the end):
  - bf16 outputs are rounded once: 2^-8 |y|.
  - a norm's sum of squares has at most 7 + 4 fp32 additions in a chain, then rsqrt (2 ulp), two
    products: below 2^-19 relative.  An angle is off by 2^-24 of half a turn (its fraction of a turn
    in fp32) and the fast sine and cosine of an angle in [-pi, pi] by 2^-21: together below 2^-19; so a
    rotated value is off by less than 2^-18 (|a| + |b|) of its pair (a, b).
  - dx = r (w g - x r^2 mean(x w g)): every factor to 2^-19, so 2^-17 r (|w g| + |x| r^2 mean |x w g|),
    with g, where it was turned back, off by 2^-18 (|g_a| + |g_b|) itself.
  - dw: a lane adds at most a few tens of terms in a row before the joins over lanes, warps and
    blocks (under 64 roundings here), each term to 2^-18: 2^-17 of the sum of |terms|.
"""
import numpy as np
import pytest
import torch

from oracle import norm_rope_ref as ref

pytestmark = pytest.mark.gpu

DN, DR = 128, 64
FREQ = 10000.0 ** (-np.arange(0, DR, 2) / DR)
EPS = 1e-6


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def randn(gen, *shape, mag=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * mag).to(dtype)


class Problem:
    def __init__(self, B, S, H, seed, norm=(1, 1, 1, 1), parts="qkr", views=False, far=5000, mag=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.S, self.H = B, S, H
        self.q = self.kn = self.kr = None
        if "q" in parts:
            self.q = randn(g, B, S, H, DN + DR, mag=mag)
        if "k" in parts:
            self.kn = randn(g, B, S, H, 2 * DN, mag=mag)[..., :DN] if views else randn(g, B, S, H, DN, mag=mag)
        if "r" in parts:
            self.kr = randn(g, B, S, 576, mag=mag)[..., 512:] if views else randn(g, B, S, DR, mag=mag)
        if views and self.q is not None:  # head-major projection output
            self.q = self.q.reshape(B * S, H, DN + DR).transpose(0, 1).contiguous().transpose(0, 1)
            self.q = self.q.unflatten(0, (B, S))
        self.pos = torch.randint(-far, far, (B, S), generator=g, device="cuda", dtype=torch.int32)
        have = (self.q, self.q, self.kn, self.kr)
        self.w = [1 + 0.3 * randn(g, d) if n and h is not None else None
                  for n, d, h in zip(norm, (DN, DR, DN, DR), have)]
        self.up = [None if h is None else randn(g, *s, dtype=dt) for h, s, dt in zip(
            have, ((B, S, H, DN), (B, S, H, DR), (B, S, H, DN), (B, S, DR)),
            (torch.bfloat16,) * 3 + (torch.float32,))]

    def kw(self, lib, interleaved):
        return dict(positions=self.pos, rope_turns=lib.rope_turns(FREQ, "cuda"), q_nope_weight=self.w[0],
                    q_rope_weight=self.w[1], k_nope_weight=self.w[2], k_rope_weight=self.w[3], eps=EPS,
                    interleaved=interleaved)

    def host(self):
        return (f64(self.q), f64(self.kn), f64(self.kr), f64(self.pos), FREQ, [f64(w) for w in self.w], EPS)


def pair_sum(x, interleaved):
    """|a| + |b| of the pair each element belongs to."""
    a = np.abs(x)
    if interleaved:
        s = a[..., 0::2] + a[..., 1::2]
        return np.repeat(s, 2, axis=-1)
    s = a[..., :DR // 2] + a[..., DR // 2:]
    return np.concatenate([s, s], axis=-1)


def check_forward(p, got, interleaved):
    want = ref.qk_norm_rope(*p.host(), interleaved)
    for name, g, w in zip(("q_nope", "q_rope", "k_nope", "k_rope"), got, want):
        if w is None:
            assert g is None
            continue
        fine = 2.0 ** -18 * (pair_sum(w, interleaved) if name.endswith("rope") else np.abs(w))
        err = np.abs(f64(g) - w)
        assert g.shape == w.shape and np.isfinite(f64(g)).all()
        assert (err <= 2.0 ** -8 * np.abs(w) + 1.01 * fine).all(), (name, (err - 2.0 ** -8 * np.abs(w)).max())


def norm_terms(x, w, g, g_err):
    """(bound of dx before its rounding, sum of |terms| of dw) of one normalised part."""
    if w is None:
        return g_err, None
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS)
    ag = np.abs(g)
    mag = r * (np.abs(w) * ag + np.abs(x) * r * r * np.mean(np.abs(x * w) * ag, -1, keepdims=True))
    prop = r * (np.abs(w) * g_err + np.abs(x) * r * r * np.mean(np.abs(x * w) * g_err, -1, keepdims=True))
    terms = (np.abs(x * r) * ag).reshape(-1, x.shape[-1]).sum(0)
    return 2.0 ** -17 * mag + prop, terms


def check_backward(p, got, interleaved):
    q, kn, kr, pos, freq, w, eps = p.host()
    up = [f64(u) for u in p.up]
    want = ref.qk_norm_rope_backward(*up, *p.host(), interleaved)
    bound = [None] * 7

    def turned(g, at):
        back = ref.rotate(g, -at, freq, interleaved)
        return back, 2.0 ** -18 * pair_sum(g, interleaved)

    if q is not None:
        a, bound[3] = norm_terms(q[..., :DN], w[0], up[0], 0 * up[0])
        b, bound[4] = norm_terms(q[..., DN:], w[1], *turned(up[1], pos[..., None]))
        bound[0] = np.concatenate([a, b], -1)
    if kn is not None:
        bound[1], bound[5] = norm_terms(kn, w[2], up[2], 0 * up[2])
    if kr is not None:
        bound[2], bound[6] = norm_terms(kr, w[3], *turned(up[3], pos))
    for i, (g, x, e) in enumerate(zip(got, want, bound)):
        if x is None:
            assert g is None
            continue
        err = np.abs(f64(g) - x)
        tol = 2.0 ** -8 * np.abs(x) + 1.01 * e if i < 3 else 2.0 ** -17 * e
        assert np.isfinite(f64(g)).all() and (err <= tol).all(), (i, (err - tol).max())


def backward(lib, p, interleaved, **kw):
    return lib.mla_qk_norm_rope_backward(*p.up, p.q, p.kn, p.kr, **p.kw(lib, interleaved), **kw)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,S,H", [(1, 1, 1), (3, 1, 16), (1, 65, 4), (2, 9, 5), (1, 7, 128), (5, 3, 2), (1, 300, 3)])
def test_shapes(lib, B, S, H, interleaved):
    p = Problem(B, S, H, seed=B * 100 + S + H)
    got = lib.mla_qk_norm_rope(p.q, p.kn, p.kr, **p.kw(lib, interleaved))
    grads = backward(lib, p, interleaved)
    lib.check_device_error()
    check_forward(p, got, interleaved)
    check_backward(p, grads, interleaved)


@pytest.mark.parametrize("parts,norm", [("q", (1, 1, 0, 0)), ("k", (0, 0, 1, 0)), ("r", (0, 0, 0, 1)),
                                        ("qkr", (0, 0, 0, 0)), ("qkr", (1, 0, 0, 1)), ("kr", (0, 0, 0, 1)),
                                        ("qr", (0, 1, 0, 0))])
def test_parts_and_absent_weights(lib, parts, norm):
    p = Problem(2, 17, 6, seed=7, norm=norm, parts=parts)
    got = lib.mla_qk_norm_rope(p.q, p.kn, p.kr, **p.kw(lib, True))
    grads = backward(lib, p, True)
    lib.check_device_error()
    check_forward(p, got, True)
    check_backward(p, grads, True)
    for y, x, w in ((got[0], None if p.q is None else p.q[..., :DN], p.w[0]), (got[2], p.kn, p.w[2])):
        if x is not None and w is None:
            assert torch.equal(y, x)  # without a norm the nope part is a copy


@pytest.mark.parametrize("interleaved", [False, True])
def test_strided_operands_and_gradients_in_views(lib, interleaved):
    p = Problem(2, 21, 6, seed=8, views=True)
    assert not p.q.is_contiguous() and not p.kn.is_contiguous() and not p.kr.is_contiguous()
    got = lib.mla_qk_norm_rope(p.q, p.kn, p.kr, **p.kw(lib, interleaved))
    # gradients land in views of joint buffers; what lies between is not touched
    dkv = torch.full((2, 21, 6, 2 * DN), 7.0, device="cuda", dtype=torch.bfloat16)
    dc = torch.full((2, 21, 576), 7.0, device="cuda", dtype=torch.bfloat16)
    grads = [torch.empty_strided(p.q.shape, p.q.stride(), device="cuda", dtype=torch.bfloat16), dkv[..., :DN],
             dc[..., 512:]] + [torch.empty(w.shape, device="cuda") for w in p.w]
    back = backward(lib, p, interleaved, grads=grads)
    lib.check_device_error()
    check_forward(p, got, interleaved)
    check_backward(p, back, interleaved)
    assert (dkv[..., DN:] == 7).all() and (dc[..., :512] == 7).all()
    with pytest.raises(ValueError, match="strides"):
        backward(lib, p, interleaved, grads=[grads[0], torch.empty_like(dkv[..., :DN].contiguous())] + grads[2:])


def test_repeated_operand_forward_and_its_refused_gradient(lib):
    p = Problem(1, 5, 8, seed=9)
    p.kn = p.kn[:, :, :1].expand(1, 5, 8, DN)  # one head for all
    check_forward(p, lib.mla_qk_norm_rope(p.q, p.kn, p.kr, **p.kw(lib, True)), True)
    with pytest.raises(lib.MLAError, match="INVALID_ARG"):
        backward(lib, p, True)


def test_far_positions_of_both_signs(lib):
    p = Problem(1, 64, 2, seed=10, norm=(0, 0, 0, 0))
    p.pos = torch.tensor([[2 ** 31 - 1 - i if i % 2 else -2 ** 31 + i for i in range(64)]], dtype=torch.int32,
                         device="cuda")
    # fp64 angles of positions near 2^31 are good to 2^31 * 2^-53 * 4 radians (2^-20): use exact
    # phases in turns for the reference instead
    turns = [int(t) % 2 ** 64 for t in lib.rope_turns(FREQ).tolist()]
    for i in range(64):
        ang = np.array([2 * np.pi * ((int(p.pos[0, i]) * t) % 2 ** 64) / 2.0 ** 64 for t in turns])
        y = ref.rotate(f64(p.kr)[0, i], 1.0, ang, True)
        got = f64(lib.mla_qk_norm_rope(None, None, p.kr, **p.kw(lib, True))[3])[0, i]
        assert (np.abs(got - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -18 * pair_sum(y, True)).all()


@pytest.mark.parametrize("mag", [0.0, 1e-20, 1e15])
def test_magnitudes_and_zero_rows(lib, mag):
    # mean(x^2) of 1e15 is 1e30, within fp32; rows of zeros give zeros, and their gradient is finite
    p = Problem(1, 6, 3, seed=11, mag=mag)
    check_forward(p, lib.mla_qk_norm_rope(p.q, p.kn, p.kr, **p.kw(lib, False)), False)
    check_backward(p, backward(lib, p, False), False)


def test_non_finite_values_stay_in_their_row_and_head(lib):
    p = Problem(1, 8, 6, seed=12)
    clean = lib.mla_qk_norm_rope(p.q, p.kn, p.kr, **p.kw(lib, True))
    p.q[0, 3, 2, 5] = float("nan")
    p.kn[0, 1, 4, 0] = float("inf")
    p.kr[0, 6, 9] = float("nan")
    got = lib.mla_qk_norm_rope(p.q, p.kn, p.kr, **p.kw(lib, True))
    for y, c, at in ((got[0], clean[0], (0, 3, 2)), (got[2], clean[2], (0, 1, 4)), (got[3], clean[3], (0, 6))):
        assert not torch.isfinite(y[at]).all()
        y, c = y.clone(), c.clone()
        y[at] = c[at] = 0
        assert torch.equal(y, c)
    assert torch.equal(got[1], clean[1])


def test_gradient_sums_over_many_rows_repeat_exactly(lib):
    p = Problem(2, 700, 24, seed=13)
    a, b = backward(lib, p, True), backward(lib, p, True)
    lib.check_device_error()
    check_backward(p, a, True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_gradient_against_differences_of_the_forward(lib):
    # fp32 master values stepped by h and rounded to bf16: the step the kernel sees is exact
    p = Problem(1, 2, 2, seed=14)
    grads = [f64(g) for g in backward(lib, p, False)]
    host = p.host()

    def loss(q):
        y = ref.qk_norm_rope(q, *host[1:], False)
        return sum((a * f64(u)).sum() for a, u in zip(y, p.up))

    rng = np.random.default_rng(0)
    for _ in range(40):
        at = tuple(rng.integers(0, n) for n in p.q.shape)
        up, dn = host[0].copy(), host[0].copy()
        up[at] += 1e-4
        dn[at] -= 1e-4
        d = (loss(up) - loss(dn)) / 2e-4
        # bf16 rounding of the gradient, 1e-8 h^2-truncation scale and the sum's 2^-17 part
        assert abs(d - grads[0][at]) <= 2.0 ** -8 * abs(d) + 1e-4


def test_captured_and_replayed_with_new_inputs(lib):
    p, p2 = Problem(2, 33, 5, seed=15), Problem(2, 33, 5, seed=16)
    p.w = p2.w
    kw = p.kw(lib, True)
    ws = torch.empty(lib.qk_norm_rope_backward_workspace_size(66, 5), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lib.mla_qk_norm_rope(p.q, p.kn, p.kr, **kw)
        lib.mla_qk_norm_rope_backward(*p.up, p.q, p.kn, p.kr, **kw, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lib.mla_qk_norm_rope(p.q, p.kn, p.kr, **kw)
        grads = lib.mla_qk_norm_rope_backward(*p.up, p.q, p.kn, p.kr, **kw, workspace=ws)
    for a, b in zip([p.q, p.kn, p.kr, p.pos] + p.up, [p2.q, p2.kn, p2.kr, p2.pos] + p2.up):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    check_forward(p2, got, True)
    check_backward(p2, grads, True)


def test_on_a_side_stream_with_its_own_allocations(lib):
    p = Problem(1, 400, 16, seed=17)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    runs = [backward(lib, p, True, stream=side) for _ in range(4)]  # workspaces freed between the calls
    fwd = lib.mla_qk_norm_rope(p.q, p.kn, p.kr, **p.kw(lib, True), stream=side)
    side.synchronize()
    check_forward(p, fwd, True)
    for g in runs:
        check_backward(p, g, True)


def test_writes_only_its_outputs_and_workspace(lib):
    from tests.test_gpu_canaries import Guarded

    B, S, H = 2, 31, 7
    p = Problem(B, S, H, seed=18)
    outs = [Guarded(s, torch.bfloat16) for s in ((B, S, H, DN), (B, S, H, DR), (B, S, H, DN), (B, S, DR))]
    lib.mla_qk_norm_rope(p.q, p.kn, p.kr, **p.kw(lib, True), out=[o.t for o in outs])
    grads = [Guarded(t.shape, torch.bfloat16) for t in (p.q, p.kn, p.kr)]
    grads += [Guarded(w.shape, torch.float32) for w in p.w]
    ws = Guarded((lib.qk_norm_rope_backward_workspace_size(B * S, H),), torch.uint8)
    backward(lib, p, True, grads=[g.t for g in grads], workspace=ws.t)
    lib.check_device_error()
    assert all(o.intact() for o in outs + grads + [ws])
    check_forward(p, [o.t for o in outs], True)
    check_backward(p, [g.t for g in grads], True)


def test_offsets_past_32_bits(lib):
    # 90112 tokens x 128 heads x 192: q alone has 2.2e9 elements; checked at both ends
    S, H = 90112, 128
    g = torch.Generator(device="cuda").manual_seed(19)
    q = torch.zeros(1, S, H, DN + DR, device="cuda", dtype=torch.bfloat16)
    q[:, :3] = randn(g, 1, 3, H, DN + DR)
    q[:, -3:] = randn(g, 1, 3, H, DN + DR)
    pos = torch.arange(S, device="cuda", dtype=torch.int32)[None]
    kw = dict(rope_turns=lib.rope_turns(FREQ, "cuda"), q_nope_weight=torch.ones(DN, device="cuda").bfloat16())
    qn, qr, _, _ = lib.mla_qk_norm_rope(q, positions=pos, **kw)
    lib.check_device_error()
    for cut in (slice(0, 3), slice(S - 3, S)):
        a, b, _, _ = lib.mla_qk_norm_rope(q[:, cut].contiguous(), positions=pos[:, cut].contiguous(), **kw)
        assert torch.equal(a, qn[:, cut]) and torch.equal(b, qr[:, cut]) and bool(a.any())
