"""GPU parity of the calls with positions on several axes (head norms, their gradient, the cache append)
against the fp64 oracle, with the tolerances of the one-axis calls (tests/test_gpu_norm_rope.py,
tests/test_gpu_rope_append.py): a phase is an exact integer sum, so nothing is added to them.

A weight's gradient of a rope part sums g x r where g, the upstream gradient turned back, is off by
2^-18 (|a| + |b|) of its pair, which can exceed any share of |g| itself where a and b nearly cancel: the sum of
|x r| times that error is added to 2^-17 of the sum of |terms|, once more than it can be off (1.01)."""
import numpy as np
import pytest
import torch

from oracle import norm_rope_ref as ref
from tests import test_gpu_norm_rope as one
from tests import test_gpu_rope_append as append
from tests.test_gpu_norm_rope import DN, DR, EPS, FREQ, f64, norm_terms, pair_sum, randn

pytestmark = pytest.mark.gpu

SECTIONS = {1: [0] * 32, 2: [0] * 16 + [1] * 16, 3: [0] * 8 + [1] * 12 + [2] * 12, 4: [i % 4 for i in range(32)]}


def table_of(axes):
    return np.where(np.array(SECTIONS[axes]) == np.arange(axes)[:, None], FREQ, 0.0)


class Problem(one.Problem):
    def __init__(self, B, S, H, axes, seed, dkr=torch.float32, far=5000, **kw):
        super().__init__(B, S, H, seed, far=far, **kw)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.axes = axes
        self.pos = torch.randint(-far, far, (B, S, axes), generator=g, device="cuda", dtype=torch.int32)
        if self.up[3] is not None:
            self.up[3] = self.up[3].to(dkr)

    def kw(self, lib, interleaved):
        return dict(super().kw(lib, interleaved), rope_turns=lib.rope_turns_axes(FREQ, SECTIONS[self.axes], "cuda"))

    def host(self):
        h = super().host()
        return h[:4] + (table_of(self.axes),) + h[5:]


def forward(lib, p, interleaved, **kw):
    return lib.mla_qk_norm_rope_axes(p.q, p.kn, p.kr, **p.kw(lib, interleaved), **kw)


def backward(lib, p, interleaved, **kw):
    return lib.mla_qk_norm_rope_axes_backward(*p.up, p.q, p.kn, p.kr, **p.kw(lib, interleaved), **kw)


def rope_terms(x, w, g, g_err):
    """norm_terms with the error of g in the weight's sum, in units of that sum's 2^-17."""
    dx, terms = norm_terms(x, w, g, g_err)
    if terms is not None:
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS)
        terms = terms + 1.01 * 2.0 ** 17 * (np.abs(x * r) * g_err).reshape(-1, x.shape[-1]).sum(0)
    return dx, terms


def check_backward(p, got, interleaved):
    """As the one-axis check, with the positions of several axes."""
    q, kn, kr, pos, freq, w, _ = p.host()
    up = [f64(u) for u in p.up]
    want = ref.qk_norm_rope_backward(*up, *p.host(), interleaved)
    bound = [None] * 7
    if q is not None:
        a, bound[3] = norm_terms(q[..., :DN], w[0], up[0], 0 * up[0])
        back = ref.rotate(up[1], -ref.for_heads(pos, freq), freq, interleaved)
        b, bound[4] = rope_terms(q[..., DN:], w[1], back, 2.0 ** -18 * pair_sum(up[1], interleaved))
        bound[0] = np.concatenate([a, b], -1)
    if kn is not None:
        bound[1], bound[5] = norm_terms(kn, w[2], up[2], 0 * up[2])
    if kr is not None:
        back = ref.rotate(up[3], -pos, freq, interleaved)
        bound[2], bound[6] = rope_terms(kr, w[3], back, 2.0 ** -18 * pair_sum(up[3], interleaved))
    for i, (g, x, e) in enumerate(zip(got, want, bound)):
        if x is None:
            assert g is None
            continue
        err = np.abs(f64(g) - x)
        tol = 2.0 ** -8 * np.abs(x) + 1.01 * e if i < 3 else 2.0 ** -17 * e
        assert np.isfinite(f64(g)).all() and (err <= tol).all(), (i, (err - tol).max())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("B,S,H", [(1, 1, 1), (3, 1, 16), (2, 9, 5), (1, 65, 8), (1, 7, 128), (1, 300, 3)])
def test_shapes(lib, B, S, H, axes, interleaved):
    p = Problem(B, S, H, axes, seed=B * 100 + S + H + axes, dkr=torch.bfloat16 if axes % 2 else torch.float32)
    got, grads = forward(lib, p, interleaved), backward(lib, p, interleaved)
    lib.check_device_error()
    one.check_forward(p, got, interleaved)
    check_backward(p, grads, interleaved)


@pytest.mark.parametrize("parts,norm", [("q", (1, 1, 0, 0)), ("k", (0, 0, 1, 0)), ("r", (0, 0, 0, 1)),
                                        ("qkr", (0, 0, 0, 0)), ("kr", (0, 0, 0, 1))])
def test_parts_and_absent_weights(lib, parts, norm):
    p = Problem(2, 17, 6, 3, seed=7, norm=norm, parts=parts, dkr=torch.bfloat16, views=True)
    got, grads = forward(lib, p, True), backward(lib, p, True)
    lib.check_device_error()
    one.check_forward(p, got, True)
    check_backward(p, grads, True)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [2, 3, 4])
def test_each_pair_as_one_axis_turns_it(lib, axes, interleaved):
    # the phase is the same integer, so the bits are the same; positions to both ends of int32
    p = Problem(2, 40, 9, axes, seed=20 + axes)
    p.pos[0, :4] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 0], device="cuda", dtype=torch.int32)[:, None]
    _, qr, _, kr = forward(lib, p, interleaved)
    kw = dict(p.kw(lib, interleaved), rope_turns=lib.rope_turns(FREQ, "cuda"))
    for a in range(axes):
        kw["positions"] = p.pos[..., a].contiguous()
        _, qa, _, ka = lib.mla_qk_norm_rope(p.q, p.kn, p.kr, **kw)
        pick = torch.tensor(SECTIONS[axes], device="cuda") == a
        pick = pick.repeat_interleave(2) if interleaved else pick.repeat(2)
        assert torch.equal(qr[..., pick], qa[..., pick]) and torch.equal(kr[..., pick], ka[..., pick])


def test_a_pair_that_two_axes_turn(lib):
    # a general table: the angles of both axes add up
    p = Problem(1, 33, 4, 2, seed=30, norm=(0, 0, 0, 0))
    turns = torch.stack([lib.rope_turns(FREQ, "cuda"), lib.rope_turns(-0.5 * FREQ, "cuda")])
    got = lib.mla_qk_norm_rope_axes(None, None, p.kr, positions=p.pos, rope_turns=turns)[3]
    want = ref.rotate(f64(p.kr), f64(p.pos), np.stack([FREQ, -0.5 * FREQ]), True)
    assert (np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * pair_sum(want, True)).all()


def test_gradient_of_the_rope_key_in_either_type(lib):
    p = Problem(2, 50, 4, 3, seed=31, dkr=torch.bfloat16)
    a = backward(lib, p, False)
    p.up[3] = p.up[3].float()
    assert all(torch.equal(x, y) for x, y in zip(a, backward(lib, p, False)))


def test_repeats_exactly_captured_on_a_side_stream(lib):
    p, p2 = Problem(2, 130, 12, 3, seed=32), Problem(2, 130, 12, 3, seed=33)
    p.w = p2.w
    kw = p.kw(lib, True)
    ws = torch.empty(lib.qk_norm_rope_backward_workspace_size(260, 12), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = lib.mla_qk_norm_rope_axes_backward(*p.up, p.q, p.kn, p.kr, **kw, workspace=ws, stream=side)
    side.synchronize()
    check_backward(p, first, True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lib.mla_qk_norm_rope_axes(p.q, p.kn, p.kr, **kw)
        grads = lib.mla_qk_norm_rope_axes_backward(*p.up, p.q, p.kn, p.kr, **kw, workspace=ws)
    for a, b in zip([p.q, p.kn, p.kr, p.pos] + p.up, [p2.q, p2.kn, p2.kr, p2.pos] + p2.up):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    one.check_forward(p2, got, True)
    check_backward(p2, grads, True)
    again = [g.clone() for g in grads]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, grads))


def test_refuses_tables_and_positions_of_other_shapes(lib):
    p = Problem(1, 4, 2, 3, seed=34)
    kw = p.kw(lib, True)
    for bad in (dict(positions=p.pos[..., :2].contiguous()), dict(positions=p.pos[..., 0].contiguous()),
                dict(rope_turns=kw["rope_turns"][:2].contiguous()), dict(positions=p.pos.transpose(0, 1))):
        with pytest.raises(ValueError):
            lib.mla_qk_norm_rope_axes(p.q, p.kn, p.kr, **dict(kw, **bad))
    with pytest.raises(TypeError):
        lib.mla_qk_norm_rope_axes(p.q, p.kn, p.kr, **dict(kw, positions=p.pos.long()))
    five = torch.zeros(5, 32, dtype=torch.int64, device="cuda")
    with pytest.raises(lib.MLAError, match="UNSUPPORTED"):
        lib.mla_qk_norm_rope_axes(p.q, p.kn, p.kr, **dict(kw, rope_turns=five, positions=torch.zeros(
            1, 4, 5, dtype=torch.int32, device="cuda")))


# ------------------------------------------------------------------------------- the append

class Append(append.Problem):
    def __init__(self, lens, T, fp8, axes, seed, **kw):
        super().__init__(lens, T, fp8, seed, **kw)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.axes = axes
        self.pos = torch.randint(-9000, 9000, (self.B, T, axes), generator=g, device="cuda", dtype=torch.int32)

    def run(self, lib, interleaved, **kw):
        self.before = self.cache.clone(), None if self.scale is None else self.scale.clone()
        lib.mla_rope_append_axes(self.c, self.cache, self.pt, self.lens, kv_scale=self.scale, positions=self.pos,
                                 rope_turns=lib.rope_turns_axes(FREQ, SECTIONS[self.axes], "cuda"), norm_weight=self.w,
                                 eps=EPS, new_lens=self.new, interleaved=interleaved, **kw)

    def check(self, interleaved, monkeypatch):
        with monkeypatch.context() as m:
            m.setattr(append, "FREQ", table_of(self.axes))
            super().check(interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,axes", [(1, 3), (2, 1), (5, 2), (67, 4)])
def test_append_page_edges(lib, fp8, T, axes, interleaved, monkeypatch):
    p = Append([1, 2, 63, 64, 65, 127, 128, 129, 3000], T, fp8, axes, seed=51 + T)
    p.run(lib, interleaved)
    lib.check_device_error()
    p.check(interleaved, monkeypatch)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_ragged_strided_without_norm(lib, fp8, monkeypatch):
    p = Append([70, 70, 2, 0, 129, 64], 6, fp8, 3, seed=61, new=[6, 1, 4, 0, 3, 0], wide=True, norm=False)
    p.run(lib, False)
    lib.check_device_error()
    p.check(False, monkeypatch)


def test_append_reports_bad_pages_and_counts(lib, monkeypatch):
    p = Append([70, 70, 90], 3, True, 3, seed=62, new=[-5, 4, 2])
    p.run(lib, True)
    with pytest.raises(lib.MLAError, match="DEVICE_CHECK"):
        lib.check_device_error()
    p.check(True, monkeypatch)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_with_equal_axes_is_the_one_axis_append(lib, fp8):
    p = Append([65, 300, 2, 130], 2, fp8, 3, seed=63)
    p.pos = p.pos[..., :1].expand(-1, -1, 3).contiguous()
    other, scale = p.cache.clone(), None if p.scale is None else p.scale.clone()
    lib.mla_rope_append(p.c, other, p.pt, p.lens, kv_scale=scale, rope_turns=lib.rope_turns(FREQ, "cuda"),
                        norm_weight=p.w, eps=EPS, positions=p.pos[..., 0].contiguous())
    p.run(lib, True)
    lib.check_device_error()
    assert torch.equal(p.cache.view(torch.uint8), other.view(torch.uint8))
    assert scale is None or torch.equal(p.scale.view(torch.int32), scale.view(torch.int32))
