"""The operators that attend to an encoder's states together, as a program uses them: a training step with
cross attention from text to images whose patches sit on three axes, and a decode step of text behind image
tokens in the latent cache that also attends to encoder states kept for it; each against one fp64 computation
of the whole, with the tolerances of tests/test_gpu_draft_step.py (2-norm, relative)."""
import pytest
import torch

from tests.test_gpu_draft_step import EPS, FREQ, SCALE, far, rms

pytestmark = pytest.mark.gpu

AXES = [0] * 8 + [1] * 12 + [2] * 12


def turn(x, pos):
    """x [.., 64], halves rotated; pos [.., 3] broadcast over what lies between."""
    axis = torch.tensor(AXES, device=x.device)
    ang = pos.double().index_select(-1, axis) * FREQ.to(x.device)
    while ang.dim() < x.dim():
        ang = ang.unsqueeze(-2)
    a, b = x.split(32, -1)
    return torch.cat((a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()), -1)


def patches(S, width, first):
    """Positions [S, 3] of an image's patches, row by row, from `first` on."""
    k = torch.arange(S, device="cuda")
    return (torch.stack((0 * k, k // width, k % width), -1) + first).to(torch.int32)


def text(S, first):
    return (torch.arange(S, device="cuda") + first)[:, None].expand(S, 3).to(torch.int32)


def test_training_step(lib):
    B, Sq, Sk, H = 2, 150, 330, 4
    lens = torch.tensor([330, 211], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, kv, kr, d_out = rnd(B, Sq, H, 192), rnd(B, Sk, H, 256), rnd(B, Sk, 64), rnd(B, Sq, H, 128)
    w = [1 + 0.2 * rnd(d) for d in (128, 64, 128, 64)]
    pos_q = torch.stack([text(Sq, 20), text(Sq, 7)]).contiguous()
    pos_k = torch.stack([patches(Sk, 22, 3), patches(Sk, 15, 0)]).contiguous()
    turns = lib.rope_turns_axes(FREQ, AXES, "cuda")
    kq = dict(positions=pos_q, rope_turns=turns, q_nope_weight=w[0], q_rope_weight=w[1], eps=EPS, interleaved=False)
    kk = dict(positions=pos_k, rope_turns=turns, k_nope_weight=w[2], k_rope_weight=w[3], eps=EPS, interleaved=False)
    v = kv[..., 128:].contiguous()
    qn, qr, _, _ = lib.mla_qk_norm_rope_axes(q, **kq)
    _, _, kn, kro = lib.mla_qk_norm_rope_axes(None, kv[..., :128], kr, **kk)
    out, lse = lib.mla_cross_attention(qn, qr, kn, kro, v, lens, softmax_scale=SCALE)
    dqn, dqr, dkn, dkr, dv = lib.mla_cross_attention_backward(qn, qr, kn, kro, v, out, lse, d_out, lens, softmax_scale=SCALE)
    gq = lib.mla_qk_norm_rope_axes_backward(dqn, dqr, None, None, q, **kq)
    dkv = torch.empty_like(kv)
    dkv[..., 128:] = dv
    gk = [None, dkv[..., :128], torch.empty_like(kr), None, None] + [torch.empty(x.shape, device="cuda") for x in w[2:]]
    lib.mla_qk_norm_rope_axes_backward(None, None, dkn, dkr, None, kv[..., :128], kr, **kk, grads=gk)
    lib.check_device_error()

    leaf = [t.double().requires_grad_() for t in (q, kv, kr, *w)]
    Q, KV, KR, w0, w1, w2, w3 = leaf
    qq = torch.cat((rms(Q[..., :128], w0), turn(rms(Q[..., 128:], w1), pos_q)), -1)
    keys = torch.cat((rms(KV[..., :128], w2), turn(rms(KR, w3), pos_k)[:, :, None].expand(B, Sk, H, 64)), -1)
    s = torch.einsum("bihd,bjhd->bhij", qq, keys) * SCALE
    s = s.masked_fill(torch.arange(Sk, device="cuda") >= lens[:, None, None, None], -float("inf"))
    o = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), KV[..., 128:])
    want = torch.autograd.grad((o * d_out.double()).sum(), leaf)
    assert far(out, o.detach()) < 2.0 ** -6
    for got, ref in zip([gq[0], dkv, gk[2], gq[3], gq[4], gk[5], gk[6]], want):
        assert far(got, ref) < 2.0 ** -6, got.shape
    assert not bool(dkv[1, 211:].any()) and not bool(gk[2][1, 211:].any())


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_step_behind_image_tokens(lib, fp8):
    # an image's tokens and some text into the latent cache, one new text token decoded over them, whose
    # attention to encoder states kept for the sequence (none for the last one) follows
    H, B, images, words = 8, 3, [200, 77, 131], [5, 60, 1]
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    turns = lib.rope_turns_axes(FREQ, AXES, "cuda")
    pages = torch.randperm(18, generator=g, device="cuda")[:15].to(torch.int32).view(B, 5)
    cache = torch.full((18, 64, 576), float("nan"), device="cuda", dtype=torch.bfloat16)
    kv_scale = None
    if fp8:
        cache, kv_scale = cache.to(torch.float8_e4m3fn), torch.full((18, 64), float("nan"), device="cuda")
    w_lat, w_uk, w_uv = 1 + 0.2 * rnd(512), rnd(H, 128, 512) / 12, rnd(H, 512, 128) / 22
    qw = 1 + 0.2 * rnd(128), 1 + 0.2 * rnd(64)
    lens = [a + b for a, b in zip(images, words)]
    raw = rnd(B, max(lens), 576)
    # the text counts on from the image's largest row or column
    pos = torch.zeros(B, max(lens), 3, dtype=torch.int32, device="cuda")
    for b in range(B):
        pos[b, :images[b]] = patches(images[b], 14, 0)
        pos[b, images[b]:lens[b]] = text(words[b], 14)
    q = rnd(B, 1, H, 192)
    pos_q = torch.stack([pos[b, lens[b] - 1] for b in range(B)])[:, None].contiguous()

    lib.mla_rope_append_axes(raw, cache, pages, i32(lens), kv_scale=kv_scale, rope_turns=turns, positions=pos,
                             norm_weight=w_lat, eps=EPS, new_lens=i32(lens), interleaved=False)
    qn, qr, _, _ = lib.mla_qk_norm_rope_axes(q, positions=pos_q, rope_turns=turns, q_nope_weight=qw[0],
                                             q_rope_weight=qw[1], eps=EPS, interleaved=False)
    ql = lib.mla_absorb(qn.view(B, H, 128), w_uk).view(B, 1, H, 512)
    o, _ = lib.mla_decode(ql, qr, cache, pages, i32(lens), kv_scale=kv_scale, softmax_scale=SCALE)
    got = lib.mla_absorb(o.view(B, H, 512), w_uv).view(B, 1, H, 128)
    states, enc = [500, 33, 0], [rnd(B, 500, H, 128), rnd(B, 500, 64), rnd(B, 500, H, 128)]
    for b, n in enumerate(states):
        for t in enc:
            t[b, n:] = float("nan")
    seen, lse = lib.mla_cross_attention(qn, qr, *enc, i32(states), softmax_scale=SCALE)
    lib.check_device_error()

    tol = 2.0 ** -4 if fp8 else 2.0 ** -6
    for b, n in enumerate(lens):
        x = q[b, 0].double()
        a, r = rms(x[:, :128], qw[0].double()), turn(rms(x[:, 128:], qw[1].double()), pos_q[b, 0])
        lat, rope = rms(raw[b, :n, :512].double(), w_lat.double()), turn(raw[b, :n, 512:].double(), pos[b, :n])
        s = torch.einsum("hd,kl,hdl->hk", a, lat, w_uk.double()) + r @ rope.T
        want = torch.einsum("hk,kl,hld->hd", (s * SCALE).softmax(-1), lat, w_uv.double())
        assert far(got[b, 0], want) < tol, b
        if states[b] == 0:
            assert not bool(seen[b].any()) and bool(torch.isneginf(lse[b]).all())
            continue
        kn, kr, v = (t[b, :states[b]].double() for t in enc)
        s = (torch.einsum("hd,khd->hk", a, kn) + r @ kr.T) * SCALE
        assert far(seen[b, 0], torch.einsum("hk,khd->hd", s.softmax(-1), v)) < 2.0 ** -6, b
