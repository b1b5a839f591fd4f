"""The operators together, as a program uses them: a training step from projections to their
gradients, and a speculative decode step from raw rows to accepted tokens, each against one fp64
computation of the whole.

Tolerances are on the 2-norm of the error relative to the result's.  Operands are rounded to bf16 by
at most 2^-8 of a value, independently of one another: a score, softmax_scale times 192 products of
unit variance, is off by about 192^-1/2 x 192^1/2 x 2^1/2 x 2^-8 = 2^-7.5, a softmax weight relatively
by as much, and the values, the result and a product before or after it by 2^-8 each; together
below 2^-6.  With e4m3 rows (2^-4 of a value at most, 2^-5.8 in the 2-norm) below 2^-4.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

FREQ = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
SCALE = 192.0 ** -0.5
EPS = 1e-6


def rms(x, w):
    return x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w


def turn(x, pos):
    ang = pos.double()[..., None] * FREQ.to(x.device)
    while ang.dim() < x.dim():
        ang = ang.unsqueeze(-2)
    z = torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) * torch.polar(torch.ones_like(ang), ang)
    return torch.view_as_real(z).flatten(-2)


def far(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm())


def test_training_step(lib):
    B, S, H = 2, 200, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, kv, kr, d_out = rnd(B, S, H, 192), rnd(B, S, H, 256), rnd(B, S, 64), rnd(B, S, H, 128)
    w = [1 + 0.2 * rnd(d) for d in (128, 64, 128, 64)]
    pos = torch.arange(S, device="cuda", dtype=torch.int32).expand(B, S).contiguous()
    kw = dict(positions=pos, rope_turns=lib.rope_turns(FREQ, "cuda"), q_nope_weight=w[0], q_rope_weight=w[1],
              k_nope_weight=w[2], k_rope_weight=w[3], eps=EPS)
    v = kv[..., 128:].contiguous()
    ops = lib.mla_qk_norm_rope(q, kv[..., :128], kr, **kw)
    out, lse = lib.mla_prefill(*ops, v, softmax_scale=SCALE)
    dqn, dqr, dkn, dkr, dv = lib.mla_prefill_backward(*ops, v, out, lse, d_out, softmax_scale=SCALE)
    dkv = torch.empty_like(kv)
    dkv[..., 128:] = dv
    grads = [torch.empty_like(q), dkv[..., :128], torch.empty_like(kr)] + [torch.empty(x.shape, device="cuda") for x in w]
    lib.mla_qk_norm_rope_backward(dqn, dqr, dkn, dkr, q, kv[..., :128], kr, **kw, grads=grads)
    lib.check_device_error()

    leaf = [t.double().requires_grad_() for t in (q, kv, kr, *w)]
    Q, KV, KR, w0, w1, w2, w3 = leaf
    qq = torch.cat((rms(Q[..., :128], w0), turn(rms(Q[..., 128:], w1), pos)), -1)
    kk = torch.cat((rms(KV[..., :128], w2), turn(rms(KR, w3), pos)[:, :, None].expand(B, S, H, 64)), -1)
    s = torch.einsum("bihd,bjhd->bhij", qq, kk) * SCALE
    s = s.masked_fill(~torch.ones(S, S, dtype=torch.bool, device="cuda").tril(), -float("inf"))
    o = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), KV[..., 128:])
    want = torch.autograd.grad((o * d_out.double()).sum(), leaf)
    assert far(out, o.detach()) < 2.0 ** -6
    for got, ref in zip([grads[0], dkv, *grads[2:]], want):
        assert far(got, ref) < 2.0 ** -6, got.shape


@pytest.mark.parametrize("fp8", [False, True])
def test_speculative_decode_step(lib, fp8):
    # prompts written by the rotated append, a ragged tree drafted over them, the accepted path
    # appended again at its final places, and one more token decoded over it
    H, T = 8, 7
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    prompt, drafts = [61, 200, 5], [7, 4, 6]
    B, most = 3, max(prompt)
    parents = torch.tensor([[-1, 0, 0, 1, 1, 3, 2], [-1, -1, 0, 1, 0, 0, 0], [-1, 0, 1, 2, -1, 4, 0]])
    mask, depth = (t.cuda() for t in lib.tree_mask_from_parents(parents))
    pages = torch.randperm(16, generator=g, device="cuda")[:12].to(torch.int32).view(B, 4)
    cache = torch.full((16, 64, 576), float("nan"), device="cuda", dtype=torch.bfloat16)
    kv_scale = None
    if fp8:
        cache, kv_scale = cache.to(torch.float8_e4m3fn), torch.full((16, 64), float("nan"), device="cuda")
    w_lat, w_uk, w_uv = 1 + 0.2 * rnd(512), rnd(H, 128, 512) / 12, rnd(H, 512, 128) / 22
    qw = 1 + 0.2 * rnd(128), 1 + 0.2 * rnd(64)
    turns = lib.rope_turns(FREQ, "cuda")
    c_prompt, c_draft, q_draft = rnd(B, most, 576), rnd(B, T, 576), rnd(B, T, H, 192)
    c_last, q_last = rnd(B, 1, 576), rnd(B, 1, H, 192)

    def append(c, lens, new, positions):
        lib.mla_rope_append(c, cache, pages, i32(lens), kv_scale=kv_scale, rope_turns=turns, norm_weight=w_lat, eps=EPS,
                            positions=positions, new_lens=i32(new))

    def attend(q, positions, lens, new, words):
        qn, qr, _, _ = lib.mla_qk_norm_rope(q, positions=positions, rope_turns=turns, q_nope_weight=qw[0],
                                            q_rope_weight=qw[1], eps=EPS)
        n = q.shape[1]
        ql = lib.mla_absorb(qn.view(B * n, H, 128), w_uk).view(B, n, H, 512)
        o, _ = lib.mla_decode_tree(ql, qr, cache, pages, i32(lens), words, kv_scale=kv_scale, new_lens=i32(new),
                                   softmax_scale=SCALE)
        return lib.mla_absorb(o.view(B * n, H, 512), w_uv).view(B, n, H, 128)

    def wanted(q, pos, latent, rope):
        """fp64: one query row [H, 192] at `pos` over finished keys (latent [K, 512], rope [K, 64])."""
        q = q.double()
        k = torch.einsum("kl,hdl->khd", latent, w_uk.double())
        qr = turn(rms(q[:, 128:], qw[1].double()), torch.tensor(float(pos), device="cuda"))
        s = torch.einsum("hd,khd->hk", rms(q[:, :128], qw[0].double()), k) + qr @ rope.T
        p = (s * SCALE).softmax(-1)
        return torch.einsum("hk,kl,hld->hd", p, latent, w_uv.double())

    def finished(c, pos):
        return rms(c[..., :512].double(), w_lat.double()), turn(c[..., 512:].double(), pos)

    append(c_prompt, prompt, prompt, None)
    lens = [p + d for p, d in zip(prompt, drafts)]
    pos = i32(prompt)[:, None] + depth
    append(c_draft, lens, drafts, pos)
    got = attend(q_draft, pos, lens, drafts, mask)
    lib.check_device_error()
    tol = 2.0 ** -4 if fp8 else 2.0 ** -6  # e4m3 rows round by 2^-4, bf16 ones by 2^-8
    keys = {}
    for b in range(B):
        keys[b] = finished(c_prompt[b, :prompt[b]], torch.arange(prompt[b], device="cuda"))
        lat, rope = finished(c_draft[b], pos[b])
        for t in range(T):
            if t >= drafts[b]:
                assert not bool(got[b, t].any())
                continue
            path, j = [], t
            while j >= 0:
                path.append(j)
                j = int(parents[b, j])
            want = wanted(q_draft[b, t], int(pos[b, t]), torch.cat((keys[b][0], lat[path])),
                          torch.cat((keys[b][1], rope[path])))
            assert far(got[b, t], want) < tol, (b, t)

    # the accepted paths, moved to the places behind the prompt by appending their raw rows again
    accepted = [[0, 1, 3], [1], [0, 1, 2, 3]]
    count = [len(a) for a in accepted]
    rows = torch.zeros(B, max(count), 576, device="cuda", dtype=torch.bfloat16)
    for b, a in enumerate(accepted):
        rows[b, :len(a)] = c_draft[b, a]
    lens = [p + n for p, n in zip(prompt, count)]
    append(rows, lens, count, None)
    lens = [n + 1 for n in lens]
    append(c_last, lens, [1] * B, None)
    last = i32(lens)[:, None] - 1
    got = attend(q_last, last, lens, [1] * B, torch.ones(1, 1, dtype=torch.int32, device="cuda"))
    lib.check_device_error()
    for b, a in enumerate(accepted):
        lat, rope = finished(torch.cat((c_prompt[b, :prompt[b]], c_draft[b, a], c_last[b])),
                             torch.arange(lens[b], device="cuda"))
        assert far(got[b, 0], wanted(q_last[b, 0], lens[b] - 1, lat, rope)) < tol, b
