"""mla_decode_tree over an fp8 cache where few keys outweigh many: a dominating key with a long tail
that holds much of the mass together, levels that rise and fall from page to page, key scales of
unlike sizes.  Scores come from two rope columns, so that a row's weights are what the test says."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE = 64


def levels(kind, n, gen):
    """Nats of the n keys at q's nominal size (rows multiply them by 0.8 .. 1.2)."""
    page = torch.arange(n) // PAGE
    lev = torch.full((n,), -11.0)
    if kind == "first":
        lev[0] = 0
    elif kind == "middle":
        lev[n // 2 + 5] = 0
    elif kind == "last":
        lev[-1] = 0
    elif kind == "two":            # a second one, larger, in the middle
        lev[0], lev[n // 2] = -5, 0
    elif kind == "every other page":
        lev = torch.where(page % 2 == 0, 0.0, -9.0)
    elif kind == "falling":
        lev = -16.0 * page / page[-1]
    elif kind == "rising":
        lev = -16.0 + 16.0 * page / page[-1]
    elif kind == "bumps":          # in every page one key far above the others, all below the first
        lev[:] = -15
        lev[::PAGE] = -10
        lev[0] = 0
    elif kind == "blocks":
        lev = torch.where(page // 16 % 2 == 0, 0.0, -9.0)
    elif kind == "deep":           # nothing but the first key, to any accuracy
        lev[:] = -26
        lev[0] = 0
    return lev


class Peaked:
    def __init__(self, kind, n, H=16, T=1, B=152, sd=0.0, scales="one", seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        pages = (n + PAGE - 1) // PAGE
        v = (1 + 0.5 * torch.randn(n, 512, generator=gen, device="cuda")).clamp(-3, 3)
        lev = levels(kind, n, gen).cuda()
        v[lev > -1] *= 0.05
        ks = torch.full((n,), 2.0 ** -7, device="cuda")
        if scales == "dominating key 2^6":
            ks[lev == 0] *= 64
            v[lev == 0] *= 64
        elif scales == "any":
            power = 2.0 ** torch.randint(-6, 7, (n,), generator=gen, device="cuda")
            ks, v = ks * power, v * power[:, None]
        k = torch.zeros(pages * PAGE, 576, device="cuda")
        # (scores are one size whatever the key's scale, as far as its codes allow: up to 448 steps)
        k[:n, :512] = v
        k[:n, 512] = lev / 8
        k[:n, 513] = sd * torch.randn(n, generator=gen, device="cuda") / 4
        s = torch.ones(pages * PAGE, device="cuda")
        s[:n] = ks
        self.cache = (k / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(pages, PAGE, 576)
        self.kv_scale = s.view(pages, PAGE)
        self.table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, pages).contiguous()
        self.lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
        self.ql = torch.zeros(B, T, H, 512, dtype=torch.bfloat16, device="cuda")
        self.qr = torch.zeros(B, T, H, 64, dtype=torch.bfloat16, device="cuda")
        self.qr[..., 0] = (8 * (0.8 + 0.4 * torch.rand(B, T, H, generator=gen, device="cuda"))).bfloat16()
        self.qr[..., 1] = 4
        self.mask = torch.tensor([[(1 << (t + 1)) - 1] for t in range(T)], dtype=torch.int32, device="cuda")
        self.n, self.T = n, T
        self.args = (self.ql, self.qr, self.cache, self.table, self.lens)

    def check(self, out, lse, b):
        """Sequence b against 64 bits.  Errors: a weight is a sum of two terms of four and three bits
        (2^-8 of itself, as bf16's) down to a step that adds up to at most 2^-9 of the sum of the pages'
        largest weights, of which a second such error is allowed for levels that fall in more than one
        step; the output's rounding, 2^-8; fp32 sums and exponents, 2^-16."""
        keys = (self.cache.view(-1, 576)[:self.n].double() * self.kv_scale.view(-1)[:self.n, None].double())
        q = torch.cat((self.ql[b], self.qr[b]), -1).double()
        s = torch.einsum("thd,kd->thk", q, keys)
        place = torch.arange(self.n, device="cuda")
        for t in range(self.T):
            s[t, :, place >= self.n - self.T + t + 1] = -math.inf
        want_lse = torch.logsumexp(s, -1)
        w = torch.exp(s - want_lse[..., None])
        v = keys[:, :512]
        want, size = w @ v, w @ v.abs()
        # weights as the product takes them: times the key's scale, the values in codes up to 448
        scaled = torch.nn.functional.pad(w * self.kv_scale.view(-1)[:self.n].double(), (0, -self.n % PAGE))
        top = scaled.unflatten(-1, (-1, PAGE)).amax(-1).sum(-1) * self.cache.float().abs().max().double()
        tol = size * (2.0 ** -8 + 2.0 ** -16) + want.abs() * 2.0 ** -8 + top[..., None] * 2.0 ** -8
        err = (out[b].double() - want).abs()
        assert bool((err <= tol).all()), "worst %.2e of %.2e allowed, value %.3f" % (
            float(err.max()), float(tol[err - tol == (err - tol).max()][0]), float(want[err - tol == (err - tol).max()][0]))
        assert float((lse[b].T.double() - want_lse).abs().max()) <= 1e-4

    def error(self, out, b):
        """The 2-norm of sequence b's error (one token) relative to 64 bits."""
        keys = (self.cache.view(-1, 576)[:self.n].double() * self.kv_scale.view(-1)[:self.n, None].double())
        s = torch.cat((self.ql[b, 0], self.qr[b, 0]), -1).double() @ keys.T
        want = torch.softmax(s, -1) @ keys[:, :512]
        return float((out[b, 0].double() - want).norm() / want.norm())


KINDS = ["first", "middle", "last", "two", "every other page", "falling", "rising", "bumps", "blocks", "deep"]


@pytest.mark.parametrize("sd", [0.0, 0.5, 2.0])
@pytest.mark.parametrize("kind", KINDS)
def test_tails_keep_their_mass(lib, kind, sd):
    # whole sequences by one work unit (a unit a pair of SMs), the largest key anywhere
    p = Peaked(kind, 16384 if sd else 8192 + 37, sd=sd)
    out, lse = lib.mla_decode_tree(*p.args, p.mask, kv_scale=p.kv_scale, softmax_scale=1.0)
    lib.check_device_error()
    for b in (0, 75, 151):
        p.check(out, lse, b)


@pytest.mark.parametrize("kind", ["first", "two", "blocks"])
@pytest.mark.parametrize("scales", ["dominating key 2^6", "any"])
def test_key_scales_of_unlike_sizes(lib, kind, scales):
    p = Peaked(kind, 16384, sd=0.5, scales=scales)
    out, lse = lib.mla_decode_tree(*p.args, p.mask, kv_scale=p.kv_scale, softmax_scale=1.0)
    lib.check_device_error()
    for b in (1, 76):
        p.check(out, lse, b)


@pytest.mark.parametrize("H,T,B", [(128, 1, 80), (16, 3, 100), (40, 5, 3), (1, 1, 1)])  # tiles, trees, split sequences
def test_tails_in_other_forms(lib, H, T, B):
    p = Peaked("first", 12000, H=H, T=T, B=B, sd=0.3)
    out, lse = lib.mla_decode_tree(*p.args, p.mask, kv_scale=p.kv_scale, softmax_scale=1.0)
    lib.check_device_error()
    for b in {0, B - 1}:
        p.check(out, lse, b)


@pytest.mark.parametrize("H", [16, 64])
def test_a_chain_is_as_accurate_as_mla_decode(lib, H):
    p = Peaked("first", 16384, H=H, B=152)
    out, lse = lib.mla_decode_tree(*p.args, p.mask, kv_scale=p.kv_scale, softmax_scale=1.0)
    o, _ = lib.mla_decode(*p.args, kv_scale=p.kv_scale, softmax_scale=1.0)
    lib.check_device_error()
    for b in (0, 151):
        p.check(out, lse, b)
        # (the output's rounding alone is 2^-8 at most)
        assert p.error(out, b) <= p.error(o, b) + 2.0 ** -9, (p.error(out, b), p.error(o, b))
