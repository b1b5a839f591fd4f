"""GPU parity of mla_rope_append (through the C ABI) against the fp64 oracle.

Tolerances: bf16 rows 2^-8 |y| for the rounding plus 2^-17 (|y|, or |a| + |b| of a rotated pair)
for the fp32 arithmetic (a 512-term sum in chains of 16 + 5 additions, rsqrt, two products; sines and
cosines to 2^-19).  e4m3 rows: scale = amax / 448 to 2^-17, codes 2^-4 |y| relative or half the smallest step,
2^-10 scale, plus the same fp32 part.
"""
import numpy as np
import pytest
import torch

import oracle
from gen import make_decode
from oracle import norm_rope_ref as ref
from tests.test_gpu_norm_rope import EPS, FREQ, f64, pair_sum, randn

pytestmark = pytest.mark.gpu

DL, DR, D = 512, 64, 576


class Problem:
    """A cache of make_decode's layout (rows past the sequences hold NaN) and raw new rows."""

    def __init__(self, lens, T, fp8, seed, norm=True, new=None, positions=True, wide=False, extra_pages=2):
        from mla_flash_attention_gb300.testing import decode_to_device

        inp = make_decode(len(lens), 1, T, lens, fp8=fp8, seed=seed, extra_pages=extra_pages)
        d = decode_to_device(inp, torch.device("cuda"))
        self.fp8, self.T, self.B = fp8, T, inp.B
        self.cache, self.pt, self.lens = d["args"][2:5]
        self.scale = d["kwargs"]["kv_scale"]
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.c = randn(g, self.B, T, 1536 + D)[..., 1536:] if wide else randn(g, self.B, T, D)
        self.w = 1 + 0.3 * randn(g, DL) if norm else None
        self.new = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
        self.pos = torch.randint(0, 9000, (self.B, T), generator=g, device="cuda", dtype=torch.int32) \
            if positions else None

    def run(self, lib, interleaved, **kw):
        self.before = self.cache.clone(), None if self.scale is None else self.scale.clone()
        lib.mla_rope_append(self.c, self.cache, self.pt, self.lens, kv_scale=self.scale,
                            rope_turns=lib.rope_turns(FREQ, "cuda"), norm_weight=self.w, eps=EPS, positions=self.pos,
                            new_lens=self.new, interleaved=interleaved, **kw)

    def check(self, interleaved):
        new = np.full(self.B, self.T) if self.new is None else self.new.cpu().numpy()
        place = ref.append_places(self.lens.cpu().numpy(), new, self.T)
        pos = place if self.pos is None else self.pos.cpu().numpy()
        y = ref.rope_append_rows(f64(self.c), pos, FREQ, f64(self.w), EPS, interleaved)
        mag = np.concatenate([np.abs(y[..., :DL]), pair_sum(y[..., DL:], interleaved)], -1)
        table = self.pt.cpu().numpy()
        b, t = np.nonzero(place >= 0)
        page, row = table[b, place[b, t] // 64], place[b, t] % 64
        y, mag = y[b, t], mag[b, t]
        got = self.cache.float().double().cpu().numpy()[page, row]
        if self.fp8:
            s = self.scale.double().cpu().numpy()[page, row]
            amax = np.abs(y).max(-1)
            want = np.where(amax > 0, amax / 448, 1.0)
            assert (np.abs(s - want) <= 2.0 ** -17 * want).all()
            err = np.abs(got * s[:, None] - y)
            tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s[:, None]) + 2.0 ** -16 * mag
        else:
            err, tol = np.abs(got - y), 2.0 ** -8 * np.abs(y) + 2.0 ** -17 * mag
        assert np.isfinite(got).all() and (err <= tol).all(), (err - tol).max()
        # every other row of the cache, and every other scale, is as it was
        for t_, old in ((self.cache, self.before[0]), (self.scale, self.before[1])):
            if t_ is None:
                continue
            a = t_.view(torch.uint8).view(t_.shape[0], 64, -1).cpu().numpy().copy()
            o = old.view(torch.uint8).view(t_.shape[0], 64, -1).cpu().numpy()
            a[page, row] = o[page, row]
            assert np.array_equal(a, o)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 2, 5, 67])
def test_page_edges_and_short_sequences(lib, fp8, T, interleaved):
    p = Problem([1, 2, 63, 64, 65, 127, 128, 129, 3000], T, fp8, seed=31 + T)
    p.run(lib, interleaved)
    lib.check_device_error()
    p.check(interleaved)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("norm,positions,wide", [(False, True, False), (True, False, False), (True, True, True)])
def test_without_norm_at_own_places_and_strided_rows(lib, fp8, norm, positions, wide):
    p = Problem([7, 200, 64], 4, fp8, seed=40, norm=norm, positions=positions, wide=wide)
    p.run(lib, True)
    lib.check_device_error()
    p.check(True)


@pytest.mark.parametrize("fp8", [False, True])
def test_ragged_new_tokens(lib, fp8):
    # padding behind a sequence's last token, none at all, fewer cached than new, an empty sequence
    p = Problem([70, 70, 2, 0, 129, 64], 6, fp8, seed=41, new=[6, 1, 4, 0, 3, 0])
    p.run(lib, False)
    lib.check_device_error()
    p.check(False)


def test_lengths_of_no_meaning_write_nothing(lib):
    p = Problem([70, 70, 90], 2, True, seed=50)
    keep = p.lens.clone()
    p.lens[0], p.lens[1] = -2 ** 31, -5
    p.run(lib, True)
    lib.check_device_error()
    p.check(True)  # places below 0: not written, not reported
    p.lens.copy_(keep)
    p.lens[1] = 2 ** 31 - 1
    p.run(lib, True)
    with pytest.raises(lib.MLAError, match="DEVICE_CHECK"):
        lib.check_device_error()  # past the page table: reported, not written
    p.lens[1] = 0
    p.check(True)


def test_negative_and_oversized_counts(lib):
    p = Problem([70, 70, 90], 3, False, seed=42, new=[-5, 4, 2])
    p.run(lib, True)
    with pytest.raises(lib.MLAError, match="DEVICE_CHECK"):
        lib.check_device_error()  # sequence 1 claims more new tokens than rows: nothing of it is written
    p.check(True)


@pytest.mark.parametrize("fp8", [False, True])
def test_at_position_zero_it_is_the_plain_append(lib, fp8):
    p = Problem([65, 300, 2], 2, fp8, seed=43, norm=False)
    p.pos.zero_()
    plain = p.cache.clone(), None if p.scale is None else p.scale.clone()
    lib.mla_cache_append(p.c, plain[0], p.pt, p.lens, kv_scale=plain[1])
    p.run(lib, False)
    lib.check_device_error()
    # (-0.0 in a rope column may come out as +0.0; randn's bf16 values hold no zeros)
    assert torch.equal(p.cache.view(torch.uint8), plain[0].view(torch.uint8))
    assert p.scale is None or torch.equal(p.scale.view(torch.int32), plain[1].view(torch.int32))


def test_zero_rows_and_magnitudes_fp8(lib):
    p = Problem([64, 64, 64, 64], 1, True, seed=44, norm=False)
    for b, m in enumerate((0.0, 1e-3, 40.0, 1e15)):
        p.c[b] *= m
    p.run(lib, True)
    p.check(True)
    page = int(p.pt[0, 0])
    assert float(p.scale[page, 63]) == 1.0 and not bool(p.cache[page, 63].float().any())


def test_a_nan_stays_a_nan(lib):
    for fp8 in (False, True):
        p = Problem([10, 10], 1, fp8, seed=45, norm=False)
        p.c[0, 0, 3] = float("nan")
        p.run(lib, True)
        page = int(p.pt[0, 0])
        row = p.cache[page, 9].float()
        assert torch.isnan(row[3]) and int(torch.isnan(row).sum()) == 1
        if fp8:
            assert bool(torch.isfinite(p.scale[page, 9]))


def test_bad_page_is_reported_and_skipped(lib):
    p = Problem([10, 70, 5], 1, True, seed=46)
    p.pt[1, 1] = p.cache.shape[0] + 5
    p.run(lib, True)
    with pytest.raises(lib.MLAError, match="DEVICE_CHECK"):
        lib.check_device_error()
    keep = p.pt.clone()
    p.pt[1, 1] = 0
    p.lens[1] = 0  # nothing was written for sequence 1
    p.check(True)
    p.pt.copy_(keep)


@pytest.mark.parametrize("fp8", [False, True])
def test_writes_only_the_cache(lib, fp8):
    from tests.test_gpu_canaries import Guarded

    p = Problem([65, 300, 2], 3, fp8, seed=47, new=[3, 2, 3])
    cache = Guarded(tuple(p.cache.shape), p.cache.dtype, fill=p.cache)
    scale = Guarded(tuple(p.scale.shape), torch.float32, fill=p.scale) if fp8 else None
    p.cache, p.scale = cache.t, scale.t if fp8 else None
    p.run(lib, True)
    lib.check_device_error()
    assert cache.intact() and (scale is None or scale.intact())
    p.check(True)


def test_captured_and_replayed_as_the_sequences_grow(lib):
    p = Problem([300, 700], 1, False, seed=48, positions=False)
    p.lens -= 70
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.run(lib, True)
    torch.cuda.synchronize()
    turns = lib.rope_turns(FREQ, "cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.mla_rope_append(p.c, p.cache, p.pt, p.lens, rope_turns=turns, norm_weight=p.w, eps=EPS)
    for _ in range(66):  # over a page's end
        p.lens += 1
        p.c.add_(0.01)
        p.before = p.cache.clone(), None
        graph.replay()
        torch.cuda.synchronize()
        p.check(True)


def test_offsets_past_32_bits(lib):
    # 60000 pages hold 2.2e9 values (4.4 GB in bf16): the last pages lie past 2^31 elements
    pages = 60000
    for fp8 in (False, True):
        cache = torch.zeros(pages, 64, D, device="cuda", dtype=torch.bfloat16)
        cache = cache.to(torch.float8_e4m3fn) if fp8 else cache
        scale = torch.ones(pages, 64, device="cuda") if fp8 else None
        g = torch.Generator(device="cuda").manual_seed(49)
        c = randn(g, 2, 3, D)
        pt = torch.tensor([[pages - 1, 0], [5, pages - 2]], dtype=torch.int32, device="cuda")
        lens = torch.tensor([64, 128], dtype=torch.int32, device="cuda")
        lib.mla_rope_append(c, cache, pt, lens, kv_scale=scale, rope_turns=lib.rope_turns(FREQ, "cuda"))
        lib.check_device_error()
        y = ref.rope_append_rows(f64(c), [[61, 62, 63], [125, 126, 127]], FREQ, None, EPS, True)
        for b, page in ((0, pages - 1), (1, pages - 2)):
            got = cache[page, 61:].float().double()
            if fp8:
                got = got * scale[page, 61:, None].double()
            # e4m3: 2^-4 relative, 2^-10 of a scale below 5 / 448; bf16 is finer
            assert np.abs(got.cpu().numpy() - y[b]).max() <= 2.0 ** -4 * np.abs(y).max()
            assert not bool(cache[page, :61].float().any())
