"""GPU parity of mla_decode_tree (through the C ABI) against the fp64 oracle.

Tolerances are mla_decode's: the arithmetic is the same, only the mask differs."""
import numpy as np
import pytest
import torch

import oracle
from gen import make_decode
from tests.parity import TOL_O_BF16, TOL_O_FP8, check

pytestmark = pytest.mark.gpu


def random_parents(B, T, seed):
    rng = np.random.default_rng(seed)
    return np.array([[int(rng.integers(max(-1, t - 4), t)) if t else -1 for t in range(T)] for _ in range(B)])


def sees_of(mask, T):
    m = mask.cpu().numpy().astype(np.int64)
    j = np.arange(T)
    return (m[..., j // 32] >> (j % 32) & 1).astype(bool)


class Problem:
    def __init__(self, H, T, lens, fp8, seed, new=None, shared=False, mask=None, extra_pages=1):
        from mla_flash_attention_gb300 import binding
        from mla_flash_attention_gb300.testing import decode_to_device

        B = len(lens)
        self.inp = inp = make_decode(B, H, T, lens, fp8=fp8, seed=seed, extra_pages=extra_pages)
        if mask is None:
            mask, _ = binding.tree_mask_from_parents(random_parents(1 if shared else B, T, seed))
            mask = mask[0] if shared else mask
        self.mask = mask.cuda()
        self.sees = np.broadcast_to(sees_of(mask, T), (B, T, T))
        self.new = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
        d = decode_to_device(inp, torch.device("cuda"))
        self.args, self.kv_scale = d["args"], d["kwargs"]["kv_scale"]

    def run(self, lib, **kw):
        return lib.mla_decode_tree(*self.args, self.mask, kv_scale=self.kv_scale, new_lens=self.new,
                                   softmax_scale=self.inp.softmax_scale, **kw)

    def check(self, out, lse, what=""):
        n = None if self.new is None else self.new.cpu().numpy().clip(0, self.inp.T)
        O, L = oracle.mla_decode_tree(self.inp, self.sees, n)
        check(out.float().cpu().numpy(), O, lse.cpu().numpy(), L, TOL_O_FP8 if self.inp.fp8 else TOL_O_BF16, what=what)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,T,lens,new", [
    (1, 1, [1], None),                                    # the smallest call
    (16, 1, [1, 64, 65, 700], None),                      # single tokens
    (8, 4, [3, 4, 64, 66, 67, 130], None),                # trees across a page's end; fewer keys than nodes
    (16, 8, [1000, 8, 72, 64], [8, 3, 5, 1]),             # ragged trees, padding rows
    (4, 33, [33, 90, 400], None),                         # two mask words
    (128, 3, [300, 65], None),                            # three tiles of query rows
    (16, 13, [13, 500, 64, 0, 77], [13, 0, 7, 5, 13]),    # no drafted token, an empty sequence
    (3, 64, [64, 63, 200], [64, 64, 50]),                 # 64 nodes: a whole page of drafted keys
    (2, 150, [140, 600], [150, 131]),                     # five mask words over three pages
    (128, 5, [300, 65, 0, 700, 9, 64], [1, 5, 3, 0, 3, 2]),  # whole tiles of query rows that are padding
    (48, 7, [2000, 130], [3, 6]),                         # tiles that end in padding, or within a token's heads
])
def test_trees(lib, H, T, lens, new, fp8):
    p = Problem(H, T, lens, fp8, seed=H * 100 + T, new=new)
    out, lse = p.run(lib)
    lib.check_device_error()
    p.check(out, lse, "H=%d T=%d fp8=%d" % (H, T, fp8))


@pytest.mark.parametrize("fp8", [False, True])
def test_one_mask_for_the_batch(lib, fp8):
    p = Problem(16, 9, [9, 70, 128, 1000], fp8, seed=5, shared=True)
    assert p.mask.dim() == 2
    p.check(*p.run(lib))
    lib.check_device_error()


@pytest.mark.parametrize("fp8,H,T", [(False, 128, 1), (False, 16, 2), (False, 40, 5), (True, 64, 2), (True, 128, 4)])
def test_a_chain_is_mla_decode(lib, fp8, H, T):
    mask, depth = lib.tree_mask_from_parents(torch.arange(T) - 1)
    assert depth.tolist() == list(range(T))
    p = Problem(H, T, [T, 64, 65, 3000], fp8, seed=6, mask=mask)
    out, lse = p.run(lib)
    o, l = lib.mla_decode(*p.args, kv_scale=p.kv_scale, softmax_scale=p.inp.softmax_scale)
    lib.check_device_error()
    if fp8:  # another kernel (e4m3 operands): both are held to the oracle, not to each other's bits
        p.check(out, lse)
        p.check(o, l)
    else:    # the same arithmetic in the same order
        assert torch.equal(out, o) and torch.equal(lse, l)


def test_a_single_key_is_its_value(lib):
    # one visible key: the weight is one, whatever the scores, so O is the key's dequantised row
    p = Problem(16, 1, [1, 1], True, seed=19)
    out, _ = p.run(lib)
    for b in range(2):
        page = int(p.inp.page_table[b, 0])
        row = p.args[2][page, 0, :512].float() * p.kv_scale[page, 0]
        assert torch.equal(out[b], row.bfloat16().expand(1, 16, 512))


@pytest.mark.parametrize("scale", [1e-30, 1e-4, 1.0, 1e4])
@pytest.mark.parametrize("spread", [1.0, 1e6])
def test_query_and_key_magnitudes_fp8(lib, scale, spread):
    # rows whose largest value is anywhere in bf16's range, elements far below it, key scales of
    # unlike sizes: scores are kept near one by the softmax scale
    p = Problem(16, 5, [70, 300], True, seed=20)
    g = torch.Generator(device="cuda").manual_seed(1)
    ql = p.args[0].float() * scale
    ql *= spread ** -torch.rand(ql.shape, generator=g, device="cuda")  # elements down to 1 / spread
    p.args[0] = ql.bfloat16()
    p.args[1] = (p.args[1].float() * scale).bfloat16()
    p.kv_scale *= 2.0 ** torch.randint(-6, 7, p.kv_scale.shape, generator=g, device="cuda")
    for name, t in (("q_latent", p.args[0]), ("q_rope", p.args[1])):
        setattr(p.inp, name, t.view(torch.int16).cpu().numpy().view(np.uint16))
    p.inp.kv_scale = p.kv_scale.cpu().numpy()
    p.inp.softmax_scale = float(np.float32(p.inp.softmax_scale / scale / 16))
    out, lse = p.run(lib)
    lib.check_device_error()
    O, L = oracle.mla_decode_tree(p.inp, p.sees)
    # the weights' two e4m3 terms and the output's rounding: 2^-8 each of the values they multiply
    # (|O| at most the largest visible one); scores: hi + lo terms to 2^-19 of a row's largest product
    vmax = np.abs(oracle.decode_gather(p.inp, 0)[:, :512]).max(), np.abs(oracle.decode_gather(p.inp, 1)[:, :512]).max()
    for b in range(2):
        assert np.abs(out[b].float().cpu().numpy() - O[b]).max() <= 2.0 ** -7 * vmax[b]
    assert np.abs(lse.cpu().numpy() - L).max() <= 1e-3


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_non_finite_query_stays_in_its_row(lib, fp8, value):
    p = Problem(40, 4, [130, 9], fp8, seed=21)
    clean = p.run(lib)
    p.args[0][0, 2, 7, 300] = value
    out, lse = p.run(lib)
    lib.check_device_error()
    assert bool(torch.isnan(out[0, 2, 7]).all()) and bool(torch.isnan(lse[0, 7, 2]))
    out[0, 2, 7], lse[0, 7, 2] = clean[0][0, 2, 7], clean[1][0, 7, 2]
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_that_see_nothing_or_anything(lib, fp8):
    # bits are taken as they are: empty rows, rows that see later tokens, bits past the tree
    T = 40
    rng = np.random.default_rng(3)
    mask = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, (3, T, 2)).astype(np.int32))
    mask[:, 5] = 0
    mask[1, :20] = 0
    p = Problem(4, T, [T, 25, 300], fp8, seed=7, mask=mask, new=[T, 30, 33])
    out, lse = p.run(lib)
    lib.check_device_error()
    p.check(out, lse)
    assert bool((out[0, 5] == 0).all()) and bool(torch.isneginf(lse[0, :, 5]).all())  # no prefix, no bit


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("H,T", [(4, 6), (128, 6)])
def test_non_finite_drafted_keys_reach_only_rows_that_see_them(lib, fp8, value, H, T):
    if fp8 and value != value:
        spots = ("code", "scale")
    elif fp8:
        spots = ("scale",)  # e4m3 has no infinity
    else:
        spots = ("latent", "rope")
    for spot in spots:
        lens = [64 + 3, 30, 400]
        p = Problem(H, T, lens, fp8, seed=8, shared=True)
        clean_out, clean_lse = p.run(lib)
        node = 2
        for b, L in enumerate(lens):
            place = L - T + node
            page, row = int(p.inp.page_table[b, place // 64]), place % 64
            if spot == "scale":
                p.kv_scale[page, row] = value
            elif spot == "code":
                p.args[2].view(torch.uint8)[page, row, 77] = 0xFF
            else:
                p.args[2][page, row, 300 if spot == "latent" else 570] = value
        out, lse = p.run(lib)
        lib.check_device_error()
        hit = torch.from_numpy(p.sees[0, :, node].copy()).cuda()
        assert bool(hit.any()) and not bool(hit.all())
        assert bool(torch.isnan(out[:, hit]).all()) and bool(torch.isnan(lse[:, :, hit]).all()), spot
        assert torch.equal(out[:, ~hit], clean_out[:, ~hit]), spot
        assert torch.equal(lse[:, :, ~hit], clean_lse[:, :, ~hit]), spot


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("node,column", [(0, 0), (99, 575), (37, 255), (36, 256), (63, 511), (64, 512), (27, 128), (28, 447)])
def test_a_non_finite_value_anywhere_in_a_tree_over_three_pages(lib, fp8, node, column):
    # 36 + 64 keys drafted up to a page's end, 28 + 64 + 8 otherwise: each page's first, last and other rows
    T, lens = 100, [64 * 3, 64 * 2 + 8, 100]
    p = Problem(4, T, lens, fp8, seed=31, shared=True)
    clean_out, clean_lse = p.run(lib)
    for b, L in enumerate(lens):
        place = L - T + node
        page, row = int(p.inp.page_table[b, place // 64]), place % 64
        if fp8:
            p.args[2].view(torch.uint8)[page, row, column] = 0x7F
        else:
            p.args[2][page, row, column] = float("-inf")
    out, lse = p.run(lib)
    lib.check_device_error()
    hit = torch.from_numpy(p.sees[0, :, node].copy()).cuda()
    assert bool(hit.any())
    assert bool(torch.isnan(out[:, hit]).all()) and bool(torch.isnan(lse[:, :, hit]).all())
    assert torch.equal(out[:, ~hit], clean_out[:, ~hit]) and torch.equal(lse[:, :, ~hit], clean_lse[:, :, ~hit])


@pytest.mark.parametrize("fp8", [False, True])
def test_padding_rows_are_zero_whatever_the_prefix_holds(lib, fp8):
    p = Problem(8, 5, [200], fp8, seed=9, new=[2])
    page = int(p.inp.page_table[0, 0])
    if fp8:
        p.args[2].view(torch.uint8)[page, 3, 5] = 0x7F
    else:
        p.args[2][page, 3, 5] = float("nan")
    out, lse = p.run(lib)
    lib.check_device_error()
    assert bool((out[0, 2:] == 0).all()) and bool(torch.isneginf(lse[0, :, 2:]).all())
    assert bool(torch.isnan(out[0, :2]).all()) and bool(torch.isnan(lse[0, :, :2]).all())


def test_counts_outside_the_range_are_clamped(lib):
    p = Problem(16, 4, [100, 100], False, seed=10, new=[9, -3])
    out, lse = p.run(lib)
    lib.check_device_error()
    p.check(out, lse)


def test_long_sequence_split_over_every_unit(lib):
    p = Problem(16, 12, [32768, 1], False, seed=11, new=[12, 1])
    out, lse = p.run(lib)
    lib.check_device_error()
    p.check(out, lse)
    again = p.run(lib)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_many_short_sequences(lib):
    rng = np.random.default_rng(4)
    new = rng.integers(0, 6, 300)
    p = Problem(4, 5, list(np.maximum(new, rng.integers(1, 130, 300))), True, seed=12, new=list(new.clip(0, 5)))
    out, lse = p.run(lib)
    lib.check_device_error()
    p.check(out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("long", [0, 900])
def test_many_query_tiles_of_one_page(lib, fp8, long):
    # each work unit takes several items, most of one page: an item's queries and its only page are
    # asked for while the item before is still loading its own
    lens = [long if long and b % 7 == 3 else 4 + b % 60 for b in range(160)]
    p = Problem(128, 4, lens, fp8, seed=29)
    p.check(*p.run(lib))
    lib.check_device_error()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,H,T,L", [(1, 16, 4, 700), (3, 64, 5, 333), (20, 16, 2, 190), (36, 8, 3, 500), (40, 16, 2, 260),
                                     (58, 16, 2, 224), (76, 8, 2, 70), (77, 8, 2, 70)])
def test_sequences_of_one_length_on_whole_units(lib, fp8, B, H, T, L):
    # items cut evenly, uncut, cut anywhere; in two splits merged by either kernel; some a page shorter, some empty
    for lens in ([L] * B, [L - 64 * (b % 3 == 1) if b % 5 else 0 for b in range(B)]):
        p = Problem(H, T, lens, fp8, seed=37)
        p.check(*p.run(lib))
    lib.check_device_error()


def test_bad_page_is_reported(lib):
    p = Problem(4, 3, [100, 100], False, seed=13)
    p.args[3][1, 1] = p.inp.num_pages + 5
    p.run(lib)
    with pytest.raises(lib.MLAError, match="DEVICE_CHECK"):
        lib.check_device_error()


@pytest.mark.parametrize("fp8", [False, True])
def test_writes_only_out_lse_and_workspace(lib, fp8):
    from tests.test_gpu_canaries import Guarded

    p = Problem(40, 5, [5, 130, 777], fp8, seed=14, new=[5, 2, 4])
    inp = p.inp
    out = Guarded((inp.B, inp.T, inp.H, 512), torch.bfloat16)
    lse = Guarded((inp.B, inp.H, inp.T), torch.float32)
    ws = Guarded((lib.decode_workspace_size(inp.B, inp.H, inp.T),), torch.uint8)
    before = p.args[2].view(torch.uint8).clone()
    p.run(lib, out=out.t, lse=lse.t, workspace=ws.t)
    lib.check_device_error()
    assert out.intact() and lse.intact() and ws.intact()
    assert torch.equal(p.args[2].view(torch.uint8), before)
    p.check(out.t, lse.t)


@pytest.mark.parametrize("fp8", [False, True])
def test_an_output_aligned_to_16_bytes_only(lib, fp8):
    # items in one split, in two and in more; rows that end a tile
    p = Problem(40, 5, [5, 130, 9000, 20, 40, 60], fp8, seed=15, new=[5, 2, 4, 0, 1, 5])
    ref, ref_lse = p.run(lib)
    flat = torch.full((ref.numel() + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = flat[8:8 + ref.numel()].view(ref.shape)
    assert out.data_ptr() % 32 == 16
    _, lse = p.run(lib, out=out)
    lib.check_device_error()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    assert (flat[:8] == 7).all() and (flat[-8:] == 7).all()


def test_captured_and_replayed_with_new_lengths_and_masks(lib):
    p = Problem(16, 7, [500, 130], False, seed=15, new=[7, 4])
    other = Problem(16, 7, [410, 128], False, seed=15, new=[2, 7])
    ws = torch.empty(lib.decode_workspace_size(2, 16, 7), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p.run(lib, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = p.run(lib, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    p.check(out, lse)
    for a, b in zip(p.args, other.args):
        a.zero_()
        a.view(-1)[:b.numel()].copy_(b.reshape(-1)) if a is p.args[2] else a.copy_(
            torch.nn.functional.pad(b, (0, a.shape[-1] - b.shape[-1])))
    p.mask.copy_(other.mask)
    p.new.copy_(other.new)
    graph.replay()
    torch.cuda.synchronize()
    lib.check_device_error()
    other.check(out, lse)


def test_two_calls_at_once_on_two_streams(lib):
    ps = [Problem(16, 6, [3000, 900, 64], bool(i % 2), seed=16 + i) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    got = [[p.run(lib, stream=s) for p, s in zip(ps, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    lib.check_device_error()
    for r in got:
        for p, (out, lse) in zip(ps, r):
            p.check(out, lse)


def test_refusals_of_the_binding(lib):
    p = Problem(4, 3, [100], False, seed=17)
    with pytest.raises(ValueError, match="tree_mask"):
        lib.mla_decode_tree(*p.args, p.mask[:, :2].contiguous(), softmax_scale=0.1)
    with pytest.raises(TypeError, match="tree_mask"):
        lib.mla_decode_tree(*p.args, p.mask.long(), softmax_scale=0.1)
    with pytest.raises(ValueError, match="new_lens"):
        lib.mla_decode_tree(*p.args, p.mask, new_lens=torch.ones(1, dtype=torch.int32), softmax_scale=0.1)
    with pytest.raises(ValueError, match="workspace"):
        lib.mla_decode_tree(*p.args, p.mask, softmax_scale=0.1, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(lib.MLAError, match="WORKSPACE"):
        lib.mla_decode_tree(*p.args, p.mask, softmax_scale=0.1,
                            workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(lib.MLAError, match="UNSUPPORTED"):
        cache = p.args[2].view(-1, 32, 576)
        lib.mla_decode_tree(p.args[0], p.args[1], cache, *p.args[3:], p.mask, softmax_scale=0.1)


def test_offsets_past_32_bits(lib):
    # 60000 pages hold 2.2e9 values: the sequence's pages lie at both ends of the pool
    p = Problem(16, 4, [130], False, seed=18)
    pages = 60000
    pool = torch.zeros(pages, 64, 576, device="cuda", dtype=torch.bfloat16)
    where = torch.tensor([pages - 1, 0, pages - 2], device="cuda")
    pool[where] = p.args[2][p.args[3][0].long()]
    want = p.run(lib)
    out, lse = lib.mla_decode_tree(p.args[0], p.args[1], pool, where.to(torch.int32)[None], p.args[4], p.mask,
                                   softmax_scale=p.inp.softmax_scale)
    lib.check_device_error()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
