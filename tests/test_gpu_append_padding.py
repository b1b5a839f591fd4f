"""The rotated append of large padded batches, whose rows of padding are not read: bit for bit what the sequences
appended one at a time leave, rows behind the last token untouched, and a bad count reported as in small ones."""
import pytest
import torch

pytestmark = pytest.mark.gpu

FREQ = [10000.0 ** (-i / 32) for i in range(32)]
T = 8191
PAGES = (T + 64) // 64


class Batch:
    def __init__(self, lib, axes, fp8):
        g = torch.Generator(device="cuda").manual_seed(axes)
        self.B, self.axes = 6, axes
        self.raw = torch.randn(self.B, T, 576, generator=g, device="cuda").bfloat16()
        self.pages = torch.randperm(self.B * PAGES, generator=g, device="cuda").to(torch.int32).view(self.B, PAGES)
        self.pos = torch.randint(-5, 9000, (self.B, T, axes) if axes > 1 else (self.B, T), generator=g, device="cuda",
                                 dtype=torch.int32)
        self.w = torch.randn(512, generator=g, device="cuda").bfloat16()
        self.fp8 = fp8
        self.turns = lib.rope_turns_axes(FREQ, [0] * 8 + [1] * 12 + [2] * 12, "cuda") if axes > 1 else lib.rope_turns(FREQ, "cuda")
        self.call = lib.mla_rope_append_axes if axes > 1 else lib.mla_rope_append

    def cache(self):
        kv = torch.full((self.B * PAGES, 64, 576), 7.0, device="cuda").to(torch.float8_e4m3fn if self.fp8 else torch.bfloat16)
        return kv, torch.full((self.B * PAGES, 64), 7.0, device="cuda") if self.fp8 else None

    def append(self, at, lens, new):
        kv, scale = at
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.call(self.raw[self.rows], kv, self.pages[self.rows], i32(lens), scale, rope_turns=self.turns,
                  positions=self.pos[self.rows], norm_weight=self.w, new_lens=i32(new))

    rows = slice(None)


def same(a, b):
    return all(x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("axes", [1, 3])
def test_padded_batch(lib, axes, fp8):
    p = Batch(lib, axes, fp8)
    new = [T, 0, 1, 4000, -3, 77]
    lens = [T, 50, 1, 8000, 9, 40]  # of the last the first 37 have no place
    whole, parts = p.cache(), p.cache()
    p.append(whole, lens, new)
    for b in range(p.B):
        p.rows = slice(b, b + 1)
        p.append(parts, lens[b:b + 1], new[b:b + 1])
    lib.check_device_error()
    assert same(whole, parts)
    for b, (n, m) in enumerate(zip(lens, new)):
        first, last = max(n - max(m, 0), 0), n if m > 0 else 0
        bits = whole[0][p.pages[b].long()].view(PAGES * 64, 576).float()
        written = torch.zeros(PAGES * 64, dtype=torch.bool, device="cuda")
        if m > 0:
            written[first:last] = True
        assert bool((bits[~written] == 7.0).all()) and bool((bits[written] != 7.0).any(-1).all())


def test_more_new_tokens_than_rows_are_reported(lib):
    p = Batch(lib, 3, False)
    at = p.cache()
    p.append(at, [T + 1] * 6, [T, 0, T + 1, 5, 6, 7])
    with pytest.raises(lib.MLAError):
        lib.check_device_error()
    untouched = at[0][p.pages[2].long()].float()
    assert bool((untouched == 7.0).all())
    lib.check_device_error()
