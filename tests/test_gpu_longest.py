"""The decode calls at the far end of their documented lengths: page tables that name one page over and
over, so that hardly any memory is needed."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def inputs(lib, H, T, pages, fp8, tree):
    gen = torch.Generator(device="cuda").manual_seed(61)
    page = torch.randn(1, 64, 576, generator=gen, device="cuda")
    scale = page.abs().amax(-1) / 448 if fp8 else None
    cache = (page / scale[..., None]).to(torch.float8_e4m3fn) if fp8 else page.bfloat16()
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    lens = torch.tensor([64 * pages], dtype=torch.int32, device="cuda")
    ql = torch.randn(1, T, H, 512, generator=gen, device="cuda").bfloat16()
    qr = torch.randn(1, T, H, 64, generator=gen, device="cuda").bfloat16()
    mask = torch.full((T, (T + 31) // 32), -1, dtype=torch.int32, device="cuda")
    def run():
        if tree:
            return lib.mla_decode_tree(ql, qr, cache, table, lens, mask, kv_scale=scale, softmax_scale=0.05)
        return lib.mla_decode(ql, qr, cache, table, lens, kv_scale=scale, softmax_scale=0.05, causal=False)
    return run, torch.cat((ql, qr), -1)[0].double(), cache[0].double() * (scale[0, :, None].double() if fp8 else 1)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_more_pages_than_can_be_numbered(lib, fp8, tree):
    # 2^25 - 1 pages for each of 64 query tiles: 2^31 - 64, and what each tile is charged
    run, _, _ = inputs(lib, 128, 64, 2 ** 25 - 1, fp8, tree)
    run()
    with pytest.raises(lib.MLAError, match="DEVICE_CHECK"):
        lib.check_device_error()
