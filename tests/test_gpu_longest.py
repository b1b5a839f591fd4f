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


@pytest.mark.parametrize("fp8,tree", [(False, True), (True, True), (False, False)])
def test_items_that_take_longer_than_a_wait_for_a_page(lib, fp8, tree):
    # 450000 pages an item, 0.6 s, in which some roles wait for its last page or for the next item's
    # queries: one query tile for each work unit (two SMs), for fp8 two
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    pages = 450000
    run, q, keys = inputs(lib, 128, sms // 2 * (2 if fp8 else 1), pages, fp8, tree)
    out, lse = run()
    lib.check_device_error()
    s = 0.05 * q @ keys.T
    w = torch.softmax(s, -1)
    # every fp32 sum of a page's share: half a step of 2^-24 at most on the row's sums, one of 2^-23 in each of the
    # four or less additions to the accumulator; 2^-8 twice for the weights and the output
    drift = pages * 2.0 ** -24
    err = (out[0].double() - w @ keys[:, :512]).abs()
    size = w @ keys[:, :512].abs()
    assert bool((err <= size * (2.0 ** -7 + 9 * drift)).all())
    want = torch.logsumexp(s, -1) + torch.tensor(float(pages)).double().log()
    assert float((lse[0].T.double() - want).abs().max()) <= 1e-3 + drift
