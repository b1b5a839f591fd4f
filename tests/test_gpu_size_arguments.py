"""Sizes past the range of the C entry points' integers are refused, not cut to their low bits."""
import pytest
import torch

from tests.test_gpu_decode_tree import Problem

pytestmark = pytest.mark.gpu


def test_a_page_table_wider_than_an_int(lib):
    # one row of 2^32 + 4 entries (17 GB, only the first few of them written); cut, it would be four wide
    p = Problem(4, 3, [130], False, seed=51)
    try:
        table = torch.empty((1, 2 ** 32 + 4), dtype=torch.int32, device="cuda")
    except torch.cuda.OutOfMemoryError:
        pytest.skip("no room for the table")
    table[:, :p.args[3].shape[1]] = p.args[3]
    ql, qr, cache, _, lens = p.args
    with pytest.raises(lib.MLAError, match="UNSUPPORTED"):
        lib.mla_decode_tree(ql, qr, cache, table, lens, p.mask, softmax_scale=0.1)
    before = cache.clone()
    turns = lib.rope_turns([1.0] * 32, "cuda")
    with pytest.raises(lib.MLAError, match="UNSUPPORTED"):
        lib.mla_rope_append(torch.zeros(1, 3, 576, dtype=torch.bfloat16, device="cuda"), cache, table, lens,
                            rope_turns=turns)
    torch.cuda.synchronize()
    assert torch.equal(cache.view(torch.uint8), before.view(torch.uint8))  # (rows behind the tokens hold NaN)
    lib.check_device_error()
