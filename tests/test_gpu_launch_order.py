"""Kernels of one call, and of calls behind one another, in the order that they rely on.

The decode calls zero their split counters (drafted trees: the list of items left to the merge kernel
too) in a kernel that the split kernel overlaps.  What comes behind the split kernel as its programmatic
dependent has to find that zeroing done, also where no sequence is split and nothing in the split kernel
needs it."""
import pytest
import torch

from gen import make_decode
from tests.test_gpu_decode_tree import Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[224] * 58, [5] * 150, [0] * 80, [70, 0, 3] * 30])
def test_a_list_left_in_the_workspace_is_not_merged(lib, fp8, lens):
    # (in the unzeroed workspace three items would be listed, all of them item 3 in splits 3, 4 and 5)
    p = Problem(16, 2, lens, fp8, seed=41, new=[min(2, L) for L in lens])
    ws = torch.empty(lib.decode_workspace_size(len(lens), 16, 2) // 4, dtype=torch.int32, device="cuda")
    got = []
    for _ in range(40):
        ws.fill_(3)
        got.append(p.run(lib, workspace=ws))
    lib.check_device_error()
    p.check(*got[0])
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("fp8,H", [(False, 16), (True, 16), (True, 64)])  # both split kernels, both cache types
def test_the_next_call_may_write_over_the_counters(lib, fp8, H):
    # the workspace's memory, its split counters among it, as the output of the call behind
    from mla_flash_attention_gb300.testing import decode_to_device

    B = 200
    inp = make_decode(B, H, 1, [60] * B, fp8=fp8, seed=42)
    d = decode_to_device(inp, torch.device("cuda"))
    ws = torch.empty(lib.decode_workspace_size(B, H, 1), dtype=torch.uint8, device="cuda")
    rows = ws.numel() // (2 * 192)
    q = torch.randn(1, rows, 1, 192, device="cuda").bfloat16()
    out = (ws[:rows * 256].view(torch.bfloat16).view(1, rows, 1, 128),
           torch.empty(1, rows, 1, 64, dtype=torch.bfloat16, device="cuda"), None, None)
    tail = (torch.empty(1, rows, 1, 128, dtype=torch.bfloat16, device="cuda"),
            ws[ws.numel() - rows * 128:].view(torch.bfloat16).view(1, rows, 1, 64), None, None)
    kw = dict(positions=torch.arange(rows, dtype=torch.int32, device="cuda")[None],
              rope_turns=lib.rope_turns([10000.0 ** (-i / 32) for i in range(32)], "cuda"))
    want = lib.mla_qk_norm_rope(q, **kw)
    for views in (out, tail):
        for _ in range(20):
            lib.mla_decode(*d["args"], **d["kwargs"], softmax_scale=inp.softmax_scale, workspace=ws)
            lib.mla_qk_norm_rope(q, **kw, out=views)
            assert torch.equal(views[0], want[0]) and torch.equal(views[1], want[1])
    lib.check_device_error()
