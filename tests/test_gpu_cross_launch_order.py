"""Cross attention and its gradient behind the calls that make their inputs, and before calls that write over them and over
their workspace, without a wait between: the kernels of a call are set up under those before them, and the gradient's
loads begin there.  Every result as with a wait after each call, bit for bit."""
import pytest
import torch

from tests.test_gpu_cross import SCALE, randn

pytestmark = pytest.mark.gpu

FREQ = [10000.0 ** (-i / 32) for i in range(32)]


@pytest.mark.parametrize("B,H,Sq,Sk", [(2, 4, 60, 300), (1, 16, 1, 3000), (3, 8, 77, 257), (1, 8, 300, 200), (16, 16, 8, 130)])
def test_back_to_back(lib, B, H, Sq, Sk):
    g = torch.Generator(device="cuda").manual_seed(Sq)
    turns = lib.rope_turns_axes(FREQ, [0, 1] * 16, "cuda")
    pos = [torch.randint(0, 500, (B, S, 2), generator=g, device="cuda", dtype=torch.int32) for S in (Sq, Sk)]
    raw = [(randn(g, B, Sq, H, 192), randn(g, B, Sk, H, 128), randn(g, B, Sk, 64), randn(g, B, Sk, H, 128),
            randn(g, B, Sq, H, 128), torch.randint(0, Sk + 1, (B,), generator=g, device="cuda", dtype=torch.int32))
           for _ in range(4)]
    shapes = (B, Sq, H, 128), (B, Sq, H, 64), (B, Sk, H, 128), (B, Sk, 64), (B, Sk, H, 128)
    ops = [torch.zeros(s, device="cuda", dtype=torch.bfloat16) for s in shapes]
    d_out, lens = torch.zeros(B, Sq, H, 128, device="cuda", dtype=torch.bfloat16), torch.zeros(B, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(d_out), torch.zeros(B, H, Sq, device="cuda")
    grads = [torch.zeros_like(t) for t in ops]
    size = max(lib.cross_attention_workspace_size(B, H, Sq, Sk), lib.cross_attention_backward_workspace_size(B, H, Sq, Sk))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def one(x, wait):
        q, kn, kr, v, do, n = x
        steps = (lambda: lens.copy_(n), lambda: ops[4].copy_(v), lambda: d_out.copy_(do),
                 lambda: lib.mla_qk_norm_rope_axes(q, positions=pos[0], rope_turns=turns, out=(ops[0], ops[1], None, None)),
                 lambda: lib.mla_qk_norm_rope_axes(None, kn, kr, positions=pos[1], rope_turns=turns,
                                                   out=(None, None, ops[2], ops[3])),
                 lambda: lib.mla_cross_attention(*ops, lens, softmax_scale=SCALE, out=out, lse=lse, workspace=ws),
                 lambda: lib.mla_cross_attention_backward(*ops, out, lse, d_out, lens, softmax_scale=SCALE, grads=grads,
                                                          workspace=ws))
        for step in steps:
            step()
            if wait:
                torch.cuda.synchronize()
        return [t.clone() for t in (out, lse, *grads)]

    want = [one(x, True) for x in raw]
    for _ in range(60):
        got = [one(x, False) for x in raw]
        for a, b in zip(want, got):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [one(x, False) for x in raw]
    for _ in range(20):
        graph.replay()
        for a, b in zip(want, got):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
    lib.check_device_error()
