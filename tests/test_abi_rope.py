"""Refusals of the head-norm, rotated-append and drafted-tree entry points, in the C ABI and in
the binding (CPU only: every call below is rejected before anything is launched)."""
import ctypes
import os

import pytest
import torch

P, I, L, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


@pytest.fixture(scope="module")
def clib():
    from mla_flash_attention_gb300 import build

    if not (os.path.exists(build.LIB) and os.path.exists(build.MARSHAL)):
        build.build()
    lib = ctypes.CDLL(build.LIB)
    lib.mla_last_error.restype = ctypes.c_char_p
    return lib


@pytest.fixture(scope="module")
def binding(clib):
    from mla_flash_attention_gb300 import binding

    return binding


def call(f, spec, defaults, **kw):
    assert set(kw) <= set(defaults), set(kw) - set(defaults)
    v = dict(defaults, **kw)
    f.restype = ctypes.c_int
    return f(*[ty(v[n]) for n, ty in spec])


APPEND = [("c", P), ("stride", L), ("w", P), ("eps", F), ("pos", P), ("turns", P), ("il", I), ("cache", P),
          ("scale", P), ("pt", P), ("lens", P), ("new", P), ("B", I), ("T", I), ("dl", I), ("dr", I), ("ps", I),
          ("mp", I), ("npages", I), ("dt", I), ("stream", P)]
APPEND0 = dict(c=16, stride=576, w=16, eps=1e-6, pos=16, turns=16, il=1, cache=16, scale=None, pt=16, lens=16,
               new=16, B=1, T=1, dl=512, dr=64, ps=64, mp=1, npages=1, dt=0, stream=None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(c=None)), (1, dict(turns=None)), (1, dict(lens=None)), (1, dict(B=0)), (1, dict(T=-1)),
    (1, dict(npages=0)), (1, dict(stride=568)), (1, dict(stride=577)), (1, dict(eps=float("nan"))),
    (1, dict(eps=-1.0)), (1, dict(dt=1)), (1, dict(scale=16)), (1, dict(c=24)), (1, dict(w=8)), (1, dict(pos=18)),
    (1, dict(new=2)), (1, dict(turns=12)), (1, dict(dt=1, scale=18)),
    (2, dict(dl=256)), (2, dict(dr=32)), (2, dict(ps=32)), (2, dict(dt=2)), (2, dict(B=2 ** 16, T=2 ** 14)),
    (2, dict(mp=2 ** 26)),
])
def test_rope_append_refuses(clib, want, kw):
    assert call(clib.mla_rope_append, APPEND, APPEND0, **kw) == want
    assert b"mla_rope_append" in clib.mla_last_error()


TREE = [("ql", P), ("qr", P), ("cache", P), ("ks", P), ("pt", P), ("lens", P), ("mask", P), ("ms", L), ("new", P),
        ("out", P), ("lse", P), ("B", I), ("H", I), ("T", I), ("dl", I), ("dr", I), ("ps", I), ("mp", I),
        ("npages", I), ("scale", F), ("dt", I), ("ws", P), ("wsb", Z), ("stream", P)]
TREE0 = dict(ql=16, qr=16, cache=16, ks=None, pt=16, lens=16, mask=16, ms=0, new=None, out=16, lse=16, B=1, H=16, T=4,
             dl=512, dr=64, ps=64, mp=1, npages=1, scale=0.1, dt=0, ws=None, wsb=0, stream=None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(ql=None)), (1, dict(mask=None)), (1, dict(B=0)), (1, dict(T=0)), (1, dict(npages=-1)),
    (1, dict(ms=3)), (1, dict(ms=-4)), (1, dict(T=40, ms=79)), (1, dict(scale=0.0)), (1, dict(scale=float("inf"))),
    (1, dict(dt=1)), (1, dict(ks=16)), (1, dict(out=8)), (1, dict(mask=18)), (1, dict(new=1)), (1, dict(ws=8)),
    (2, dict(dl=256)), (2, dict(ps=128)), (2, dict(dt=2)), (2, dict(B=65536)), (2, dict(H=128, T=513)),
    (2, dict(B=65535, H=128, T=512)), (2, dict(B=65535, H=32769, T=1)),  # 65535 * 32769 > 2^31 - 1
    (2, dict(mp=2 ** 26)),
    (2, dict(npages=2 ** 26)),
])
def test_decode_tree_refuses(clib, want, kw):
    assert call(clib.mla_decode_tree, TREE, TREE0, **kw) == want
    assert b"mla_decode_tree" in clib.mla_last_error()


OPERANDS = [("q", P), ("qs", L), ("qh", L), ("kn", P), ("ks", L), ("kh", L), ("kr", P), ("krs", L), ("wqn", P),
            ("wqr", P), ("wkn", P), ("wkr", P), ("pos", P), ("turns", P), ("eps", F), ("il", I)]
OPERANDS0 = dict(q=16, qs=384, qh=192, kn=16, ks=256, kh=128, kr=16, krs=64, wqn=16, wqr=16, wkn=16, wkr=16, pos=16,
                 turns=16, eps=1e-6, il=1, R=3, H=2, dn=128, dr=64, stream=None)
SIZES = [("R", L), ("H", I), ("dn", I), ("dr", I)]
FORWARD = OPERANDS + [("oqn", P), ("oqr", P), ("okn", P), ("okr", P)] + SIZES + [("stream", P)]
FORWARD0 = dict(OPERANDS0, oqn=16, oqr=16, okn=16, okr=16)
BACKWARD = ([("uqn", P), ("uqr", P), ("ukn", P), ("ukr", P)] + OPERANDS +
            [("dq", P), ("dkn", P), ("dkr", P), ("dwqn", P), ("dwqr", P), ("dwkn", P), ("dwkr", P)] + SIZES +
            [("ws", P), ("wsb", Z), ("stream", P)])
BACKWARD0 = dict(OPERANDS0, uqn=16, uqr=16, ukn=16, ukr=16, dq=16, dkn=16, dkr=16, dwqn=16, dwqr=16, dwkn=16,
                 dwkr=16, ws=None, wsb=0)

SHARED = [
    (1, dict(q=None, kn=None, kr=None)), (1, dict(pos=None)), (1, dict(turns=None)), (1, dict(q=None)),
    (1, dict(kn=None)), (1, dict(kr=None)), (1, dict(R=0)), (1, dict(H=0)), (1, dict(eps=-1e-6)),
    (1, dict(eps=float("inf"))), (1, dict(q=24)), (1, dict(wqr=8)), (1, dict(pos=18)), (1, dict(turns=20)),
    (1, dict(qs=385)), (1, dict(kh=-128)), (1, dict(krs=4)),
    (2, dict(dn=64)), (2, dict(dr=128)), (2, dict(H=65536)), (2, dict(R=2 ** 31)), (2, dict(R=2 ** 28, H=100)),
    (2, dict(qs=2 ** 62)),
]


@pytest.mark.parametrize("want,kw", SHARED + [(1, dict(oqr=None)), (1, dict(okn=None)), (1, dict(okr=8))])
def test_qk_norm_rope_refuses(clib, want, kw):
    assert call(clib.mla_qk_norm_rope, FORWARD, FORWARD0, **kw) == want
    assert b"mla_qk_norm_rope" in clib.mla_last_error()


@pytest.mark.parametrize("want,kw", SHARED + [
    (1, dict(uqn=None)), (1, dict(ukr=None)), (1, dict(dq=None)), (1, dict(dkr=8)), (1, dict(dwqn=None)),
    (1, dict(wqn=None)), (1, dict(dwkr=18)),
    (1, dict(qh=0)), (1, dict(qs=0)), (1, dict(kh=64)), (1, dict(krs=0)),   # gradients would overlap
    (1, dict(qs=192, qh=192)),
])
def test_qk_norm_rope_backward_refuses(clib, want, kw):
    assert call(clib.mla_qk_norm_rope_backward, BACKWARD, BACKWARD0, **kw) == want
    assert b"mla_qk_norm_rope_backward" in clib.mla_last_error()


def test_backward_workspace_size_of_refused_sizes(clib):
    f = clib.mla_qk_norm_rope_backward_workspace_size
    f.restype, f.argtypes = Z, [L, I]
    assert f(0, 4) == 0 and f(4, 0) == 0 and f(4, 65536) == 0 and f(2 ** 40, 4) == 0


# ------------------------------------------------------------------------------- the binding

def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_host_tensors_types_and_shapes(binding):
    turns = binding.rope_turns([1.0] * 32)
    pos = cpu(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="one of q"):
        binding.mla_qk_norm_rope(positions=pos, rope_turns=turns)
    with pytest.raises(ValueError, match="CUDA"):
        binding.mla_qk_norm_rope(cpu(1, 2, 3, 192), positions=pos, rope_turns=turns)
    with pytest.raises(TypeError, match="bfloat16"):
        binding.mla_qk_norm_rope(cpu(1, 2, 3, 192, dtype=torch.float16), positions=pos, rope_turns=turns)
    with pytest.raises(ValueError, match="dimensions"):
        binding.mla_qk_norm_rope(cpu(2, 3, 192), positions=pos, rope_turns=turns)
    with pytest.raises(ValueError, match="CUDA"):
        binding.mla_rope_append(cpu(1, 1, 576), cpu(2, 64, 576), cpu(1, 1, dtype=torch.int32),
                                cpu(1, dtype=torch.int32), rope_turns=turns)
    with pytest.raises(ValueError, match="dimensions"):
        binding.mla_rope_append(cpu(1, 576), cpu(2, 64, 576), cpu(1, 1, dtype=torch.int32),
                                cpu(1, dtype=torch.int32), rope_turns=turns)
    with pytest.raises(ValueError, match="CUDA"):
        binding.mla_decode_tree(cpu(1, 1, 4, 512), cpu(1, 1, 4, 64), cpu(2, 64, 576), cpu(1, 1, dtype=torch.int32),
                                cpu(1, dtype=torch.int32), cpu(1, 1, dtype=torch.int32), softmax_scale=0.1)
