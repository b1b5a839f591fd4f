"""Refusals of the cross attention entry points in the C ABI and the binding (CPU only: every call
below is rejected before anything is launched)."""
import pytest
import torch

from tests.test_abi_rope import F, I, P, Z, binding, call, clib, cpu  # noqa: F401

SIZES = [("B", I), ("H", I), ("Sq", I), ("Sk", I), ("dn", I), ("dr", I), ("dv", I), ("scale", F), ("ws", P), ("wsb", Z),
         ("stream", P)]
OPERANDS = [("qn", P), ("qr", P), ("kn", P), ("kr", P), ("v", P), ("lens", P)]
FORWARD = OPERANDS + [("out", P), ("lse", P)] + SIZES
FORWARD0 = dict(qn=16, qr=16, kn=16, kr=16, v=16, lens=16, out=16, lse=16, B=2, H=3, Sq=4, Sk=5, dn=128, dr=64, dv=128,
                scale=0.1, ws=None, wsb=0, stream=None)

BACKWARD = OPERANDS + [("out", P), ("lse", P)] + [(n, P) for n in ("do", "dqn", "dqr", "dkn", "dkr", "dv_")] + SIZES
BACKWARD0 = dict(FORWARD0, do=16, dqn=16, dqr=16, dkn=16, dkr=16, dv_=16)
SHARED = [(1, {n: None}) for n in ("qn", "qr", "kn", "kr", "v", "out", "lse")]
SHARED += [(1, {n: 24}) for n in ("qn", "qr", "kn", "kr", "v", "out", "lse", "ws")]
SHARED += [(1, {n: bad}) for n in ("B", "H", "Sq", "Sk") for bad in (0, -1)]
SHARED += [(1, dict(lens=18)), (1, dict(scale=0.0)), (1, dict(scale=-1.0)), (1, dict(scale=float("nan"))),
           (1, dict(scale=float("inf"))), (2, dict(dn=64)), (2, dict(dr=32)), (2, dict(dv=64)), (2, dict(B=65536)),
           (2, dict(H=65536)), (2, dict(H=65535, Sk=2 ** 17)), (2, dict(H=65535, Sq=2 ** 17)),
           (2, dict(B=65535, H=65535, Sq=300))]


@pytest.mark.parametrize("want,kw", SHARED)
def test_forward_refuses(clib, want, kw):
    assert call(clib.mla_cross_attention, FORWARD, FORWARD0, **kw) == want
    assert b"mla_cross_attention" in clib.mla_last_error()


@pytest.mark.parametrize("want,kw", SHARED + [(1, {n: bad}) for n in ("do", "dqn", "dqr", "dkn", "dkr", "dv_")
                                              for bad in (None, 8)] + [(2, dict(B=65535, H=65535, Sq=1, Sk=3000))])
def test_backward_refuses(clib, want, kw):
    assert call(clib.mla_cross_attention_backward, BACKWARD, BACKWARD0, **kw) == want
    assert b"mla_cross_attention_backward" in clib.mla_last_error()


@pytest.mark.parametrize("name", ["mla_cross_attention_workspace_size", "mla_cross_attention_backward_workspace_size"])
def test_workspace_size_of_refused_sizes(clib, name):
    f = getattr(clib, name)
    f.restype, f.argtypes = Z, [I, I, I, I]
    assert f(0, 1, 1, 1) == f(1, 0, 1, 1) == f(1, 1, -1, 1) == f(1, 1, 1, 0) == f(65536, 1, 1, 1) == 0


def test_binding_refuses(binding):
    args = [cpu(1, 2, 3, 128), cpu(1, 2, 3, 64), cpu(1, 5, 3, 128), cpu(1, 5, 64), cpu(1, 5, 3, 128)]
    with pytest.raises(ValueError, match="CUDA"):
        binding.mla_cross_attention(*args, softmax_scale=0.1)
    grads = [cpu(1, 2, 3, 128), cpu(1, 3, 2, dtype=torch.float32), cpu(1, 2, 3, 128)]
    with pytest.raises(ValueError, match="CUDA"):
        binding.mla_cross_attention_backward(*args, *grads, softmax_scale=0.1)
    with pytest.raises(TypeError, match="tensor"):
        binding.mla_cross_attention(None, *args[1:], softmax_scale=0.1)
    with pytest.raises(ValueError, match="dimensions"):
        binding.mla_cross_attention(args[0][0], *args[1:], softmax_scale=0.1)
    with pytest.raises(TypeError, match="bfloat16"):
        binding.mla_cross_attention(args[0].half(), *args[1:], softmax_scale=0.1)
