"""Thin binding of the C ABI (include/mla.h).

Argument marshalling only: torch tensors are checked for device, dtype, shape and
contiguity, then their device pointers and the current CUDA stream are passed to
the library, through ctypes or, for the calls around the attention (norms, rotated
append, drafted trees) and cross attention, through the compiled module ``_marshal``.  Every step of the
attention runs inside the library's CUDA kernels; there is no fallback of any kind:
if the shared library is missing, importing this module raises, and if ``_marshal``
is missing or does not fit the installed torch, the calls that it marshals raise.
"""
from __future__ import annotations

import ctypes
import math
import numbers
import os
from typing import Optional

import torch



class _NoMarshal:
    """Stands in for ``_marshal`` where that does not load: the calls it marshals raise."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError("the marshalling module is not built (%s); run "
                          "`python -c 'import __graft_entry__ as g; g.build()'`" % self._why)


try:
    from . import _marshal
except ImportError as e:
    _marshal = _NoMarshal(e)

# MLA_GB300_LIB selects another build of the same library, e.g. the bounds-checked
# libmla_gb300_debug.so (mla_flash_attention_gb300.build.build(debug=True))
_LIB_PATH = os.environ.get("MLA_GB300_LIB") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libmla_gb300.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(
        "%s is not built; run `python -c 'import __graft_entry__ as g; g.build()'`" % _LIB_PATH)
_lib = ctypes.CDLL(_LIB_PATH)

MLA_OK = 0
MLA_BF16, MLA_FP8_E4M3, MLA_FP32 = 0, 1, 2
STATUS = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_WORKSPACE",
          4: "MLA_ERR_CUDA", 5: "MLA_ERR_TIMEOUT", 6: "MLA_ERR_DEVICE_CHECK"}

_vp, _fp, _ip = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
_i, _f, _sz = ctypes.c_int, ctypes.c_float, ctypes.c_size_t

_lib.mla_prefill.restype = _i
_lib.mla_prefill.argtypes = [_vp, _vp, _vp, _vp, _vp, _fp, _fp, _vp, _fp, _i, _i, _i, _i, _i, _i,
                             _f, _i, _i, _i, _vp]
_lib.mla_decode_workspace_size.restype = _sz
_lib.mla_decode_workspace_size.argtypes = [_i, _i, _i, _i]
_lib.mla_decode.restype = _i
_lib.mla_decode.argtypes = [_vp, _vp, _vp, _fp, _ip, _ip, _vp, _fp, _i, _i, _i, _i, _i, _i, _i, _i,
                            _f, _i, _i, _vp, _sz, _vp]
_lib.mla_decode_noalloc.restype = _i
_lib.mla_decode_noalloc.argtypes = [_vp, _vp, _vp, _fp, _ip, _ip, _vp, _fp, _i, _i, _i, _i, _i, _i,
                                    _i, _i, _f, _i, _i, _vp]
_lib.mla_decode_noalloc_max_workspace.restype = _sz
_lib.mla_decode_noalloc_max_workspace.argtypes = []
_lib.mla_absorb.restype = _i
_lib.mla_absorb.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _vp]
_lib.mla_cache_append.restype = _i
_lib.mla_cache_append.argtypes = [_vp, _vp, _fp, _ip, _ip, _i, _i, _i, _i, _i, _i, _i, _i, _vp]
_ll = ctypes.c_int64
_lib.mla_rope_append.restype = _i
_lib.mla_rope_append.argtypes = [_vp, _ll, _vp, _f, _ip, _vp, _i, _vp, _fp, _ip, _ip, _ip, _i, _i, _i, _i, _i, _i,
                                 _i, _i, _vp]
_lib.mla_decode_tree.restype = _i
_lib.mla_decode_tree.argtypes = [_vp, _vp, _vp, _fp, _ip, _ip, _vp, _ll, _ip, _vp, _fp, _i, _i, _i, _i, _i, _i, _i,
                                 _i, _f, _i, _vp, _sz, _vp]
_lib.mla_qk_norm_rope.restype = _i
_lib.mla_qk_norm_rope.argtypes = [_vp, _ll, _ll, _vp, _ll, _ll, _vp, _ll, _vp, _vp, _vp, _vp, _ip, _vp, _f, _i, _vp,
                                  _vp, _vp, _vp, _ll, _i, _i, _i, _vp]
_lib.mla_qk_norm_rope_backward_workspace_size.restype = _sz
_lib.mla_qk_norm_rope_backward_workspace_size.argtypes = [_ll, _i]
_lib.mla_qk_norm_rope_backward.restype = _i
_lib.mla_qk_norm_rope_backward.argtypes = [_vp, _vp, _vp, _fp, _vp, _ll, _ll, _vp, _ll, _ll, _vp, _ll, _vp, _vp, _vp,
                                           _vp, _ip, _vp, _f, _i, _vp, _vp, _vp, _fp, _fp, _fp, _fp, _ll, _i, _i, _i,
                                           _vp, _sz, _vp]
_lib.mla_rope_append_axes.restype = _i
_lib.mla_rope_append_axes.argtypes = [_vp, _ll, _vp, _f, _ip, _vp, _i, _i, _vp, _fp, _ip, _ip, _ip, _i, _i, _i, _i, _i,
                                      _i, _i, _i, _vp]
_lib.mla_qk_norm_rope_axes.restype = _i
_lib.mla_qk_norm_rope_axes.argtypes = [_vp, _ll, _ll, _vp, _ll, _ll, _vp, _ll, _vp, _vp, _vp, _vp, _ip, _vp, _i, _f, _i,
                                       _vp, _vp, _vp, _vp, _ll, _i, _i, _i, _vp]
_lib.mla_qk_norm_rope_axes_backward.restype = _i
_lib.mla_qk_norm_rope_axes_backward.argtypes = [_vp, _vp, _vp, _vp, _i, _vp, _ll, _ll, _vp, _ll, _ll, _vp, _ll, _vp, _vp,
                                                _vp, _vp, _ip, _vp, _i, _f, _i, _vp, _vp, _vp, _fp, _fp, _fp, _fp, _ll,
                                                _i, _i, _i, _vp, _sz, _vp]
_lib.mla_cross_attention_workspace_size.restype = _sz
_lib.mla_cross_attention_workspace_size.argtypes = [_i, _i, _i, _i]
_lib.mla_cross_attention.restype = _i
_lib.mla_cross_attention.argtypes = [_vp, _vp, _vp, _vp, _vp, _ip, _vp, _fp, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _sz, _vp]
_lib.mla_cross_attention_backward_workspace_size.restype = _sz
_lib.mla_cross_attention_backward_workspace_size.argtypes = [_i, _i, _i, _i]
_lib.mla_cross_attention_backward.restype = _i
_lib.mla_cross_attention_backward.argtypes = [_vp, _vp, _vp, _vp, _vp, _ip, _vp, _fp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i,
                                              _i, _i, _i, _i, _i, _f, _vp, _sz, _vp]
_lib.mla_prefill_backward_workspace_size.restype = _sz
_lib.mla_prefill_backward_workspace_size.argtypes = [_i, _i, _i]
_lib.mla_prefill_backward.restype = _i
_lib.mla_prefill_backward.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _fp, _vp, _vp, _vp, _vp, _fp,
                                      _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _sz, _vp]
_lib.mla_check_device_error.restype = _i
_lib.mla_check_device_error.argtypes = [_vp]
_lib.mla_last_error.restype = ctypes.c_char_p
_lib.mla_last_error.argtypes = []
_lib.mla_version.restype = _i
_lib.mla_version.argtypes = []
_lib.mla_testing_decode_stall.restype = None
_lib.mla_testing_decode_stall.argtypes = [_i, ctypes.c_longlong]
_lib.mla_testing_bounds_checked.restype = _i
_lib.mla_testing_bounds_checked.argtypes = []
_lib.mla_testing_bounds_shrink.restype = None
_lib.mla_testing_bounds_shrink.argtypes = [ctypes.c_longlong]
_lib.mla_testing_cross_plan.restype = _i
_lib.mla_testing_cross_plan.argtypes = [_i, _i, _i, _i, _i, _i, _ip]
_lib.mla_testing_cross_backward_plan.restype = _i
_lib.mla_testing_cross_backward_plan.argtypes = [_i, _i, _i, _i, _i, _ip, _ip]

EXPORTED = ("mla_prefill", "mla_decode_workspace_size", "mla_decode", "mla_decode_noalloc",
            "mla_decode_noalloc_max_workspace", "mla_cache_append", "mla_absorb",
            "mla_prefill_backward_workspace_size", "mla_prefill_backward",
            "mla_rope_append", "mla_decode_tree", "mla_qk_norm_rope",
            "mla_qk_norm_rope_backward_workspace_size", "mla_qk_norm_rope_backward",
            "mla_rope_append_axes", "mla_qk_norm_rope_axes", "mla_qk_norm_rope_axes_backward",
            "mla_cross_attention_workspace_size", "mla_cross_attention",
            "mla_cross_attention_backward_workspace_size", "mla_cross_attention_backward",
            "mla_check_device_error",
            "mla_last_error", "mla_version", "mla_testing_decode_stall", "mla_testing_bounds_checked",
            "mla_testing_bounds_shrink", "mla_testing_cross_plan", "mla_testing_cross_backward_plan")


class MLAError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("%s: %s" % (STATUS.get(status, status), msg))
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def _check(st: int):
    if st != MLA_OK:
        raise MLAError(st, _lib.mla_last_error().decode(errors="replace"))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, name, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must have dtype %s (got %s)" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def version() -> int:
    return _lib.mla_version()


def testing_decode_stall(skip_unit: int = -1, wait_limit_cycles: int = 0) -> None:
    """Test hook (include/mla_testing.h): later fp8 decode calls with q_len*H <= 32 leave
    pipeline unit `skip_unit` unloaded and give each device wait `wait_limit_cycles` SM clocks.
    ``testing_decode_stall()`` restores normal calls."""
    _lib.mla_testing_decode_stall(int(skip_unit), int(wait_limit_cycles))


def testing_bounds_checked() -> bool:
    """True when the loaded library is the bounds-checked build (include/mla_testing.h)."""
    return bool(_lib.mla_testing_bounds_checked())


def testing_bounds_shrink(nbytes: int = 0) -> None:
    """Test hook (include/mla_testing.h): later launches report `out` as `nbytes` smaller to
    the store checks of the bounds-checked build; ``testing_bounds_shrink()`` restores them."""
    _lib.mla_testing_bounds_shrink(int(nbytes))


def testing_cross_plan(B: int, H: int, Sq: int, Sk: int, ragged: bool = False, sms: int = 0):
    """Test hook (include/mla_testing.h): (form, shares) of mla_cross_attention with key lengths or
    without; form 0 without tiles, 1 one query tile, 2 two."""
    n = _i()
    return int(_lib.mla_testing_cross_plan(B, H, Sq, Sk, int(ragged), sms, ctypes.addressof(n))), n.value


def testing_cross_backward_plan(B: int, H: int, Sq: int, Sk: int, sms: int = 0):
    """Test hook (include/mla_testing.h): (form, query shares, key shares) of
    mla_cross_attention_backward; form 0 without tiles, 1 by tiles."""
    q, k = _i(), _i()
    form = _lib.mla_testing_cross_backward_plan(B, H, Sq, Sk, sms, ctypes.addressof(q), ctypes.addressof(k))
    return int(form), q.value, k.value


def check_device_error(stream=None) -> None:
    _check(_lib.mla_check_device_error(_stream(stream)))


def mla_prefill(q_nope, q_rope, k_nope, k_rope, v, q_scale=None, k_scale=None, *,
                softmax_scale: float, causal: bool = True, out=None, lse=None,
                out_dtype=None, stream=None):
    """Fused MLA prefill.  Returns (out [B,S,H,d_v], lse [B,H,S] fp32).

    bf16 inputs: q_nope/k_nope/v bf16.  fp8 inputs: q_nope/k_nope/v float8_e4m3fn with
    q_scale/k_scale fp32 [B,S].  Rope parts are always bf16 (k_rope [B,S,d_rope]).
    """
    B, S, H, dn = q_nope.shape
    dr = q_rope.shape[-1]
    dv = v.shape[-1]
    fp8 = q_nope.dtype == torch.float8_e4m3fn
    qkv_dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    _need(q_nope, "q_nope", qkv_dt, (B, S, H, dn))
    _need(q_rope, "q_rope", torch.bfloat16, (B, S, H, dr))
    _need(k_nope, "k_nope", qkv_dt, (B, S, H, dn))
    _need(k_rope, "k_rope", torch.bfloat16, (B, S, dr))
    _need(v, "v", qkv_dt, (B, S, H, dv))
    if fp8:
        _need(q_scale, "q_scale", torch.float32, (B, S))
        _need(k_scale, "k_scale", torch.float32, (B, S))
    elif q_scale is not None or k_scale is not None:
        raise ValueError("q_scale/k_scale are only used with fp8 inputs")
    if out_dtype is None:
        out_dtype = torch.float32 if fp8 else torch.bfloat16
    dev = q_nope.device
    if out is None:
        out = torch.empty((B, S, H, dv), dtype=out_dtype, device=dev)
    if lse is None:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=dev)
    _need(out, "out", out_dtype, (B, S, H, dv))
    _need(lse, "lse", torch.float32, (B, H, S))
    st = _lib.mla_prefill(_ptr(q_nope), _ptr(q_rope), _ptr(k_nope), _ptr(k_rope), _ptr(v),
                          _ptr(q_scale), _ptr(k_scale), _ptr(out), _ptr(lse), B, H, S, dn, dr,
                          dv, float(softmax_scale), int(bool(causal)),
                          MLA_FP8_E4M3 if fp8 else MLA_BF16,
                          MLA_FP32 if out_dtype == torch.float32 else MLA_BF16, _stream(stream))
    _check(st)
    return out, lse


def prefill_backward_workspace_size(B: int, H: int, S: int) -> int:
    return int(_lib.mla_prefill_backward_workspace_size(B, H, S))


def mla_prefill_backward(q_nope, q_rope, k_nope, k_rope, v, out, lse, d_out, *,
                         softmax_scale: float, causal: bool = True, grads=None, workspace=None,
                         stream=None):
    """Gradients of bf16 MLA prefill.  Returns (dq_nope, dq_rope, dk_nope, dk_rope, dv).

    out/lse are the forward's results, d_out the upstream gradient [B,S,H,d_v] bf16.
    dk_rope [B,S,d_rope] is fp32 (summed over heads); the others are bf16 in the layouts of
    their operands.  ``grads`` may pass those five tensors preallocated.
    """
    B, S, H, dn = q_nope.shape
    dr = q_rope.shape[-1]
    dv_ = v.shape[-1]
    bf = torch.bfloat16
    _need(q_nope, "q_nope", bf, (B, S, H, dn))
    _need(q_rope, "q_rope", bf, (B, S, H, dr))
    _need(k_nope, "k_nope", bf, (B, S, H, dn))
    _need(k_rope, "k_rope", bf, (B, S, dr))
    _need(v, "v", bf, (B, S, H, dv_))
    _need(out, "out", bf, (B, S, H, dv_))
    _need(lse, "lse", torch.float32, (B, H, S))
    _need(d_out, "d_out", bf, (B, S, H, dv_))
    dev = q_nope.device
    if grads is None:
        grads = (torch.empty((B, S, H, dn), dtype=bf, device=dev),
                 torch.empty((B, S, H, dr), dtype=bf, device=dev),
                 torch.empty((B, S, H, dn), dtype=bf, device=dev),
                 torch.empty((B, S, dr), dtype=torch.float32, device=dev),
                 torch.empty((B, S, H, dv_), dtype=bf, device=dev))
    dq_n, dq_r, dk_n, dk_r, dv = grads
    _need(dq_n, "dq_nope", bf, (B, S, H, dn))
    _need(dq_r, "dq_rope", bf, (B, S, H, dr))
    _need(dk_n, "dk_nope", bf, (B, S, H, dn))
    _need(dk_r, "dk_rope", torch.float32, (B, S, dr))
    _need(dv, "dv", bf, (B, S, H, dv_))
    need = prefill_backward_workspace_size(B, H, S)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    st = _lib.mla_prefill_backward(_ptr(q_nope), _ptr(q_rope), _ptr(k_nope), _ptr(k_rope), _ptr(v),
                                   _ptr(out), _ptr(lse), _ptr(d_out), _ptr(dq_n), _ptr(dq_r),
                                   _ptr(dk_n), _ptr(dk_r), _ptr(dv), B, H, S, dn, dr, dv_,
                                   float(softmax_scale), int(bool(causal)), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st)
    return dq_n, dq_r, dk_n, dk_r, dv


def decode_workspace_size(B: int, H: int, q_len: int, d_latent: int = 512) -> int:
    return int(_lib.mla_decode_workspace_size(B, H, q_len, d_latent))


def mla_decode(q_latent, q_rope, kv_cache, page_table, cache_lens, kv_scale=None, *,
               softmax_scale: float, causal: bool = True, out=None, lse=None, workspace=None,
               stream=None):
    """Absorbed MLA decode over a paged latent cache.  Returns (out [B,T,H,dl] bf16,
    lse [B,H,T] fp32).  kv_cache bf16 or float8_e4m3fn [num_pages, page_size, dl+dr];
    kv_scale fp32 [num_pages, page_size] for fp8."""
    B, T, H, dl = q_latent.shape
    dr = q_rope.shape[-1]
    num_pages, page_size, D = kv_cache.shape
    fp8 = kv_cache.dtype == torch.float8_e4m3fn
    _need(q_latent, "q_latent", torch.bfloat16, (B, T, H, dl))
    _need(q_rope, "q_rope", torch.bfloat16, (B, T, H, dr))
    _need(kv_cache, "kv_cache", torch.float8_e4m3fn if fp8 else torch.bfloat16,
          (num_pages, page_size, dl + dr))
    if fp8:
        _need(kv_scale, "kv_scale", torch.float32, (num_pages, page_size))
    elif kv_scale is not None:
        raise ValueError("kv_scale is only used with an fp8 cache")
    max_pages = page_table.shape[1]
    _need(page_table, "page_table", torch.int32, (B, max_pages))
    _need(cache_lens, "cache_lens", torch.int32, (B,))
    dev = q_latent.device
    if out is None:
        out = torch.empty((B, T, H, dl), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=dev)
    _need(out, "out", torch.bfloat16, (B, T, H, dl))
    _need(lse, "lse", torch.float32, (B, H, T))
    need = decode_workspace_size(B, H, T, dl)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    st = _lib.mla_decode(_ptr(q_latent), _ptr(q_rope), _ptr(kv_cache), _ptr(kv_scale),
                         _ptr(page_table), _ptr(cache_lens), _ptr(out), _ptr(lse), B, H, T, dl,
                         dr, page_size, max_pages, num_pages, float(softmax_scale),
                         int(bool(causal)), MLA_FP8_E4M3 if fp8 else MLA_BF16, _ptr(workspace),
                         workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st)
    return out, lse


def mla_absorb(x, w, *, out=None, stream=None):
    """y[r, h, :] = x[r, h, :] @ w[h] for x [R, H, K] and w [H, K, N] (bf16); returns y [R, H, N]."""
    R, H, K = x.shape
    N = w.shape[-1]
    _need(x, "x", torch.bfloat16, (R, H, K))
    _need(w, "w", torch.bfloat16, (H, K, N))
    if out is None:
        out = torch.empty((R, H, N), dtype=torch.bfloat16, device=x.device)
    _need(out, "out", torch.bfloat16, (R, H, N))
    _check(_lib.mla_absorb(_ptr(x), _ptr(w), _ptr(out), R, H, K, N, _stream(stream)))
    return out


def mla_cache_append(c_new, kv_cache, page_table, cache_lens, kv_scale=None, *, stream=None):
    """Write the q_len new tokens' rows c_new [B, q_len, dl+dr] (bf16) into the paged cache
    (bf16, or float8_e4m3fn with per-row fp32 kv_scale [num_pages, page_size]) at positions
    cache_lens[b] - q_len + t.  Modifies kv_cache (and kv_scale) in place."""
    B, T, D = c_new.shape
    num_pages, page_size, Dc = kv_cache.shape
    fp8 = kv_cache.dtype == torch.float8_e4m3fn
    _need(c_new, "c_new", torch.bfloat16, (B, T, D))
    _need(kv_cache, "kv_cache", torch.float8_e4m3fn if fp8 else torch.bfloat16, (num_pages, page_size, D))
    if fp8:
        _need(kv_scale, "kv_scale", torch.float32, (num_pages, page_size))
    elif kv_scale is not None:
        raise ValueError("kv_scale is only used with an fp8 cache")
    max_pages = page_table.shape[1]
    _need(page_table, "page_table", torch.int32, (B, max_pages))
    _need(cache_lens, "cache_lens", torch.int32, (B,))
    st = _lib.mla_cache_append(_ptr(c_new), _ptr(kv_cache), _ptr(kv_scale), _ptr(page_table),
                               _ptr(cache_lens), B, T, D - 64, 64, page_size,
                               max_pages, num_pages, MLA_FP8_E4M3 if fp8 else MLA_BF16,
                               _stream(stream))
    _check(st)
    return kv_cache, kv_scale


def decode_noalloc_max_workspace() -> int:
    return int(_lib.mla_decode_noalloc_max_workspace())


def mla_decode_noalloc_setup() -> None:
    """The set-up call of mla_decode_noalloc on the current device (B = 0): the built-in
    scratch array is reserved and the decode kernels are loaded, so that later calls on this
    device allocate nothing.  Make it before reserving device memory and before any stream
    capture."""
    _check(_lib.mla_decode_noalloc(None, None, None, None, None, None, None, None, 0, 0, 0, 0, 0,
                                   0, 0, 0, 0.0, 1, MLA_BF16, None))


def mla_decode_noalloc(q_latent, q_rope, kv_cache, page_table, cache_lens, kv_scale=None, *,
                       softmax_scale: float, causal: bool = True, out=None, lse=None, stream=None):
    """mla_decode without a workspace: for callers that cannot allocate device memory at
    call time.  The split partials use the library's built-in scratch array (see
    include/mla.h); calls on one device must not overlap on the GPU.  ``out``/``lse`` may
    be passed in so that the call itself allocates nothing."""
    B, T, H, dl = q_latent.shape
    dr = q_rope.shape[-1]
    num_pages, page_size, _ = kv_cache.shape
    fp8 = kv_cache.dtype == torch.float8_e4m3fn
    _need(q_latent, "q_latent", torch.bfloat16, (B, T, H, dl))
    _need(q_rope, "q_rope", torch.bfloat16, (B, T, H, dr))
    _need(kv_cache, "kv_cache", torch.float8_e4m3fn if fp8 else torch.bfloat16,
          (num_pages, page_size, dl + dr))
    if fp8:
        _need(kv_scale, "kv_scale", torch.float32, (num_pages, page_size))
    elif kv_scale is not None:
        raise ValueError("kv_scale is only used with an fp8 cache")
    max_pages = page_table.shape[1]
    _need(page_table, "page_table", torch.int32, (B, max_pages))
    _need(cache_lens, "cache_lens", torch.int32, (B,))
    dev = q_latent.device
    if out is None:
        out = torch.empty((B, T, H, dl), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=dev)
    _need(out, "out", torch.bfloat16, (B, T, H, dl))
    _need(lse, "lse", torch.float32, (B, H, T))
    st = _lib.mla_decode_noalloc(_ptr(q_latent), _ptr(q_rope), _ptr(kv_cache), _ptr(kv_scale),
                                 _ptr(page_table), _ptr(cache_lens), _ptr(out), _ptr(lse), B, H, T,
                                 dl, dr, page_size, max_pages, num_pages, float(softmax_scale),
                                 int(bool(causal)), MLA_FP8_E4M3 if fp8 else MLA_BF16,
                                 _stream(stream))
    _check(st)
    return out, lse


# ------------------------------------------------- around the attention: norms, rotation, trees

# Their arguments are checked, their outputs and workspaces allocated and the C entry points
# called by the compiled module _marshal (csrc/marshal.cpp): in Python that took several times as
# long as the kernels of a decode step.

def _address(f) -> int:
    return ctypes.cast(f, ctypes.c_void_p).value


if not isinstance(_marshal, _NoMarshal):
    _marshal.connect(tuple(_address(f) for f in (
        _lib.mla_qk_norm_rope, _lib.mla_qk_norm_rope_axes, _lib.mla_qk_norm_rope_backward,
        _lib.mla_qk_norm_rope_axes_backward, _lib.mla_qk_norm_rope_backward_workspace_size, _lib.mla_rope_append,
        _lib.mla_rope_append_axes, _lib.mla_decode_tree, _lib.mla_decode_workspace_size, _lib.mla_cross_attention,
        _lib.mla_cross_attention_workspace_size, _lib.mla_cross_attention_backward,
        _lib.mla_cross_attention_backward_workspace_size)), _check)


def _call(stream, tensor, f, *args):
    """f(*args) with `stream` (a torch.cuda.Stream) the stream that outputs and workspaces are
    allocated and the kernels launched on; None: the current stream of the tensors' device."""
    if stream is None:
        return f(*args)
    if isinstance(tensor, torch.Tensor) and stream.device != tensor.device:
        raise ValueError("stream must be on the tensors' device %s (got %s)" % (tensor.device, stream.device))
    with torch.cuda.stream(stream):
        return f(*args)


def rope_turns(inv_freq, device=None) -> torch.Tensor:
    """Position rotation of the entry points below: turns per position in units of 2^-64
    (int64 bits of the uint64 values, include/mla.h) for the angular frequencies ``inv_freq``
    [d_rope / 2] in radians per position.  Positions times these are exact modulo whole turns,
    however far.  Make it once and keep it; any scaling of the frequencies goes in here."""
    freqs = [float(f) for f in (inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else inv_freq)]
    if not all(math.isfinite(f) for f in freqs):
        raise ValueError("inv_freq must be finite")
    turns = [int(round(f / (2 * math.pi) * 2.0 ** 64)) % 2 ** 64 for f in freqs]
    return torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=device)


def rope_turns_axes(inv_freq, pair_axes, device=None) -> torch.Tensor:
    """rope_turns for positions on several axes (time, height, width): a table int64 [axes, d_rope / 2] for the
    entry points that end in ``_axes``.  ``inv_freq`` [d_rope / 2] as for ``rope_turns``; ``pair_axes``
    [d_rope / 2] names the axis whose position turns each pair (0, 1, ..), in any order: sections one
    after another ([0] * 8 + [1] * 12 + [2] * 12), axes in turn, halves for rows and columns."""
    freqs = inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else list(inv_freq)
    axis = pair_axes.tolist() if isinstance(pair_axes, torch.Tensor) else list(pair_axes)  # (an array's integers too)
    if len(freqs) != len(axis) or not axis:
        raise ValueError("pair_axes must name an axis for each of the %d pairs (got %d)" % (len(freqs), len(axis)))
    if not all(isinstance(a, numbers.Integral) and not isinstance(a, bool) and 0 <= a < 4 for a in axis):
        raise ValueError("pair_axes must be integers from 0 to 3")
    return torch.stack([rope_turns([f if a == row else 0.0 for f, a in zip(freqs, axis)], device)
                        for row in range(int(max(axis)) + 1)])


def tree_mask_from_parents(parents):
    """The tree_mask words and the depths of drafted trees.  parents [q_len] or [B, q_len]
    integers: token t's parent among the drafted tokens, an index below t, or -1 for a child of
    the last accepted token.  Returns (mask int32 [..., q_len, ceil(q_len / 32)] with the bits of
    every token's ancestors and itself, depth int32 [..., q_len], 0 for a child of the last
    accepted token).  Reads ``parents`` on the host."""
    par = parents if isinstance(parents, torch.Tensor) else torch.as_tensor(parents)
    if par.dim() not in (1, 2) or par.shape[-1] == 0 or par.dtype.is_floating_point or par.dtype == torch.bool:
        raise ValueError("parents must be integers of shape [q_len] or [B, q_len]")
    dev, par = par.device, par.cpu().to(torch.int64)
    with torch.device("cpu"):  # whatever the program's default device
        T = par.shape[-1]
        if bool(((par >= torch.arange(T)) | (par < -1)).any()):
            raise ValueError("a parent must be -1 or the index of an earlier token")
        sees = torch.zeros(*par.shape, T + 1)  # column T stands for the last accepted token
        sees.scatter_(-1, torch.where(par < 0, T, par)[..., None], 1.0)
        sees = sees[..., :T] + torch.eye(T)
        for _ in range(max(1, T.bit_length())):  # ancestors up to 2, 4, 8, ... generations back
            sees = ((sees @ sees) > 0).float()
        W = (T + 31) // 32
        bits = torch.zeros(*par.shape, W * 32, dtype=torch.int64)
        bits[..., :T] = sees.to(torch.int64)
        words = (bits.unflatten(-1, (W, 32)) << torch.arange(32)).sum(-1)
        words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    return words.to(dev), (sees.sum(-1).to(torch.int32) - 1).to(dev)


def mla_qk_norm_rope(q=None, k_nope=None, k_rope=None, *, positions, rope_turns, q_nope_weight=None,
                     q_rope_weight=None, k_nope_weight=None, k_rope_weight=None, eps: float = 1e-6,
                     interleaved: bool = True, out=None, stream=None):
    """RMS norms of queries and keys for each head, with the position rotation in the same pass
    (before mla_prefill; queries alone before mla_absorb and the decode calls).

    q [B,S,H,dn+dr], k_nope [B,S,H,dn], k_rope [B,S,dr] bf16, each optional, strided views allowed
    whose last dimension is contiguous and whose B and S dimensions have one stride; weights bf16 (None: that part is not normalised);
    positions [B,S] int32; rope_turns from ``rope_turns()``.  Returns (q_nope [B,S,H,dn],
    q_rope [B,S,H,dr], k_nope, k_rope), contiguous bf16, None for operands not given; ``out``
    may pass those four preallocated."""
    return _call(stream, q if q is not None else k_nope if k_nope is not None else k_rope, _marshal.qk_norm_rope,
                 q, k_nope, k_rope, positions, rope_turns, q_nope_weight, q_rope_weight, k_nope_weight, k_rope_weight,
                 eps, interleaved, out)


def qk_norm_rope_backward_workspace_size(rows: int, H: int) -> int:
    return int(_lib.mla_qk_norm_rope_backward_workspace_size(rows, H))


def mla_qk_norm_rope_backward(dq_nope, dq_rope, dk_nope, dk_rope, q=None, k_nope=None, k_rope=None, *, positions,
                              rope_turns, q_nope_weight=None, q_rope_weight=None, k_nope_weight=None,
                              k_rope_weight=None, eps: float = 1e-6, interleaved: bool = True, grads=None,
                              workspace=None, stream=None):
    """Gradients of mla_qk_norm_rope.  dq_nope, dq_rope, dk_nope bf16 and dk_rope fp32 are the
    upstream gradients as mla_prefill_backward gives them (None where the operand is not given);
    the rest are the forward's arguments.  Returns (dq, dk_nope, dk_rope, dq_nope_weight,
    dq_rope_weight, dk_nope_weight, dk_rope_weight): bf16 with the operands' own strides, the
    weights' in fp32, None for what was not given.  ``grads`` may pass those seven
    preallocated (e.g. dk_nope as a view of a joint key and value gradient)."""
    return _call(stream, q if q is not None else k_nope if k_nope is not None else k_rope,
                 _marshal.qk_norm_rope_backward, q, k_nope, k_rope, positions, rope_turns, q_nope_weight,
                 q_rope_weight, k_nope_weight, k_rope_weight, eps, interleaved, dq_nope, dq_rope, dk_nope, dk_rope,
                 grads, workspace)


def mla_qk_norm_rope_axes(q=None, k_nope=None, k_rope=None, *, positions, rope_turns, q_nope_weight=None,
                          q_rope_weight=None, k_nope_weight=None, k_rope_weight=None, eps: float = 1e-6,
                          interleaved: bool = True, out=None, stream=None):
    """mla_qk_norm_rope with positions on several axes (images, video): positions int32 [B,S,axes],
    rope_turns [axes, dr/2] from ``rope_turns_axes()``; a pair is turned by the sum over the axes of
    position times turns.  Everything else is as for mla_qk_norm_rope."""
    return _call(stream, q if q is not None else k_nope if k_nope is not None else k_rope, _marshal.qk_norm_rope_axes,
                 q, k_nope, k_rope, positions, rope_turns, q_nope_weight, q_rope_weight, k_nope_weight, k_rope_weight,
                 eps, interleaved, out)


def mla_qk_norm_rope_axes_backward(dq_nope, dq_rope, dk_nope, dk_rope, q=None, k_nope=None, k_rope=None, *, positions,
                                   rope_turns, q_nope_weight=None, q_rope_weight=None, k_nope_weight=None,
                                   k_rope_weight=None, eps: float = 1e-6, interleaved: bool = True, grads=None,
                                   workspace=None, stream=None):
    """Gradients of mla_qk_norm_rope_axes.  dk_rope is fp32 (from mla_prefill_backward) or bf16 (from
    mla_cross_attention_backward; with positions on one axis too: positions [B,S,1], rope_turns [1, dr/2]);
    everything else is as for mla_qk_norm_rope_backward."""
    return _call(stream, q if q is not None else k_nope if k_nope is not None else k_rope,
                 _marshal.qk_norm_rope_axes_backward, q, k_nope, k_rope, positions, rope_turns, q_nope_weight,
                 q_rope_weight, k_nope_weight, k_rope_weight, eps, interleaved, dq_nope, dq_rope, dk_nope, dk_rope,
                 grads, workspace)


def mla_rope_append(c_new, kv_cache, page_table, cache_lens, kv_scale=None, *, rope_turns, norm_weight=None,
                    eps: float = 1e-6, positions=None, new_lens=None, interleaved: bool = True, stream=None):
    """mla_cache_append of raw rows c_new [B, q_len, dl+dr] (bf16, strided views allowed
    as for mla_qk_norm_rope): the latent's RMS norm (norm_weight bf16 [dl], None: none)
    and the rope part's rotation are applied on the way.  positions int32 [B, q_len] (None: the
    token's place in its sequence); new_lens int32 [B] (None: q_len): the tokens of each
    sequence that are real, its rows behind them padding.  Modifies kv_cache (and kv_scale) in
    place and returns them."""
    _call(stream, c_new, _marshal.rope_append, c_new, kv_cache, kv_scale, page_table, cache_lens, new_lens, rope_turns,
          norm_weight, eps, positions, interleaved)
    return kv_cache, kv_scale


def mla_rope_append_axes(c_new, kv_cache, page_table, cache_lens, kv_scale=None, *, rope_turns, positions,
                         norm_weight=None, eps: float = 1e-6, new_lens=None, interleaved: bool = True, stream=None):
    """mla_rope_append with positions on several axes: positions int32 [B, q_len, axes], rope_turns
    [axes, dr/2] from ``rope_turns_axes()``.  Everything else is as for mla_rope_append."""
    _call(stream, c_new, _marshal.rope_append_axes, c_new, kv_cache, kv_scale, page_table, cache_lens, new_lens,
          rope_turns, norm_weight, eps, positions, interleaved)
    return kv_cache, kv_scale


def mla_decode_tree(q_latent, q_rope, kv_cache, page_table, cache_lens, tree_mask, kv_scale=None, *, new_lens=None,
                    softmax_scale: float, out=None, lse=None, workspace=None, stream=None):
    """mla_decode for a tree of drafted tokens.  tree_mask int32 words [B, q_len, ceil(q_len/32)],
    or [q_len, ceil(q_len/32)] for the whole batch (``tree_mask_from_parents``): bit j of row t
    says whether token t sees drafted token j; the prefix is seen by all.  new_lens int32 [B]
    (None: q_len): the drafted tokens of each sequence, the newest of its cache; the rows behind
    them are padding (O = 0, LSE = -inf).  The rest is as for mla_decode."""
    return _call(stream, q_latent, _marshal.decode_tree, q_latent, q_rope, kv_cache, kv_scale, page_table, cache_lens,
                 new_lens, tree_mask, softmax_scale, out, lse, workspace)


# ------------------------------------------------- cross attention

def cross_attention_workspace_size(B: int, H: int, Sq: int, Sk: int) -> int:
    return int(_lib.mla_cross_attention_workspace_size(B, H, Sq, Sk))


def mla_cross_attention(q_nope, q_rope, k_nope, k_rope, v, key_lens=None, *, softmax_scale: float, out=None, lse=None,
                        workspace=None, stream=None):
    """Attention to an encoder's states, or any keys of another length.  Returns (out [B,Sq,H,d_v] bf16,
    lse [B,H,Sq] fp32).

    q_nope [B,Sq,H,dn], q_rope [B,Sq,H,dr]; k_nope [B,Sk,H,dn], k_rope [B,Sk,dr], v [B,Sk,H,d_v], all bf16;
    key_lens int32 [B] (None: Sk): the keys of each sequence that exist, what stands behind them does
    not matter; a sequence without keys gives O = 0 and LSE = -inf.  One query a sequence (a decode step)
    and few queries over long keys are cut along the keys.  ``workspace`` may pass
    cross_attention_workspace_size() bytes that the program keeps."""
    return _call(stream, q_nope, _marshal.cross_attention, q_nope, q_rope, k_nope, k_rope, v, key_lens, softmax_scale,
                 out, lse, workspace)


def cross_attention_backward_workspace_size(B: int, H: int, Sq: int, Sk: int) -> int:
    return int(_lib.mla_cross_attention_backward_workspace_size(B, H, Sq, Sk))


def mla_cross_attention_backward(q_nope, q_rope, k_nope, k_rope, v, out, lse, d_out, key_lens=None, *,
                                 softmax_scale: float, grads=None, workspace=None, stream=None):
    """Gradients of mla_cross_attention.  Returns (dq_nope, dq_rope, dk_nope, dk_rope, dv), bf16 in the layouts
    of their operands (dk_rope summed over the heads in fp32), zeros for keys behind a sequence's last.

    out/lse are the forward's results, d_out the upstream gradient [B,Sq,H,d_v] bf16.  ``grads`` may pass
    those five tensors preallocated."""
    return _call(stream, q_nope, _marshal.cross_attention_backward, q_nope, q_rope, k_nope, k_rope, v, key_lens, out,
                 lse, d_out, softmax_scale, grads, workspace)
