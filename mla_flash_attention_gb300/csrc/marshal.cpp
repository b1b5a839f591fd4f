// Argument marshalling of the operators around the attention kernels, compiled: the checks of types,
// shapes, strides and devices, the allocation of outputs and workspaces, and the call of the C
// entry point (include/mla.h).  Nothing is computed here and nothing is kept between calls.  In
// Python the same checks and allocations took 14 to 60 us a call on the GPU's host, several times the
// kernels of a decode step.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <array>
#include <limits>
#include <optional>
#include <string>
#include <vector>

#include "../../include/mla.h"

namespace {

using at::Tensor;
using Shape = std::vector<int64_t>;

// The C entry points of the loaded library and the Python function that raises for a status.
decltype(&mla_qk_norm_rope) f_norm = nullptr;
decltype(&mla_qk_norm_rope_backward) f_grad = nullptr;
decltype(&mla_qk_norm_rope_backward_workspace_size) f_grad_ws = nullptr;
decltype(&mla_rope_append) f_append = nullptr;
decltype(&mla_decode_tree) f_tree = nullptr;
decltype(&mla_decode_workspace_size) f_tree_ws = nullptr;
PyObject* raise_status = nullptr;

[[noreturn]] void fail(PyObject* type, const std::string& msg) {
  PyErr_SetString(type, msg.c_str());
  throw python_error();
}

std::string show(c10::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

std::string show(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
  }
}

const Tensor& tensor(PyObject* o, const char* name, int dims = -1) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + " must be a torch tensor");
  const Tensor& t = THPVariable_Unpack(o);
  if (dims >= 0 && t.dim() != dims)
    fail(PyExc_ValueError, std::string(name) + " must be a tensor of " + std::to_string(dims) + " dimensions");
  return t;
}

// The checks of one tensor; strided: any strides with the last dimension contiguous.
void need(const Tensor& t, const char* name, at::ScalarType dtype, c10::IntArrayRef shape,
          const std::optional<at::Device>& dev, bool strided = false) {
  const std::string n(name);
  if (t.scalar_type() != dtype)
    fail(PyExc_TypeError, n + " must have dtype " + show(dtype) + " (got " + show(t.scalar_type()) + ")");
  if (t.sizes() != shape) fail(PyExc_ValueError, n + " must have shape " + show(shape) + " (got " + show(t.sizes()) + ")");
  if (!t.is_cuda()) fail(PyExc_ValueError, n + " must be a CUDA tensor");
  if (dev && t.device() != *dev) fail(PyExc_ValueError, n + " must be on " + dev->str() + " (got " + t.device().str() + ")");
  if (strided) {
    if (t.size(-1) != 1 && t.stride(-1) != 1) fail(PyExc_ValueError, n + " must have a contiguous last dimension");
  } else if (!t.is_contiguous()) {
    fail(PyExc_ValueError, n + " must be contiguous");
  }
}

void* ptr(const Tensor& t) { return t.defined() ? const_cast<void*>(t.const_data_ptr()) : nullptr; }

// An optional tensor argument: undefined for None.
Tensor optional(PyObject* o, const char* name, int dims = -1) { return o == Py_None ? Tensor() : tensor(o, name, dims); }

// A workspace passed in: contiguous bytes on the device of the call.
void scratch(const Tensor& t, const at::Device& dev) {
  if (t.device() != dev || !t.is_contiguous())
    fail(PyExc_ValueError, "workspace must be a contiguous tensor on " + dev.str());
}

// Elements from one token of t [B, S, ...] to the next, over all B * S tokens.
int64_t row_stride(const Tensor& t, const char* name) {
  const int64_t B = t.size(0), S = t.size(1), sb = t.stride(0), ss = t.stride(1);
  if (S == 1) return B > 1 ? sb : t.size(-1);  // a single token's strides may be anything
  if (B > 1 && sb != S * ss)
    fail(PyExc_ValueError, std::string(name) + ": the B and S dimensions must have one stride (got " +
                               std::to_string(sb) + " and " + std::to_string(ss) + ")");
  return ss;
}

Tensor empty(c10::IntArrayRef shape, at::ScalarType dtype, const at::Device& dev) {
  return at::detail::empty_cuda(shape, dtype, dev, std::nullopt);
}

// A size as the C entry points take it.  One past an int's range is one that they refuse, not its low bits.
int size_arg(int64_t v) { return static_cast<int>(std::min<int64_t>(v, std::numeric_limits<int>::max())); }

void* stream_of(const at::Device& dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// Raises for a status that is not MLA_OK (the library's message is the calling thread's).
void check(mla_status st) {
  if (st == MLA_OK) return;
  PyObject* r = PyObject_CallFunction(raise_status, "i", static_cast<int>(st));
  Py_XDECREF(r);
  if (r) PyErr_SetString(PyExc_RuntimeError, "a call failed without a message");
  throw python_error();
}

template <typename F>
mla_status unlocked(F&& f) {
  mla_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

PyObject* wrap_all(const Tensor* t, Py_ssize_t n) {
  PyObject* r = PyTuple_New(n);
  if (!r) throw python_error();
  for (Py_ssize_t i = 0; i < n; ++i) PyTuple_SET_ITEM(r, i, wrap(t[i]));
  return r;
}

// Member i of a list or tuple of n passed in.
PyObject* member(PyObject* seq, const char* name, Py_ssize_t n, Py_ssize_t i) {
  if ((!PyTuple_Check(seq) && !PyList_Check(seq)) || PySequence_Fast_GET_SIZE(seq) != n)
    fail(PyExc_ValueError, std::string(name) + " must hold " + std::to_string(n) + " tensors (None for those not given)");
  return PySequence_Fast_GET_ITEM(seq, i);
}

// ------------------------------------------------------------------ the norm-and-rotation calls

const char* const kWeightNames[4] = {"q_nope_weight", "q_rope_weight", "k_nope_weight", "k_rope_weight"};

struct Operands {
  Tensor q, kn, kr, pos, turns, w[4];
  int64_t B = 0, S = 0, H = 1, dn = 128, dr = 64;
  int64_t q_row = 0, q_head = 0, kn_row = 0, kn_head = 0, kr_row = 0;
  at::Device dev{at::kCPU};
  Shape q_shape() const { return {B, S, H, dn + dr}; }
  Shape nope_shape() const { return {B, S, H, dn}; }
  Shape rope_shape() const { return {B, S, H, dr}; }
  Shape key_shape() const { return {B, S, dr}; }

  // q, k_nope, k_rope, positions, rope_turns, four weights
  explicit Operands(PyObject* const* a) {
    if (a[0] == Py_None && a[1] == Py_None && a[2] == Py_None)
      fail(PyExc_ValueError, "one of q, k_nope, k_rope must be given");
    q = optional(a[0], "q", 4);
    kn = optional(a[1], "k_nope", 4);
    kr = optional(a[2], "k_rope", 3);
    turns = tensor(a[4], "rope_turns", 1);
    const Tensor& some = q.defined() ? q : kn.defined() ? kn : kr;
    B = some.size(0);
    S = some.size(1);
    if (some.dim() == 4) H = some.size(2);
    dr = 2 * turns.size(0);
    if (q.defined()) dn = q.size(3) - dr;
    else if (kn.defined()) dn = kn.size(3);
    dev = some.device();
    const auto stride = [&](const Tensor& t, const char* name, const Shape& shape, int64_t& row, int64_t* head) {
      if (!t.defined()) return;
      need(t, name, at::kBFloat16, shape, dev, true);
      row = row_stride(t, name);
      if (head) *head = H > 1 ? t.stride(2) : t.size(3);
    };
    stride(q, "q", q_shape(), q_row, &q_head);
    stride(kn, "k_nope", nope_shape(), kn_row, &kn_head);
    stride(kr, "k_rope", key_shape(), kr_row, nullptr);
    pos = tensor(a[3], "positions");
    need(pos, "positions", at::kInt, {B, S}, dev);
    need(turns, "rope_turns", at::kLong, {dr / 2}, dev);
    for (int i = 0; i < 4; ++i) {
      w[i] = optional(a[5 + i], kWeightNames[i]);
      if (w[i].defined()) need(w[i], kWeightNames[i], at::kBFloat16, {i % 2 ? dr : dn}, dev);
    }
  }
};

// (q, k_nope, k_rope, positions, rope_turns, 4 weights, eps, interleaved, out or None)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12) fail(PyExc_TypeError, "qk_norm_rope takes 12 arguments");
  const Operands o(a);
  const c10::cuda::CUDAGuard guard(o.dev);
  const bool given[4] = {o.q.defined(), o.q.defined(), o.kn.defined(), o.kr.defined()};
  const Shape shapes[4] = {o.nope_shape(), o.rope_shape(), o.nope_shape(), o.key_shape()};
  const char* const names[4] = {"out[0]", "out[1]", "out[2]", "out[3]"};
  Tensor out[4];
  for (int i = 0; i < 4; ++i) {
    if (!given[i]) continue;
    if (a[11] == Py_None) {
      out[i] = empty(shapes[i], at::kBFloat16, o.dev);
    } else {
      out[i] = tensor(member(a[11], "out", 4, i), names[i]);
      need(out[i], names[i], at::kBFloat16, shapes[i], o.dev);
    }
  }
  const float eps = static_cast<float>(number(a[9]));
  const int il = truth(a[10]);
  void* st = stream_of(o.dev);
  check(unlocked([&] {
    return f_norm(ptr(o.q), o.q_row, o.q_head, ptr(o.kn), o.kn_row, o.kn_head, ptr(o.kr), o.kr_row, ptr(o.w[0]),
                  ptr(o.w[1]), ptr(o.w[2]), ptr(o.w[3]), static_cast<const int*>(ptr(o.pos)), ptr(o.turns), eps, il,
                  ptr(out[0]), ptr(out[1]), ptr(out[2]), ptr(out[3]), o.B * o.S, size_arg(o.H),
                  size_arg(o.dn), size_arg(o.dr), st);
  }));
  return wrap_all(out, 4);
  END_HANDLE_TH_ERRORS
}

// (q, k_nope, k_rope, positions, rope_turns, 4 weights, eps, interleaved, dq_nope, dq_rope, dk_nope,
//  dk_rope, grads or None, workspace or None)
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 17) fail(PyExc_TypeError, "qk_norm_rope_backward takes 17 arguments");
  const Operands o(a);
  const c10::cuda::CUDAGuard guard(o.dev);
  const bool has_up[4] = {o.q.defined(), o.q.defined(), o.kn.defined(), o.kr.defined()};
  const Shape up_shapes[4] = {o.nope_shape(), o.rope_shape(), o.nope_shape(), o.key_shape()};
  const char* const up_names[4] = {"dq_nope", "dq_rope", "dk_nope", "dk_rope"};
  Tensor up[4];
  for (int i = 0; i < 4; ++i) {
    if (!has_up[i]) continue;
    up[i] = tensor(a[11 + i], up_names[i]);
    need(up[i], up_names[i], i == 3 ? at::kFloat : at::kBFloat16, up_shapes[i], o.dev);
  }
  const Tensor* given[7] = {&o.q, &o.kn, &o.kr, &o.w[0], &o.w[1], &o.w[2], &o.w[3]};
  const char* const names[7] = {"grads[0]", "grads[1]", "grads[2]", "grads[3]", "grads[4]", "grads[5]", "grads[6]"};
  Tensor g[7];
  bool weights = false;
  for (int i = 0; i < 7; ++i) {
    const Tensor& of = *given[i];
    if (a[15] != Py_None) member(a[15], "grads", 7, i);
    if (!of.defined()) continue;
    weights |= i >= 3;
    const at::ScalarType dtype = i < 3 ? at::kBFloat16 : at::kFloat;
    if (a[15] == Py_None) {
      g[i] = i < 3 && !of.is_contiguous()
                 ? at::empty_strided(of.sizes(), of.strides(), at::TensorOptions().dtype(dtype).device(o.dev))
                 : empty(of.sizes(), dtype, o.dev);
      continue;
    }
    g[i] = tensor(member(a[15], "grads", 7, i), names[i]);
    need(g[i], names[i], dtype, of.sizes(), o.dev, i < 3);
    for (int64_t d = 0; i < 3 && d < of.dim(); ++d)
      if (of.size(d) > 1 && of.stride(d) != g[i].stride(d))
        fail(PyExc_ValueError, std::string(names[i]) + " must have its operand's strides");
  }
  Tensor ws = optional(a[16], "workspace");
  if (ws.defined()) scratch(ws, o.dev);
  else if (weights)
    ws = empty({std::max<int64_t>(static_cast<int64_t>(f_grad_ws(o.B * o.S, size_arg(o.H))), 16)}, at::kByte, o.dev);
  const size_t ws_bytes = ws.defined() ? ws.nbytes() : 0;
  const float eps = static_cast<float>(number(a[9]));
  const int il = truth(a[10]);
  void* st = stream_of(o.dev);
  const auto f32 = [](const Tensor& t) { return static_cast<float*>(ptr(t)); };
  check(unlocked([&] {
    return f_grad(ptr(up[0]), ptr(up[1]), ptr(up[2]), f32(up[3]), ptr(o.q), o.q_row, o.q_head, ptr(o.kn), o.kn_row,
                  o.kn_head, ptr(o.kr), o.kr_row, ptr(o.w[0]), ptr(o.w[1]), ptr(o.w[2]), ptr(o.w[3]),
                  static_cast<const int*>(ptr(o.pos)), ptr(o.turns), eps, il, ptr(g[0]), ptr(g[1]), ptr(g[2]),
                  f32(g[3]), f32(g[4]), f32(g[5]), f32(g[6]), o.B * o.S, size_arg(o.H),
                  size_arg(o.dn), size_arg(o.dr), ptr(ws), ws_bytes, st);
  }));
  return wrap_all(g, 7);
  END_HANDLE_TH_ERRORS
}

// -------------------------------------------------------------------------- the paged cache

struct Cache {
  Tensor kv, scale, table, lens, fresh;
  int64_t pages, page_size, max_pages;
  bool fp8;
  // kv_cache, kv_scale, page_table, cache_lens, new_lens of a call on B sequences, rows of D
  Cache(PyObject* const* a, int64_t B, int64_t D, const at::Device& dev) {
    kv = tensor(a[0], "kv_cache", 3);
    pages = kv.size(0);
    page_size = kv.size(1);
    fp8 = kv.scalar_type() == at::kFloat8_e4m3fn;
    need(kv, "kv_cache", fp8 ? at::kFloat8_e4m3fn : at::kBFloat16, {pages, page_size, D}, dev);
    if (fp8) {
      scale = tensor(a[1], "kv_scale");
      need(scale, "kv_scale", at::kFloat, {pages, page_size}, dev);
    } else if (a[1] != Py_None) {
      fail(PyExc_ValueError, "kv_scale is only used with an fp8 cache");
    }
    table = tensor(a[2], "page_table", 2);
    max_pages = table.size(1);
    need(table, "page_table", at::kInt, {B, max_pages}, dev);
    lens = tensor(a[3], "cache_lens");
    need(lens, "cache_lens", at::kInt, {B}, dev);
    fresh = optional(a[4], "new_lens");
    if (fresh.defined()) need(fresh, "new_lens", at::kInt, {B}, dev);
  }
  mla_dtype type() const { return fp8 ? MLA_FP8_E4M3 : MLA_BF16; }
};

const int* ints(const Tensor& t) { return static_cast<const int*>(ptr(t)); }

// (c_new, kv_cache, kv_scale, page_table, cache_lens, new_lens, rope_turns, norm_weight, eps,
//  positions, interleaved)
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 11) fail(PyExc_TypeError, "rope_append takes 11 arguments");
  const Tensor& c = tensor(a[0], "c_new", 3);
  const int64_t B = c.size(0), T = c.size(1), D = c.size(2);
  need(c, "c_new", at::kBFloat16, {B, T, D}, std::nullopt, true);
  const at::Device dev = c.device();
  const Cache k(a + 1, B, D, dev);
  const Tensor& turns = tensor(a[6], "rope_turns", 1);
  const int64_t dr = 2 * turns.size(0);
  need(turns, "rope_turns", at::kLong, {dr / 2}, dev);
  const Tensor w = optional(a[7], "norm_weight"), pos = optional(a[9], "positions");
  if (w.defined()) need(w, "norm_weight", at::kBFloat16, {D - dr}, dev);
  if (pos.defined()) need(pos, "positions", at::kInt, {B, T}, dev);
  const c10::cuda::CUDAGuard guard(dev);
  const int64_t stride = row_stride(c, "c_new");
  const float eps = static_cast<float>(number(a[8]));
  const int il = truth(a[10]);
  void* st = stream_of(dev);
  check(unlocked([&] {
    return f_append(ptr(c), stride, ptr(w), eps, ints(pos), ptr(turns), il, ptr(k.kv), static_cast<float*>(ptr(k.scale)),
                    ints(k.table), ints(k.lens), ints(k.fresh), size_arg(B), size_arg(T),
                    size_arg(D - dr), size_arg(dr), size_arg(k.page_size),
                    size_arg(k.max_pages), size_arg(k.pages), k.type(), st);
  }));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (q_latent, q_rope, kv_cache, kv_scale, page_table, cache_lens, new_lens, tree_mask, softmax_scale,
//  out, lse, workspace)
PyObject* decode_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12) fail(PyExc_TypeError, "decode_tree takes 12 arguments");
  const Tensor &ql = tensor(a[0], "q_latent", 4), &qr = tensor(a[1], "q_rope", 4);
  const int64_t B = ql.size(0), T = ql.size(1), H = ql.size(2), dl = ql.size(3), dr = qr.size(3);
  need(ql, "q_latent", at::kBFloat16, {B, T, H, dl}, std::nullopt);
  const at::Device dev = ql.device();
  need(qr, "q_rope", at::kBFloat16, {B, T, H, dr}, dev);
  const Cache k(a + 2, B, dl + dr, dev);
  const Tensor& mask = tensor(a[7], "tree_mask");
  const int64_t words = (T + 31) / 32;
  const bool shared = mask.dim() == 2;
  need(mask, "tree_mask", at::kInt, shared ? Shape{T, words} : Shape{B, T, words}, dev);
  const float scale = static_cast<float>(number(a[8]));
  const c10::cuda::CUDAGuard guard(dev);
  Tensor out = optional(a[9], "out"), lse = optional(a[10], "lse"), ws = optional(a[11], "workspace");
  if (out.defined()) need(out, "out", at::kBFloat16, {B, T, H, dl}, dev);
  else out = empty({B, T, H, dl}, at::kBFloat16, dev);
  if (lse.defined()) need(lse, "lse", at::kFloat, {B, H, T}, dev);
  else lse = empty({B, H, T}, at::kFloat, dev);
  if (ws.defined()) scratch(ws, dev);
  else
    ws = empty({std::max<int64_t>(static_cast<int64_t>(f_tree_ws(size_arg(B), size_arg(H),
                                                                 size_arg(T), size_arg(dl))), 16)},
               at::kByte, dev);
  void* st = stream_of(dev);
  check(unlocked([&] {
    return f_tree(ptr(ql), ptr(qr), ptr(k.kv), static_cast<const float*>(ptr(k.scale)), ints(k.table), ints(k.lens),
                  ptr(mask), shared ? 0 : T * words, ints(k.fresh), ptr(out), static_cast<float*>(ptr(lse)),
                  size_arg(B), size_arg(H), size_arg(T), size_arg(dl),
                  size_arg(dr), size_arg(k.page_size), size_arg(k.max_pages),
                  size_arg(k.pages), scale, k.type(), ptr(ws), ws.nbytes(), st);
  }));
  const Tensor res[2] = {out, lse};
  return wrap_all(res, 2);
  END_HANDLE_TH_ERRORS
}

// connect(addresses of the six C functions, the function that raises for a status)
PyObject* connect(PyObject*, PyObject* args) {
  unsigned long long f[6];
  PyObject* raise;
  if (!PyArg_ParseTuple(args, "KKKKKKO", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &raise)) return nullptr;
  f_norm = reinterpret_cast<decltype(f_norm)>(f[0]);
  f_grad = reinterpret_cast<decltype(f_grad)>(f[1]);
  f_grad_ws = reinterpret_cast<decltype(f_grad_ws)>(f[2]);
  f_append = reinterpret_cast<decltype(f_append)>(f[3]);
  f_tree = reinterpret_cast<decltype(f_tree)>(f[4]);
  f_tree_ws = reinterpret_cast<decltype(f_tree_ws)>(f[5]);
  Py_INCREF(raise);
  Py_XSETREF(raise_status, raise);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {{"connect", connect, METH_VARARGS, nullptr},
                         {"qk_norm_rope", fast<qk_norm_rope>(), METH_FASTCALL, nullptr},
                         {"qk_norm_rope_backward", fast<qk_norm_rope_backward>(), METH_FASTCALL, nullptr},
                         {"rope_append", fast<rope_append>(), METH_FASTCALL, nullptr},
                         {"decode_tree", fast<decode_tree>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
