// The operators over torch tensors: a CPython extension module that checks
// arguments, allocates results and workspaces, and calls the C ABI on the
// current stream. No arithmetic happens here.
//
// It exists for the smallest calls. Their kernels take a few microseconds;
// reading seven tensors' types, sizes and strides from Python takes ten.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <optional>

#include "muon_adamw.h"

namespace {

using at::Tensor;

// A refusal with a Python exception of its own type, raised where the C++ exception ends.
struct Refused {};

[[noreturn]] void refuse(PyObject* type, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(type, fmt, ap);
  va_end(ap);
  throw Refused();
}

PyObject* g_check = nullptr;  // the package's _check(status): raises MuonAdamWError with the library's message

void check(ma_status st) {
  if (st == MA_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "i", (int)st);
  Py_XDECREF(r);
  if (r) PyErr_Format(PyExc_RuntimeError, "status %d", (int)st);
  throw Refused();
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor, not %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// A tensor on the first one's device.
const Tensor& tensor(PyObject* o, const char* name, const Tensor& first) {
  const Tensor& t = tensor(o, name);
  if (t.device() != first.device())
    refuse(PyExc_ValueError, "%s is on %s, not %s", name, t.device().str().c_str(), first.device().str().c_str());
  return t;
}

void need_cuda(const Tensor& t) {
  if (!t.is_cuda())
    refuse(PyExc_ValueError, "the operators take CUDA tensors, not %s ones", t.device().str().c_str());
}

int dtype_of(const Tensor& t, const char* name) {
  const at::ScalarType s = t.scalar_type();
  if (s == at::kBFloat16) return MA_DT_BF16;
  if (s == at::kFloat) return MA_DT_F32;
  refuse(PyExc_TypeError, "%s must be fp32 or bf16, not %s", name, c10::toString(s));
}

int int_bytes(const Tensor& t, const char* name) {
  const at::ScalarType s = t.scalar_type();
  if (s == at::kLong) return 8;
  if (s == at::kInt) return 4;
  refuse(PyExc_TypeError, "%s must be int32 or int64, not %s", name, c10::toString(s));
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}

// A number past 64 bits counts as the largest, or the smallest, of them.
int64_t integer(PyObject* o) {
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (over) return over > 0 ? INT64_MAX : INT64_MIN;
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v != 0;
}

Tensor make(at::IntArrayRef size, at::ScalarType type, const Tensor& like) {
  return at::detail::empty_cuda(size, type, like.device(), std::nullopt);
}

void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

// f(stream) on the tensor's device, without the interpreter's lock.
template <typename F>
void call(const Tensor& t, F f) {
  void* s = stream_of(t);
  ma_status st;
  PyThreadState* state = PyEval_SaveThread();
  {
    c10::cuda::OptionalCUDAGuard guard(t.device());
    st = f(s);
  }
  PyEval_RestoreThread(state);
  check(st);
}

// A tensor's own contiguous copy where it is not contiguous.
Tensor packed(const Tensor& t) { return t.is_contiguous() ? t : t.detach().contiguous(); }

// ---- embedding ----

struct Rows {
  int64_t vocab, width, stride;
};
Rows table_of(const Tensor& t, const char* name) {
  if (t.dim() != 2) refuse(PyExc_ValueError, "%s must be [vocab, width], not of %d dimensions", name, (int)t.dim());
  if (t.size(1) > 1 && t.stride(1) != 1)
    refuse(PyExc_ValueError, "%s must have consecutive elements in a row", name);
  return {t.size(0), t.size(1), t.size(0) > 1 ? t.stride(0) : t.size(1)};
}

PyObject* embedding(PyObject* const* a) {
  const Tensor& weight = tensor(a[0], "weight");
  need_cuda(weight);
  const Tensor ids = packed(tensor(a[1], "ids", weight));
  const Rows w = table_of(weight, "weight");
  const int wdt = dtype_of(weight, "weight"), ib = int_bytes(ids, "ids");
  const double scale = real(a[2]);
  at::ScalarType type = weight.scalar_type();
  if (a[3] != Py_None) {
    if (!THPDtype_Check(a[3])) refuse(PyExc_TypeError, "dtype must be a torch.dtype");
    type = reinterpret_cast<THPDtype*>(a[3])->scalar_type;
  }
  c10::SmallVector<int64_t, 5> size(ids.sizes().begin(), ids.sizes().end());
  size.push_back(w.width);
  Tensor out = make(size, type, weight);
  const int odt = dtype_of(out, "the result");
  call(weight, [&](void* s) {
    return muon_adamw_embedding(weight.const_data_ptr(), wdt, w.stride, w.vocab, w.width, ids.const_data_ptr(), ib,
                                ids.numel(), scale, out.mutable_data_ptr(), odt, w.width, s);
  });
  return THPVariable_Wrap(std::move(out));
}

PyObject* embedding_backward(PyObject* const* a) {
  const Tensor& grad = tensor(a[2], "grad");
  need_cuda(grad);
  const Tensor ids = packed(tensor(a[1], "ids", grad));
  Tensor dout = tensor(a[0], "dout", grad);
  const Rows g = table_of(grad, "grad");
  const int gdt = dtype_of(grad, "grad"), ddt = dtype_of(dout, "dout"), ib = int_bytes(ids, "ids");
  if (dout.dim() != ids.dim() + 1 || dout.sizes().slice(0, ids.dim()) != ids.sizes())
    refuse(PyExc_ValueError, "dout does not have the shape of ids and one dimension more");
  if (dout.size(-1) != g.width)
    refuse(PyExc_ValueError, "dout has rows of %lld elements, not %lld", (long long)dout.size(-1), (long long)g.width);
  int64_t dstride = g.width;
  if (!dout.is_contiguous()) {
    if (dout.dim() == 2 && dout.stride(1) == 1 && dout.stride(0) >= g.width)
      dstride = dout.stride(0);
    else
      dout = packed(dout);
  }
  const double scale = real(a[3]);
  const int acc = truth(a[4]);
  const int64_t n = ids.numel();
  int64_t bytes = 0;
  check(muon_adamw_embedding_backward_workspace(n, g.vocab, g.width, &bytes));
  Tensor ws = make({bytes}, at::kByte, grad);
  call(grad, [&](void* s) {
    return muon_adamw_embedding_backward(dout.const_data_ptr(), ddt, dstride, ids.const_data_ptr(), ib, n, scale,
                                         grad.mutable_data_ptr(), gdt, g.stride, g.vocab, g.width, acc,
                                         ws.mutable_data_ptr(), bytes, s);
  });
  // as any write in place: a graph that saved the tensor is to notice (inference tensors count no versions)
  if (!grad.is_inference()) grad.unsafeGetTensorImpl()->bump_version();
  return Py_NewRef(a[2]);
}

// ---- queries and keys ----

// [token, head, head_dim] with consecutive elements in a head; the stride of a
// single token or head says nothing and counts as 0. apart: no two heads on the
// same elements, as in an expanded tensor.
struct Heads {
  Tensor t;
  int64_t n, h, d, ts, hs;
};
Heads heads_of(const Tensor& t, const char* name, bool apart) {
  if (t.dim() != 3)
    refuse(PyExc_ValueError, "%s must be [token, head, head_dim], not of %d dimensions", name, (int)t.dim());
  Heads r{t, t.size(0), t.size(1), t.size(2), 0, 0};
  const bool loose = (r.d > 1 && t.stride(2) != 1) ||
                     (apart && ((r.n > 1 && t.stride(0) < r.d) || (r.h > 1 && t.stride(1) < r.d)));
  if (loose) r.t = t.detach().contiguous();
  r.ts = r.n > 1 ? r.t.stride(0) : 0;
  r.hs = r.h > 1 ? r.t.stride(1) : 0;
  return r;
}

// The same with every row on a 16-byte boundary, by a copy where one is not. For
// gradients and saved outputs: autograd chooses their layout (a slice of a wider
// row, say), and a caller of a backward pass can do nothing about it.
Heads aligned_heads(const Tensor& t, const char* name, bool apart) {
  Heads r = heads_of(t, name, apart);
  const int64_t e = (int64_t)r.t.element_size();
  if (r.ts * e % 16 || r.hs * e % 16 || reinterpret_cast<uintptr_t>(r.t.const_data_ptr()) % 16)
    r = heads_of(r.t.detach().clone(at::MemoryFormat::Contiguous), name, apart);
  return r;
}

struct Qk {
  Heads q, k;
  Tensor keep[5];
  ma_qk_norm_rope d;
};

// a: q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours
void read_qk(Qk& r, PyObject* const* a) {
  const Tensor& q = tensor(a[0], "q");
  need_cuda(q);
  r.q = heads_of(q, "q", false);
  r.k = heads_of(tensor(a[1], "k", q), "k", false);
  if (r.k.d != r.q.d || r.k.n != r.q.n) refuse(PyExc_ValueError, "q and k differ in tokens or head_dim");
  if (r.k.t.scalar_type() != q.scalar_type()) refuse(PyExc_TypeError, "q and k differ in type");
  static const char* const names[5] = {"q_weight", "k_weight", "cos", "sin", "positions"};
  for (int i = 0; i < 5; ++i) {
    r.keep[i] = tensor(a[2 + i], names[i], q);
    if (i < 4 && r.keep[i].scalar_type() != at::kFloat) refuse(PyExc_ValueError, "%s must be fp32", names[i]);
    if (!r.keep[i].is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", names[i]);
    if (i < 2 && (r.keep[i].dim() != 1 || r.keep[i].size(0) != r.q.d))
      refuse(PyExc_ValueError, "%s must be %lld values", names[i], (long long)r.q.d);
  }
  const Tensor &cos = r.keep[2], &sin = r.keep[3], &pos = r.keep[4];
  if (cos.dim() != 2 || cos.sizes() != sin.sizes())
    refuse(PyExc_ValueError, "cos and sin must be tables of one shape [position, rotated pairs]");
  const int pb = int_bytes(pos, "positions");
  if (pos.dim() != 1 || pos.size(0) != r.q.n)
    refuse(PyExc_ValueError, "positions must be %lld values", (long long)r.q.n);
  ma_qk_norm_rope& d = r.d;
  d.n_tokens = r.q.n;
  d.n_heads = (int32_t)r.q.h;
  d.n_kv_heads = (int32_t)r.k.h;
  d.head_dim = (int32_t)r.q.d;
  d.rot_dim = (int32_t)(2 * cos.size(1));
  d.dtype = dtype_of(q, "q");
  d.eps = real(a[7]);
  d.neighbours = truth(a[8]);
  d.position_bytes = pb;
  d.reserved = 0;
  d.q = r.q.t.const_data_ptr();
  d.k = r.k.t.const_data_ptr();
  d.q_token_stride = r.q.ts;
  d.q_head_stride = r.q.hs;
  d.k_token_stride = r.k.ts;
  d.k_head_stride = r.k.hs;
  d.q_weight = static_cast<const float*>(r.keep[0].const_data_ptr());
  d.k_weight = static_cast<const float*>(r.keep[1].const_data_ptr());
  d.cos_table = static_cast<const float*>(cos.const_data_ptr());
  d.sin_table = static_cast<const float*>(sin.const_data_ptr());
  d.table_rows = cos.size(0);
  d.positions = pos.const_data_ptr();
}

PyObject* qk_norm_rope(PyObject* const* a) {
  Qk x;
  read_qk(x, a);
  const at::ScalarType type = x.q.t.scalar_type();
  Tensor qo = make(x.q.t.sizes(), type, x.q.t), ko = make(x.k.t.sizes(), type, x.q.t);
  call(x.q.t, [&](void* s) { return muon_adamw_qk_norm_rope(&x.d, qo.mutable_data_ptr(), ko.mutable_data_ptr(), s); });
  return Py_BuildValue("NN", THPVariable_Wrap(std::move(qo)), THPVariable_Wrap(std::move(ko)));
}

// a: dq_out, dk_out, then as read_qk()
PyObject* qk_norm_rope_backward(PyObject* const* a) {
  Qk x;
  read_qk(x, a + 2);
  const Tensor& q = x.q.t;
  const at::ScalarType type = q.scalar_type();
  const Heads dqo = aligned_heads(tensor(a[0], "dq_out", q), "dq_out", false);
  const Heads dko = aligned_heads(tensor(a[1], "dk_out", q), "dk_out", false);
  if (dqo.t.sizes() != q.sizes() || dko.t.sizes() != x.k.t.sizes() || dqo.t.scalar_type() != type ||
      dko.t.scalar_type() != type)
    refuse(PyExc_ValueError, "dq_out and dk_out must have the shapes and the type of q and k");
  int64_t bytes = 0;
  ma_status st;
  {
    c10::cuda::OptionalCUDAGuard guard(q.device());
    st = muon_adamw_qk_norm_rope_backward_workspace(&x.d, &bytes);
  }
  check(st);
  Tensor ws = make({bytes}, at::kByte, q), dq = make(q.sizes(), type, q), dk = make(x.k.t.sizes(), type, q);
  Tensor dqw = make({x.q.d}, at::kFloat, q), dkw = make({x.q.d}, at::kFloat, q);
  call(q, [&](void* s) {
    return muon_adamw_qk_norm_rope_backward(
        &x.d, dqo.t.const_data_ptr(), dqo.ts, dqo.hs, dko.t.const_data_ptr(), dko.ts, dko.hs, dq.mutable_data_ptr(),
        dk.mutable_data_ptr(), static_cast<float*>(dqw.mutable_data_ptr()), static_cast<float*>(dkw.mutable_data_ptr()),
        ws.mutable_data_ptr(), bytes, s);
  });
  return Py_BuildValue("NNNN", THPVariable_Wrap(std::move(dq)), THPVariable_Wrap(std::move(dk)),
                       THPVariable_Wrap(std::move(dqw)), THPVariable_Wrap(std::move(dkw)));
}

// ---- attention ----

struct Attn {
  Heads q, k, v;
  Tensor cu;
  ma_window_attention d;
};

// a: q, k, v, then o: window or None, sinks, scale or None, cu_seqlens or None
void read_attention(Attn& r, PyObject* const* a, PyObject* const* o) {
  const Tensor& q = tensor(a[0], "q");
  need_cuda(q);
  r.q = heads_of(q, "q", true);
  r.k = heads_of(tensor(a[1], "k", q), "k", true);
  r.v = heads_of(tensor(a[2], "v", q), "v", true);
  if (r.k.d != r.q.d || r.k.n != r.q.n || r.v.t.sizes() != r.k.t.sizes())
    refuse(PyExc_ValueError, "the shapes of q, k and v do not fit together");
  if (q.scalar_type() != at::kBFloat16 || r.k.t.scalar_type() != at::kBFloat16 || r.v.t.scalar_type() != at::kBFloat16)
    refuse(PyExc_TypeError, "q, k and v must be bf16");
  ma_window_attention& d = r.d;
  d.cu_seqlens = nullptr;
  d.n_seqs = 0;
  if (o[3] != Py_None) {
    r.cu = tensor(o[3], "cu_seqlens", q);
    if (r.cu.scalar_type() != at::kInt || r.cu.dim() != 1 || r.cu.size(0) < 2 || !r.cu.is_contiguous())
      refuse(PyExc_ValueError, "cu_seqlens must be at least 2 contiguous int32 values");
    d.cu_seqlens = static_cast<const int32_t*>(r.cu.const_data_ptr());
    d.n_seqs = (int32_t)(r.cu.size(0) - 1);
  }
  d.n_tokens = r.q.n;
  d.n_heads = (int32_t)r.q.h;
  d.n_kv_heads = (int32_t)r.k.h;
  d.head_dim = (int32_t)r.q.d;
  d.window = o[0] == Py_None ? r.q.n : integer(o[0]);
  const int64_t sinks = integer(o[1]);
  d.sinks = (int32_t)(sinks < -1 ? -1 : sinks > 1 << 20 ? 1 << 20 : sinks);  // out of range either way
  d.scale = o[2] == Py_None ? 1.0 / std::sqrt((double)r.q.d) : real(o[2]);
  d.reserved = 0;
  d.q = r.q.t.const_data_ptr();
  d.k = r.k.t.const_data_ptr();
  d.v = r.v.t.const_data_ptr();
  d.q_token_stride = r.q.ts;
  d.q_head_stride = r.q.hs;
  d.k_token_stride = r.k.ts;
  d.k_head_stride = r.k.hs;
  d.v_token_stride = r.v.ts;
  d.v_head_stride = r.v.hs;
  d.out_token_stride = d.out_head_stride = 0;
}

PyObject* window_attention(PyObject* const* a) {
  Attn x;
  read_attention(x, a, a + 3);
  Tensor out = make(x.q.t.sizes(), at::kBFloat16, x.q.t), lse = make({x.q.h, x.q.n}, at::kFloat, x.q.t);
  call(x.q.t, [&](void* s) {
    return muon_adamw_window_attention(&x.d, out.mutable_data_ptr(), static_cast<float*>(lse.mutable_data_ptr()), s);
  });
  return Py_BuildValue("NN", THPVariable_Wrap(std::move(out)), THPVariable_Wrap(std::move(lse)));
}

// a: dout, q, k, v, out, lse, then as read_attention()'s o
PyObject* window_attention_backward(PyObject* const* a) {
  Attn x;
  read_attention(x, a + 1, a + 6);
  const Tensor& q = x.q.t;
  const Heads dout = aligned_heads(tensor(a[0], "dout", q), "dout", true);
  const Heads out = aligned_heads(tensor(a[4], "out", q), "out", true);
  const Tensor& lse = tensor(a[5], "lse", q);
  if (dout.t.sizes() != q.sizes() || out.t.sizes() != q.sizes() || dout.t.scalar_type() != at::kBFloat16 ||
      out.t.scalar_type() != at::kBFloat16)
    refuse(PyExc_ValueError, "dout and out must have the shape and the type of q");
  if (lse.dim() != 2 || lse.size(0) != x.q.h || lse.size(1) != x.q.n || lse.scalar_type() != at::kFloat ||
      !lse.is_contiguous())
    refuse(PyExc_ValueError, "lse must be contiguous fp32 [head, token]");
  x.d.out_token_stride = out.ts;
  x.d.out_head_stride = out.hs;
  int64_t bytes = 0;
  check(muon_adamw_window_attention_backward_workspace(&x.d, &bytes));
  Tensor ws = make({bytes}, at::kByte, q), dq = make(q.sizes(), at::kBFloat16, q);
  Tensor dk = make(x.k.t.sizes(), at::kBFloat16, q), dv = make(x.k.t.sizes(), at::kBFloat16, q);
  call(q, [&](void* s) {
    return muon_adamw_window_attention_backward(&x.d, dout.t.const_data_ptr(), dout.ts, dout.hs, out.t.const_data_ptr(),
                                                static_cast<const float*>(lse.const_data_ptr()), dq.mutable_data_ptr(),
                                                dk.mutable_data_ptr(), dv.mutable_data_ptr(), ws.mutable_data_ptr(),
                                                bytes, s);
  });
  return Py_BuildValue("NNN", THPVariable_Wrap(std::move(dq)), THPVariable_Wrap(std::move(dk)),
                       THPVariable_Wrap(std::move(dv)));
}

// ---- module ----

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyCFunction method() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>));
}

PyObject* set_check(PyObject*, PyObject* f) {
  Py_XSETREF(g_check, Py_NewRef(f));
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"set_check", set_check, METH_O, "The function that raises for a status."},
    {"embedding", method<embedding, 4>(), METH_FASTCALL, "weight, ids, scale, dtype or None"},
    {"embedding_backward", method<embedding_backward, 5>(), METH_FASTCALL, "dout, ids, grad, scale, accumulate"},
    {"qk_norm_rope", method<qk_norm_rope, 9>(), METH_FASTCALL,
     "q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours"},
    {"qk_norm_rope_backward", method<qk_norm_rope_backward, 11>(), METH_FASTCALL,
     "dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours"},
    {"window_attention", method<window_attention, 7>(), METH_FASTCALL, "q, k, v, window, sinks, scale, cu_seqlens"},
    {"window_attention_backward", method<window_attention_backward, 10>(), METH_FASTCALL,
     "dout, q, k, v, out, lse, window, sinks, scale, cu_seqlens"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_ops", "The operators over torch tensors.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__torch_ops() { return PyModule_Create(&g_module); }
