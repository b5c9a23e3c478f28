// ops_binding.cpp — the second-pass operators' path from torch tensors to the C
// calls: checks, results, argument blocks.
//
// A call for one token is over on the GPU in a few microseconds, and Python
// takes longer than that to ask some ten tensors for their types, devices,
// shapes and strides (norm_rotate 15 us a call, sample_tokens 24).  So the calls
// that go on a step's path ask them here, all at once.  A call returns its
// tensors; 1 when an argument is wrong, which the Python side then looks for and
// names; or the library's error, which is negative.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/wfst_gb300.h"

namespace {

using at::ScalarType;
using at::Tensor;

constexpr int kLook = 1;  // an argument is wrong

int type_code(ScalarType t) {
  switch (t) {
    case ScalarType::Float: return WFST_F32;
    case ScalarType::Half: return WFST_F16;
    case ScalarType::BFloat16: return WFST_BF16;
    default: return -1;
  }
}

// One call's arguments as they are read; `ok` says whether all were right.
struct Reader {
  bool ok = true;
  int dev = -1;
  ScalarType type = ScalarType::Undefined;

  // a tensor of `dim` axes on the call's device, which the first one sets; none
  // that waits for a gradient, since there is none to give
  const Tensor* tensor(PyObject* o, int64_t dim, ScalarType t) {
    if (!THPVariable_Check(o)) return fail();
    const Tensor& x = THPVariable_Unpack(o);
    if (x.requires_grad() && at::GradMode::is_enabled()) return fail();
    if (!x.is_cuda() || x.layout() != at::kStrided || x.dim() != dim || x.scalar_type() != t) return fail();
    if (dev < 0) dev = x.get_device();
    if (x.get_device() != dev) return fail();
    return &x;
  }
  // the first tensor, whose type the others share
  const Tensor* first(PyObject* o, int64_t dim) {
    if (!THPVariable_Check(o)) return fail();
    type = THPVariable_Unpack(o).scalar_type();
    return tensor(o, dim, type);
  }
  // the elements of a contiguous vector of n, or NULL for None
  void* vector(PyObject* o, int64_t n, ScalarType t) {
    const Tensor* x = tensor(o, 1, t);
    if (!x || x->size(0) != n || !x->is_contiguous()) return fail();
    return x->data_ptr();
  }
  void* vector_or_none(PyObject* o, int64_t n, ScalarType t) { return o == Py_None ? nullptr : vector(o, n, t); }
  int32_t i32(int64_t v) {
    if (v < INT32_MIN || v > INT32_MAX) ok = false;
    return (int32_t)v;
  }
  // (a Python error is left for the caller to find)
  int32_t number(PyObject* o) { return i32(PyLong_AsLongLong(o)); }
  std::nullptr_t fail() {
    ok = false;
    return nullptr;
  }
};

// Unit stride over the last axis, which may have one entry.
bool unit(const Tensor& t) { return t.stride(-1) == 1 || t.size(-1) < 2; }

Tensor empty(at::IntArrayRef size, ScalarType t, int dev) {
  return at::detail::empty_cuda(size, t, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
}

// Lets torch know that a caller's tensor has other values now.
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

PyObject* look() { return PyLong_FromLong(kLook); }

template <typename Block>
int call(int (*f)(const Block*, void*), const Block& b, int dev) {
  void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f(&b, stream);
  Py_END_ALLOW_THREADS
  return rc;
}

// matvec_quant(x, matrix, bias, out); matrix: (packed, dtype, n, k, group, zeros, device)
PyObject* matvec_quant(PyObject*, PyObject* const* arg, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 4 || !PyTuple_Check(arg[1]) || PyTuple_GET_SIZE(arg[1]) != 7) return look();
  long long m[7];
  for (int i = 0; i < 7; i++) m[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(arg[1], i));
  if (PyErr_Occurred()) return nullptr;
  Reader r;
  r.dev = (int)m[6];
  const Tensor* x = r.first(arg[0], 2);
  if (!x || type_code(r.type) != m[1] || x->size(1) != m[3] || x->stride(1) != 1) return look();
  const int64_t rows = x->size(0), n = m[2];
  wfst_matvec_args a = {};
  a.bias = r.vector_or_none(arg[2], n, r.type);
  Tensor y;
  if (arg[3] == Py_None) {
    if (!r.ok) return look();
    y = empty({rows, n}, r.type, r.dev);
  } else {
    const Tensor* out = r.tensor(arg[3], 2, r.type);
    if (!out || out->size(0) != rows || out->size(1) != n || !unit(*out)) return look();
    y = *out;
  }
  a.packed = (const void*)(uintptr_t)m[0];
  a.x = x->data_ptr();
  a.y = y.data_ptr();
  a.stride_x = x->stride(0);
  a.stride_y = y.stride(0);
  a.device = r.dev;
  a.dtype = (int32_t)m[1];
  a.n = (int32_t)n;
  a.k = (int32_t)m[3];
  a.group = (int32_t)m[4];
  a.zeros = (int32_t)m[5];
  a.rows = r.i32(rows);
  if (!r.ok) return look();
  if (const int rc = call(wfst_matvec_quant, a, r.dev)) return PyLong_FromLong(rc);
  if (arg[3] != Py_None) written(y);
  return THPVariable_Wrap(std::move(y));
  END_HANDLE_TH_ERRORS
}

// norm_rotate(q, k, v, positions, table, q_gain, k_gain, k_pages, v_pages, slots, eps, interleaved, out)
PyObject* norm_rotate(PyObject*, PyObject* const* arg, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 13) return look();
  Reader r;
  const Tensor* q = r.first(arg[0], 3);
  if (!q || type_code(r.type) <= 0) return look();
  const Tensor *k = r.tensor(arg[1], 3, r.type), *v = r.tensor(arg[2], 3, r.type);
  const Tensor *kp = r.tensor(arg[7], 4, r.type), *vp = r.tensor(arg[8], 4, r.type);
  const Tensor* table = r.tensor(arg[4], 2, ScalarType::Float);
  if (!r.ok) return look();
  const int64_t tokens = q->size(0), hq = q->size(1), d = q->size(2), hkv = k->size(1);
  if (k->size(0) != tokens || k->size(2) != d || v->sizes() != k->sizes() || kp->size(2) != hkv || kp->size(3) != d ||
      vp->sizes() != kp->sizes() || !unit(*q) || !unit(*k) || !unit(*v) || !unit(*kp) || !unit(*vp) ||
      !table->is_contiguous())
    return look();
  wfst_rotate_args a = {};
  a.positions = (const int32_t*)r.vector(arg[3], tokens, ScalarType::Int);
  a.slots = (const int32_t*)r.vector(arg[9], tokens, ScalarType::Int);
  a.q_gain = r.vector_or_none(arg[5], d, r.type);
  a.k_gain = r.vector_or_none(arg[6], d, r.type);
  a.eps = (float)PyFloat_AsDouble(arg[10]);
  a.interleaved = PyObject_IsTrue(arg[11]);
  if (PyErr_Occurred()) return nullptr;
  if (!r.ok) return look();
  Tensor y;
  if (arg[12] == Py_None) {
    y = empty({tokens, hq, d}, r.type, r.dev);
  } else {
    const Tensor* out = r.tensor(arg[12], 3, r.type);
    if (!out || out->sizes() != q->sizes() || !unit(*out)) return look();
    y = *out;
  }
  a.q = q->data_ptr();
  a.k = k->data_ptr();
  a.v = v->data_ptr();
  a.table = (const float*)table->data_ptr();
  a.q_out = y.data_ptr();
  a.k_pages = kp->data_ptr();
  a.v_pages = vp->data_ptr();
  for (int i = 0; i < 2; i++) {
    a.q_stride[i] = q->stride(i);
    a.k_stride[i] = k->stride(i);
    a.v_stride[i] = v->stride(i);
    a.out_stride[i] = y.stride(i);
  }
  for (int i = 0; i < 3; i++) {
    a.k_page_stride[i] = kp->stride(i);
    a.v_page_stride[i] = vp->stride(i);
  }
  a.device = r.dev;
  a.dtype = type_code(r.type);
  a.tokens = r.i32(tokens);
  a.q_heads = r.i32(hq);
  a.kv_heads = r.i32(hkv);
  a.head_dim = r.i32(d);
  a.rot = r.i32(table->size(1));
  a.contexts = r.i32(table->size(0));
  a.num_pages = r.i32(kp->size(0));
  a.page_size = r.i32(kp->size(1));
  if (!r.ok) return look();
  if (const int rc = call(wfst_norm_rotate, a, r.dev)) return PyLong_FromLong(rc);
  written(*kp), written(*vp);
  if (arg[12] != Py_None) written(y);
  return THPVariable_Wrap(std::move(y));
  END_HANDLE_TH_ERRORS
}

// attend_paged(q, k_pages, v_pages, page_table, lengths, scale, window, sinks, workspace, with_lse, out)
PyObject* attend_paged(PyObject*, PyObject* const* arg, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 11) return look();
  Reader r;
  const Tensor* q = r.first(arg[0], 3);
  if (!q || type_code(r.type) <= 0) return look();
  const Tensor *kp = r.tensor(arg[1], 4, r.type), *vp = r.tensor(arg[2], 4, r.type);
  const Tensor* table = r.tensor(arg[3], 2, ScalarType::Int);
  const Tensor* ws = arg[8] == Py_None ? nullptr : r.tensor(arg[8], 1, ScalarType::Byte);
  if (!r.ok) return look();
  const int64_t lanes = q->size(0), hq = q->size(1), d = q->size(2);
  static const int64_t ws_bytes = [] {
    int64_t n = INT64_MAX;
    wfst_attend_size(&n);
    return n;
  }();
  if (kp->size(3) != d || vp->sizes() != kp->sizes() || table->size(0) != lanes || !unit(*q) || !unit(*kp) ||
      !unit(*vp) || !unit(*table) || (ws && (!ws->is_contiguous() || ws->numel() < ws_bytes)))
    return look();
  wfst_attend_args a = {};
  a.lengths = (const int32_t*)r.vector(arg[4], lanes, ScalarType::Int);
  a.scale = arg[5] == Py_None ? (float)(1.0 / std::sqrt((double)d)) : (float)PyFloat_AsDouble(arg[5]);
  a.window = r.number(arg[6]);
  a.sinks = r.number(arg[7]);
  const int with_lse = PyObject_IsTrue(arg[9]);
  if (PyErr_Occurred()) return nullptr;
  if (!r.ok) return look();
  Tensor y, lse;
  if (arg[10] == Py_None) {
    y = empty({lanes, hq, d}, r.type, r.dev);
  } else {
    const Tensor* out = r.tensor(arg[10], 3, r.type);
    if (!out || out->sizes() != q->sizes() || !unit(*out)) return look();
    y = *out;
  }
  Tensor own;
  if (!ws) {  // as attend_workspace makes it
    own = empty({ws_bytes}, ScalarType::Byte, r.dev);
    own.narrow(0, 0, WFST_ATTEND_ZEROED).zero_();
    ws = &own;
  }
  if (with_lse) {
    lse = empty({lanes, hq}, ScalarType::Float, r.dev);
    a.lse = (float*)lse.data_ptr();
    a.lse_stride = hq;
  }
  a.q = q->data_ptr();
  a.k_pages = kp->data_ptr();
  a.v_pages = vp->data_ptr();
  a.table = (const int32_t*)table->data_ptr();
  a.o = y.data_ptr();
  a.workspace = ws->data_ptr();
  for (int i = 0; i < 2; i++) {
    a.q_stride[i] = q->stride(i);
    a.o_stride[i] = y.stride(i);
  }
  for (int i = 0; i < 3; i++) {
    a.k_page_stride[i] = kp->stride(i);
    a.v_page_stride[i] = vp->stride(i);
  }
  a.table_stride = table->stride(0);
  a.device = r.dev;
  a.dtype = type_code(r.type);
  a.lanes = r.i32(lanes);
  a.q_heads = r.i32(hq);
  a.kv_heads = r.i32(kp->size(2));
  a.head_dim = r.i32(d);
  a.table_width = r.i32(table->size(1));
  a.num_pages = r.i32(kp->size(0));
  a.page_size = r.i32(kp->size(1));
  if (!r.ok) return look();
  if (const int rc = call(wfst_attend_paged, a, r.dev)) return PyLong_FromLong(rc);
  if (arg[10] != Py_None) written(y);
  if (!with_lse) return THPVariable_Wrap(std::move(y));
  PyObject* both = PyTuple_New(2);
  if (!both) return nullptr;
  PyTuple_SET_ITEM(both, 0, THPVariable_Wrap(std::move(y)));
  PyTuple_SET_ITEM(both, 1, THPVariable_Wrap(std::move(lse)));
  return both;
  END_HANDLE_TH_ERRORS
}

// sample_tokens(logits, uniform, temperature, top_k, top_p, min_p)
PyObject* sample_tokens(PyObject*, PyObject* const* arg, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 6) return look();
  Reader r;
  const Tensor* x = r.first(arg[0], 2);
  if (!x || type_code(r.type) < 0 || !unit(*x)) return look();
  const int64_t lanes = x->size(0);
  wfst_sample_args a = {};
  a.uniform = (const float*)r.vector(arg[1], lanes, ScalarType::Float);
  auto setting = [&](PyObject* o, const float*& each, float& all) {
    if (THPVariable_Check(o))
      each = (const float*)r.vector(o, lanes, ScalarType::Float);
    else
      all = (float)PyFloat_AsDouble(o);
  };
  setting(arg[2], a.temperature_v, a.temperature);
  if (THPVariable_Check(arg[3]))
    a.top_k_v = (const int32_t*)r.vector(arg[3], lanes, ScalarType::Int);
  else
    a.top_k = r.number(arg[3]);
  setting(arg[4], a.top_p_v, a.top_p);
  setting(arg[5], a.min_p_v, a.min_p);
  if (PyErr_Occurred()) return nullptr;
  a.logits = x->data_ptr();
  a.stride = x->stride(0);
  a.device = r.dev;
  a.dtype = type_code(r.type);
  a.lanes = r.i32(lanes);
  a.vocab = r.i32(x->size(1));
  if (!r.ok) return look();
  Tensor tokens = empty({lanes}, ScalarType::Int, r.dev), logprobs = empty({lanes}, ScalarType::Float, r.dev),
         kept = empty({lanes}, ScalarType::Int, r.dev);
  a.tokens = (int32_t*)tokens.data_ptr();
  a.logprobs = (float*)logprobs.data_ptr();
  a.kept = (int32_t*)kept.data_ptr();
  if (const int rc = call(wfst_sample_tokens, a, r.dev)) return PyLong_FromLong(rc);
  PyObject* all = PyTuple_New(3);
  if (!all) return nullptr;
  PyTuple_SET_ITEM(all, 0, THPVariable_Wrap(std::move(tokens)));
  PyTuple_SET_ITEM(all, 1, THPVariable_Wrap(std::move(logprobs)));
  PyTuple_SET_ITEM(all, 2, THPVariable_Wrap(std::move(kept)));
  return all;
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, (PyCFunction)(void (*)(void))F, METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<matvec_quant>("matvec_quant"), method<norm_rotate>("norm_rotate"),
                         method<attend_paged>("attend_paged"), method<sample_tokens>("sample_tokens"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "ops_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ops_binding() { return PyModule_Create(&module); }
