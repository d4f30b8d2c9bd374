// The common case of the torch-facing row operators, without the interpreter:
// plain CUDA tensors on the current device, contiguous, of supported types, output
// to be allocated, current stream. A small call's time is its host's: describing
// four tensors and allocating two in Python takes about as long as the launch.
//
// Everything else returns NotImplemented, and the Python code answers it with its
// own checks and errors: this file refuses nothing and computes nothing. The library
// is called through the addresses that bind() is given, so that it is the same
// loaded libwf.so.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "wf.h"

namespace {

using at::Tensor;

decltype(&wf_linear) g_linear = nullptr;
decltype(&wf_add_rms_norm) g_norm = nullptr;
decltype(&wf_quantize_rows) g_quantize = nullptr;
decltype(&wf_dequantize_rows) g_dequantize = nullptr;

bool given(PyObject *o) { return o != Py_None; }

// A contiguous strided tensor of at least one dimension on the current device, of
// one of two types, that records no gradient and carries no tangent (and has memory
// of its own: what a function transform wraps has none). Clears *ok otherwise.
const Tensor &plain(PyObject *o, at::ScalarType a, at::ScalarType b, bool *ok) {
  static const Tensor none;
  if (!THPVariable_CheckExact(o)) {
    *ok = false;
    return none;
  }
  const Tensor &t = THPVariable_Unpack(o);
  const auto type = t.scalar_type();
  if (!t.is_cuda() || t.layout() != at::kStrided || !t.has_storage() || (type != a && type != b) || t.dim() < 1 ||
      !t.is_contiguous() || t.is_conj() || t.is_neg() || t.size(-1) == 0 ||
      t.get_device() != c10::cuda::current_device() ||
      (c10::GradMode::is_enabled() && t.requires_grad()) ||
      (t.unsafeGetTensorImpl()->autograd_meta() && t._fw_grad(/*level=*/0).defined()))
    *ok = false;
  return t;
}

wf_rows rows_of(const Tensor &t, const Tensor *scales = nullptr) {
  wf_rows r{};
  r.data = t.data_ptr();
  r.cols = r.ld = t.size(-1);
  r.rows = t.numel() / r.cols;
  r.dtype = t.scalar_type() == at::kFloat ? WF_DTYPE_F32 : t.scalar_type() == at::kBFloat16 ? WF_DTYPE_BF16 : WF_DTYPE_FP8_E4M3;
  if (scales) r.scales = scales->data_ptr();
  return r;
}

// Whether codes [rows][cols] and their scale bytes describe E4M3 rows.
bool e4m3_rows(const Tensor &codes, const Tensor &scales) {
  return codes.dim() == 2 && codes.size(1) % 32 == 0 &&
         scales.numel() >= (codes.size(0) + 127) / 128 * ((codes.size(1) + 127) / 128) * 512;
}

Tensor new_scales(int64_t rows, int64_t cols, const Tensor &like) {
  return at::empty({(rows + 127) / 128 * ((cols + 127) / 128) * 512}, like.options().dtype(at::kByte));
}

wf_stream_t stream_of(const Tensor &t) {
  return reinterpret_cast<wf_stream_t>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
}

template <typename F>
wf_status without_gil(F call) {
  PyThreadState *save = PyEval_SaveThread();
  const wf_status st = call();
  PyEval_RestoreThread(save);
  return st;
}

// A status on failure; on success the tensors (one, or a tuple).
PyObject *answer(wf_status st, const Tensor &a, const Tensor *b = nullptr, const Tensor *c = nullptr) {
  if (st != WF_OK) return PyLong_FromLong(st);
  if (!b && !c) return THPVariable_Wrap(a);
  PyObject *t = PyTuple_New(c ? 3 : 2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  if (b) PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(*b));
  else if (c) { Py_INCREF(Py_None); PyTuple_SET_ITEM(t, 1, Py_None); }
  if (c) PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(*c));
  return t;
}

// linear(x, x_scales, w, w_scales, bias, act, residual, out8)
//   -> out, or (codes, scales) | status | NotImplemented
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8 || !g_linear) Py_RETURN_NOTIMPLEMENTED;
  bool ok = true;
  const bool e4m3 = given(a[1]), out8 = a[7] == Py_True;
  const auto type = e4m3 ? at::kFloat8_e4m3fn : at::kBFloat16;
  const Tensor &x = plain(a[0], type, type, &ok);
  const Tensor &w = plain(a[2], type, type, &ok);
  if (!ok || e4m3 != given(a[3]) || w.dim() != 2 || w.size(0) == 0 || x.size(-1) != w.size(1)) Py_RETURN_NOTIMPLEMENTED;
  const Tensor *xs = nullptr, *ws = nullptr, *bias = nullptr, *res = nullptr;
  if (e4m3) {
    xs = &plain(a[1], at::kByte, at::kByte, &ok);
    ws = &plain(a[3], at::kByte, at::kByte, &ok);
    if (!ok || !e4m3_rows(x, *xs) || !e4m3_rows(w, *ws)) Py_RETURN_NOTIMPLEMENTED;
  }
  const int64_t N = w.size(0), K = w.size(1), M = x.numel() / K;
  at::DimVector shape(x.sizes().begin(), x.sizes().end());
  shape.back() = N;
  if (given(a[4])) {
    bias = &plain(a[4], at::kFloat, at::kFloat, &ok);
    if (!ok || bias->dim() != 1 || bias->size(0) != N) Py_RETURN_NOTIMPLEMENTED;
  }
  if (given(a[6])) {
    res = &plain(a[6], at::kBFloat16, at::kBFloat16, &ok);
    if (!ok || res->sizes() != at::IntArrayRef(shape)) Py_RETURN_NOTIMPLEMENTED;
  }
  if (out8 && (res || N % 32 != 0)) Py_RETURN_NOTIMPLEMENTED;
  const long act = PyLong_AsLong(a[5]);
  if (act == -1 && PyErr_Occurred()) return nullptr;
  Tensor out, scales;
  if (out8) {
    out = at::empty({M, N}, x.options().dtype(at::kFloat8_e4m3fn));
    scales = new_scales(M, N, x);
  } else {
    out = at::empty(shape, x.options().dtype(at::kBFloat16));
  }
  const wf_rows rx = rows_of(x, xs), rw = rows_of(w, ws), ro = rows_of(out, out8 ? &scales : nullptr);
  wf_rows rr{};
  if (res) rr = rows_of(*res);
  const float *b = bias ? bias->const_data_ptr<float>() : nullptr;
  const wf_stream_t st = stream_of(x);
  const wf_status s = without_gil([&] {
    return g_linear(&rx, &rw, b, static_cast<int32_t>(act), res ? &rr : nullptr, &ro, st);
  });
  return answer(s, out, out8 ? &scales : nullptr);
  END_HANDLE_TH_ERRORS
}

// add_rms_norm(x, weight, residual, eps, out8)
//   -> out | (out, sum) | (codes, scales) | (codes, scales, sum) | status | NotImplemented
PyObject *add_rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5 || !g_norm) Py_RETURN_NOTIMPLEMENTED;
  bool ok = true;
  const bool out8 = a[4] == Py_True;
  const Tensor &x = plain(a[0], at::kBFloat16, at::kFloat, &ok);
  if (!ok) Py_RETURN_NOTIMPLEMENTED;
  const int64_t cols = x.size(-1), rows = x.numel() / cols;
  const Tensor *weight = nullptr, *res = nullptr;
  if (given(a[1])) {
    weight = &plain(a[1], at::kFloat, at::kFloat, &ok);
    if (!ok || weight->dim() != 1 || weight->size(0) != cols) Py_RETURN_NOTIMPLEMENTED;
  }
  if (given(a[2])) {
    res = &plain(a[2], x.scalar_type(), x.scalar_type(), &ok);
    if (!ok || res->sizes() != x.sizes()) Py_RETURN_NOTIMPLEMENTED;
  }
  if (out8 && cols % 32 != 0) Py_RETURN_NOTIMPLEMENTED;
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  Tensor out, scales, sum;
  if (out8) {
    out = at::empty({rows, cols}, x.options().dtype(at::kFloat8_e4m3fn));
    scales = new_scales(rows, cols, x);
  } else {
    out = at::empty(x.sizes(), x.options());
  }
  if (res) sum = at::empty(x.sizes(), x.options());
  const wf_rows rx = rows_of(x), ro = rows_of(out, out8 ? &scales : nullptr);
  wf_rows rr{}, rs{};
  if (res) {
    rr = rows_of(*res);
    rs = rows_of(sum);
  }
  const float *w = weight ? weight->const_data_ptr<float>() : nullptr;
  const wf_stream_t st = stream_of(x);
  const wf_status s = without_gil([&] {
    return g_norm(&rx, res ? &rr : nullptr, w, static_cast<float>(eps), res ? &rs : nullptr, &ro, st);
  });
  if (out8) return answer(s, out, &scales, res ? &sum : nullptr);
  return answer(s, out, res ? &sum : nullptr);
  END_HANDLE_TH_ERRORS
}

// quantize_rows(x) -> (codes, scales) | status | NotImplemented
PyObject *quantize_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 1 || !g_quantize) Py_RETURN_NOTIMPLEMENTED;
  bool ok = true;
  const Tensor &x = plain(a[0], at::kBFloat16, at::kFloat, &ok);
  if (!ok || x.size(-1) % 32 != 0) Py_RETURN_NOTIMPLEMENTED;
  const int64_t cols = x.size(-1), rows = x.numel() / cols;
  const Tensor out = at::empty({rows, cols}, x.options().dtype(at::kFloat8_e4m3fn));
  const Tensor scales = new_scales(rows, cols, x);
  const wf_rows rx = rows_of(x), ro = rows_of(out, &scales);
  const wf_stream_t st = stream_of(x);
  const wf_status s = without_gil([&] { return g_quantize(&rx, &ro, st); });
  return answer(s, out, &scales);
  END_HANDLE_TH_ERRORS
}

// dequantize_rows(codes, scales, f32) -> out | status | NotImplemented
PyObject *dequantize_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 3 || !g_dequantize) Py_RETURN_NOTIMPLEMENTED;
  bool ok = true;
  const Tensor &x = plain(a[0], at::kFloat8_e4m3fn, at::kFloat8_e4m3fn, &ok);
  const Tensor &s8 = plain(a[1], at::kByte, at::kByte, &ok);
  if (!ok || !e4m3_rows(x, s8)) Py_RETURN_NOTIMPLEMENTED;
  const Tensor out = at::empty(x.sizes(), x.options().dtype(a[2] == Py_True ? at::kFloat : at::kBFloat16));
  const wf_rows rx = rows_of(x, &s8), ro = rows_of(out);
  const wf_stream_t st = stream_of(x);
  const wf_status s = without_gil([&] { return g_dequantize(&rx, &ro, st); });
  return answer(s, out);
  END_HANDLE_TH_ERRORS
}

// bind(linear, add_rms_norm, quantize_rows, dequantize_rows): addresses in libwf.so.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  void *p[4];
  if (n != 4) Py_RETURN_NOTIMPLEMENTED;
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "null address");
  }
  g_linear = reinterpret_cast<decltype(g_linear)>(p[0]);
  g_norm = reinterpret_cast<decltype(g_norm)>(p[1]);
  g_quantize = reinterpret_cast<decltype(g_quantize)>(p[2]);
  g_dequantize = reinterpret_cast<decltype(g_dequantize)>(p[3]);
  Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<linear>("linear"), method<add_rms_norm>("add_rms_norm"),
                           method<quantize_rows>("quantize_rows"), method<dequantize_rows>("dequantize_rows"),
                           method<bind>("bind"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_rows_bind", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rows_bind() {
  PyObject *m = PyModule_Create(&g_module);
  // The torch whose headers this was built with; the package compares it with the one it runs under.
  if (m && PyModule_AddStringConstant(m, "torch_version", WF_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
