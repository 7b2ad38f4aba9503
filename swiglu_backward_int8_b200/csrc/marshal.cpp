// The short way from torch tensors to the entry points of lowbit.py: the call
// that a decoding step makes again and again, with all outputs given, all of
// them on the current device.  Each function takes the arguments of its Python
// namesake, checks what that checks, and calls the C entry on the current
// stream; it returns the entry's status, or -1 for anything out of the ordinary
// (an output to allocate, another device, an argument that does not fit), which
// the Python code then handles or refuses with its reason.  The same checks in
// Python cost 5 us a call, twice what such a call's kernel takes.
//
// The interpreter's lock is given back around the C entry: a launch waits while
// the stream's queue is full, and what the queue waits for may need the lock (a
// host function, another thread's launch).
//
// The C entries' addresses come from the loaded library (bind).
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>

#include "sdq.h"

namespace {

decltype(&sdq_rmsnorm_quant) g_norm;
decltype(&sdq_rmsnorm_backward) g_norm_backward;
decltype(&sdq_rmsnorm_backward_workspace_bytes) g_workspace_bytes;
decltype(&sdq_quantize_fp4) g_quantize;
decltype(&sdq_dequantize_fp4) g_dequantize;
decltype(&sdq_matmul_fp4) g_matmul;

// f(args...) without the interpreter's lock; the arguments are made before it is
// given back.  (The caller's references keep the tensors alive.)
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <class F, class... A>
int unlocked(F f, A... args) {
  const Unlocked u;
  return f(args...);
}

struct Unusual {};   // thrown inside a function here, answered with -1 by its caller

// An operand on device `dev`.
struct Operand {
  const void* p = nullptr;
  int64_t ld = 0;
};

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw Unusual();
  return THPVariable_Unpack(o);
}

void on(const at::Tensor& t, int dev) {
  if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != dev) throw Unusual();
}

// A row-major [rows, cols] operand; rows may be padded.
Operand rows_of(const at::Tensor& t, int64_t rows, int64_t cols, at::ScalarType type, int dev) {
  on(t, dev);
  if (t.dim() != 2 || t.scalar_type() != type || t.size(0) != rows || t.size(1) != cols) throw Unusual();
  if ((cols > 1 && t.stride(1) != 1) || (rows > 1 && t.stride(0) < cols)) throw Unusual();
  return {t.data_ptr(), rows > 1 ? t.stride(0) : cols};
}

const void* vector_of(const at::Tensor& t, int64_t n, int dev) {
  on(t, dev);
  if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1)) throw Unusual();
  return t.data_ptr();
}

const float* global_of(PyObject* o, bool e4m3, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o);
  on(t, dev);
  if (!e4m3 || t.numel() != 1 || t.scalar_type() != at::kFloat) throw Unusual();
  return static_cast<const float*>(t.data_ptr());
}

bool is_e4m3(const at::Tensor& s) {
  const at::ScalarType t = s.scalar_type();
  if (t == at::kFloat8_e4m3fn) return true;
  if (t == at::kFloat8_e8m0fnu || t == at::kByte) return false;
  throw Unusual();
}

const void* tiles_of(const at::Tensor& s, int64_t rows, int64_t k, bool e4m3, int dev) {
  on(s, dev);
  const int64_t groups = k / (e4m3 ? 16 : 32);
  if (s.dim() != 3 || s.size(0) != (rows + 127) / 128 || s.size(1) != (groups + 3) / 4 || s.size(2) != 512 ||
      is_e4m3(s) != e4m3 || !s.is_contiguous())
    throw Unusual();
  return s.data_ptr();
}

// None, or the name that has to be given.
void named(PyObject* o, const char* name) {
  if (o != Py_None && (!PyUnicode_Check(o) || PyUnicode_CompareWithASCIIString(o, name) != 0)) throw Unusual();
}

// The device of the first operand, where it is the current one.
int card_of(const at::Tensor& t) {
  if (!t.defined() || !t.is_cuda() || t.get_device() != c10::cuda::current_device()) throw Unusual();
  return static_cast<int>(t.get_device());
}

void* stream(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

void two_d(const at::Tensor& t) {
  if (t.dim() != 2) throw Unusual();
}

// x, weight, residual, eps, group_size, codes, scales, q, s, h, y, rstd, global_scale
int norm(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0]), &w = tensor(a[1]), &q = tensor(a[7]), &s = tensor(a[8]);
  const int dev = card_of(x);
  two_d(x);
  const int64_t rows = x.size(0), channels = x.size(1);
  const at::ScalarType qt = q.scalar_type(), st = s.scalar_type();
  const bool e2m1 = qt == at::kByte;
  if (!e2m1 && qt != at::kChar && qt != at::kFloat8_e4m3fn) throw Unusual();
  named(a[5], e2m1 ? "e2m1" : qt == at::kChar ? "int8" : "e4m3");
  const bool s4 = st == at::kFloat8_e4m3fn, f32 = st == at::kFloat;
  if (!f32 && !s4 && st != at::kFloat8_e8m0fnu && st != at::kByte) throw Unusual();
  if (e2m1 ? f32 : s4) throw Unusual();
  named(a[6], s4 ? "e4m3" : f32 ? "fp32" : "e8m0");
  const double eps = PyFloat_AsDouble(a[3]);
  const long given = a[4] == Py_None ? (e2m1 ? (s4 ? 16 : 32) : 128) : PyLong_AsLong(a[4]);
  if (PyErr_Occurred()) throw Unusual();
  if (e2m1 ? given != (s4 ? 16 : 32) : given != 0 && given != 32 && given != 64 && given != 128 && given != 256)
    throw Unusual();
  if (channels < 1 || channels % (e2m1 ? SDQ_FP4_K_MULTIPLE : SDQ_K_MULTIPLE)) throw Unusual();
  uint32_t fmt = (e2m1 ? SDQ_FMT_E2M1 : qt == at::kFloat8_e4m3fn ? SDQ_FMT_E4M3 : 0) |
                 (s4 ? SDQ_FMT_SCALE_E4M3 : f32 ? 0 : SDQ_FMT_E8M0);
  const Operand ox = rows_of(x, rows, channels, at::kBFloat16, dev);
  if (w.scalar_type() == at::kFloat)
    fmt |= SDQ_FMT_WEIGHT_F32;
  else if (w.scalar_type() != at::kBFloat16)
    throw Unusual();
  const void* wp = vector_of(w, channels, dev);
  Operand residual, h, y, oq, os;
  if (a[2] != Py_None) {
    residual = rows_of(tensor(a[2]), rows, channels, at::kBFloat16, dev);
    h = rows_of(tensor(a[9]), rows, channels, at::kBFloat16, dev);
  } else if (a[9] != Py_None) {
    throw Unusual();
  }
  if (a[10] != Py_None) y = rows_of(tensor(a[10]), rows, channels, at::kBFloat16, dev);
  if (e2m1) {
    oq = rows_of(q, rows, channels / 2, at::kByte, dev);
    os.p = tiles_of(s, rows, channels, s4, dev);
  } else {
    oq = rows_of(q, rows, channels, qt, dev);
    os = rows_of(s, rows, given ? (channels + given - 1) / given : 1, st, dev);
  }
  const float* rstd = nullptr;
  if (a[11] != Py_None) {
    const at::Tensor& t = tensor(a[11]);
    if (t.scalar_type() != at::kFloat) throw Unusual();
    rstd = static_cast<const float*>(vector_of(t, rows, dev));
  }
  return unlocked(g_norm, ox.p, ox.ld, residual.p, residual.ld, wp, const_cast<void*>(h.p), h.ld, const_cast<void*>(oq.p),
                  oq.ld, const_cast<void*>(os.p), os.ld, const_cast<void*>(y.p), y.ld, const_cast<float*>(rstd),
                  global_of(a[12], s4, dev), rows, channels, static_cast<int32_t>(given), fmt, static_cast<float>(eps),
                  stream(dev));
}

// grad_y, h, weight, rstd, grad_h, grad_x, grad_weight, workspace
int norm_backward(PyObject* const* a) {
  const at::Tensor &gy = tensor(a[0]), &w = tensor(a[2]), &rstd = tensor(a[3]), &gw = tensor(a[6]);
  const int dev = card_of(gy);
  two_d(gy);
  const int64_t rows = gy.size(0), channels = gy.size(1);
  const Operand ogy = rows_of(gy, rows, channels, at::kBFloat16, dev);
  const Operand oh = rows_of(tensor(a[1]), rows, channels, at::kBFloat16, dev);
  const Operand ogx = rows_of(tensor(a[5]), rows, channels, at::kBFloat16, dev);
  Operand ogh;
  if (a[4] != Py_None) ogh = rows_of(tensor(a[4]), rows, channels, at::kBFloat16, dev);
  const bool f32 = w.scalar_type() == at::kFloat;
  if ((!f32 && w.scalar_type() != at::kBFloat16) || rstd.scalar_type() != at::kFloat || gw.scalar_type() != at::kFloat)
    throw Unusual();
  const void* wp = vector_of(w, channels, dev);
  const float* rp = static_cast<const float*>(vector_of(rstd, rows, dev));
  float* gp = static_cast<float*>(const_cast<void*>(vector_of(gw, channels, dev)));
  const size_t need = g_workspace_bytes(rows, channels);
  if (need == 0) throw Unusual();
  at::Tensor ws;
  if (a[7] == Py_None) {
    ws = at::empty({static_cast<int64_t>(need)}, gy.options().dtype(at::kByte));
  } else {
    ws = tensor(a[7]);
    on(ws, dev);
    if (!ws.is_contiguous()) throw Unusual();
  }
  return unlocked(g_norm_backward, ogy.p, ogy.ld, oh.p, oh.ld, wp, rp, ogh.p, ogh.ld, const_cast<void*>(ogx.p), ogx.ld, gp,
                  rows, channels, f32 ? SDQ_FMT_WEIGHT_F32 : 0, ws.data_ptr(),
                  static_cast<size_t>(ws.numel() * ws.element_size()), stream(dev));
}

void fp4_length(int64_t k) {
  if (k < SDQ_FP4_K_MULTIPLE || k % SDQ_FP4_K_MULTIPLE) throw Unusual();
}

// x, scales, axis, q, s, q_t, s_t, global_scale
int quantize(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0]);
  const int dev = card_of(x);
  two_d(x);
  const int64_t rows = x.size(0), channels = x.size(1), padded = (rows + 31) / 32 * 32;
  fp4_length(channels);
  if (rows == 0 || !PyUnicode_Check(a[2])) throw Unusual();
  const bool both = PyUnicode_CompareWithASCIIString(a[2], "both") == 0;
  const bool on_rows = both || PyUnicode_CompareWithASCIIString(a[2], "rows") == 0;
  const bool on_cols = both || PyUnicode_CompareWithASCIIString(a[2], "columns") == 0;
  if (!on_rows && !on_cols) throw Unusual();
  if (on_rows ? false : a[3] != Py_None || a[4] != Py_None) throw Unusual();
  if (on_cols ? false : a[5] != Py_None || a[6] != Py_None) throw Unusual();
  const bool e4m3 = is_e4m3(tensor(on_rows ? a[4] : a[6]));
  named(a[1], e4m3 ? "e4m3" : "e8m0");
  const Operand ox = rows_of(x, rows, channels, at::kBFloat16, dev);
  Operand q, qt;
  const void *s = nullptr, *st = nullptr;
  if (on_rows) {
    q = rows_of(tensor(a[3]), rows, channels / 2, at::kByte, dev);
    s = tiles_of(tensor(a[4]), rows, channels, e4m3, dev);
  }
  if (on_cols) {
    qt = rows_of(tensor(a[5]), channels, padded / 2, at::kByte, dev);
    st = tiles_of(tensor(a[6]), channels, padded, e4m3, dev);
  }
  return unlocked(g_quantize, ox.p, ox.ld, const_cast<void*>(q.p), q.ld, const_cast<void*>(s), const_cast<void*>(qt.p),
                  qt.ld, const_cast<void*>(st), global_of(a[7], e4m3, dev), rows, channels,
                  e4m3 ? SDQ_FMT_SCALE_E4M3 : SDQ_FMT_E8M0, stream(dev));
}

// q, s, global_scale, out
int dequantize(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0]), &s = tensor(a[1]);
  const int dev = card_of(q);
  two_d(q);
  const int64_t rows = q.size(0), k = 2 * q.size(1);
  fp4_length(k);
  const bool e4m3 = is_e4m3(s);
  const Operand oq = rows_of(q, rows, k / 2, at::kByte, dev);
  const void* sp = tiles_of(s, rows, k, e4m3, dev);
  const Operand out = rows_of(tensor(a[3]), rows, k, at::kBFloat16, dev);
  return unlocked(g_dequantize, oq.p, oq.ld, sp, global_of(a[2], e4m3, dev), const_cast<void*>(out.p), out.ld, rows, k,
                  e4m3 ? SDQ_FMT_SCALE_E4M3 : SDQ_FMT_E8M0, stream(dev));
}

// a, a_s, b, b_s, a_global, b_global, out, out_dtype
int matmul(PyObject* const* a) {
  const at::Tensor &qa = tensor(a[0]), &sa = tensor(a[1]), &qb = tensor(a[2]), &sb = tensor(a[3]), &out = tensor(a[6]);
  if (a[7] != Py_None) throw Unusual();
  const int dev = card_of(qa);
  two_d(qa);
  two_d(qb);
  const int64_t m = qa.size(0), n = qb.size(0), k = 2 * qa.size(1);
  fp4_length(k);
  const bool e4m3 = is_e4m3(sa), f32 = out.scalar_type() == at::kFloat;
  const Operand oa = rows_of(qa, m, k / 2, at::kByte, dev), ob = rows_of(qb, n, k / 2, at::kByte, dev);
  const void *ap = tiles_of(sa, m, k, e4m3, dev), *bp = tiles_of(sb, n, k, e4m3, dev);
  const Operand oo = rows_of(out, m, n, f32 ? at::kFloat : at::kBFloat16, dev);
  return unlocked(g_matmul, oa.p, oa.ld, ap, global_of(a[4], e4m3, dev), ob.p, ob.ld, bp, global_of(a[5], e4m3, dev),
                  const_cast<void*>(oo.p), oo.ld, m, n, k,
                  (e4m3 ? SDQ_FMT_SCALE_E4M3 : SDQ_FMT_E8M0) | (f32 ? SDQ_FMT_OUT_F32 : 0u), stream(dev));
}

template <int (*kCall)(PyObject* const*), int kArgs>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  int status = -1;
  if (n == kArgs) {
    try {
      status = kCall(args);
    } catch (...) {   // Unusual, or torch's own: the Python code says what is wrong
      status = -1;
    }
  }
  PyErr_Clear();
  return PyLong_FromLong(status);
}

PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void* p[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i]) return PyErr_Occurred() ? nullptr : (PyErr_SetString(PyExc_ValueError, "a null address"), nullptr);
  }
  g_norm = reinterpret_cast<decltype(g_norm)>(p[0]);
  g_norm_backward = reinterpret_cast<decltype(g_norm_backward)>(p[1]);
  g_workspace_bytes = reinterpret_cast<decltype(g_workspace_bytes)>(p[2]);
  g_quantize = reinterpret_cast<decltype(g_quantize)>(p[3]);
  g_dequantize = reinterpret_cast<decltype(g_dequantize)>(p[4]);
  g_matmul = reinterpret_cast<decltype(g_matmul)>(p[5]);
  Py_RETURN_NONE;
}

template <PyObject* (*kFn)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kFn)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<bind>("bind"),
    method<call<norm, 13>>("rmsnorm_quant"),
    method<call<norm_backward, 8>>("rmsnorm_backward"),
    method<call<quantize, 8>>("quantize_fp4"),
    method<call<dequantize, 4>>("dequantize_fp4"),
    method<call<matmul, 8>>("matmul_fp4"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&g_module); }
