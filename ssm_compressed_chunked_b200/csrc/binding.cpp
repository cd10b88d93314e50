// Argument marshalling of the SSM block's operators for PyTorch tensors (module _binding).
//
// A decode step makes several of these calls per layer, each a few microseconds of GPU work, and a Python
// wrapper that checks ten tensors one attribute at a time takes longer than the kernel.  This module
// makes the same checks on the tensors themselves (type, device, shape, strides), takes the current stream of
// their device and calls the C ABI of include/attamba.h through function pointers handed over by init():
// it links no kernel, computes nothing and keeps no state but those pointers.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "attamba.h"

namespace {
using Shape = at::IntArrayRef;

PyObject* g_error = nullptr;   // AttambaError
decltype(&attamba_status_string) g_status_string = nullptr;
decltype(&attamba_last_error) g_last_error = nullptr;
decltype(&attamba_causal_conv) g_causal_conv = nullptr;
decltype(&attamba_conv_step) g_conv_step = nullptr;
decltype(&attamba_selective_scan) g_selective_scan = nullptr;
decltype(&attamba_scan_step) g_scan_step = nullptr;
decltype(&attamba_clear_rows) g_clear_rows = nullptr;
decltype(&attamba_block_norm) g_block_norm = nullptr;

// Every check returns false with the Python error set; what torch itself throws is caught at the entry (entry<>).
bool refuse(const std::string& text) {
  PyErr_SetString(g_error, text.c_str());
  return false;
}
std::string text_of(Shape s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}
std::string device_of(const at::Tensor& t) { return t.is_cuda() ? "cuda:" + std::to_string(t.get_device()) : "the CPU"; }
bool refuse_tensor(const at::Tensor& t, const char* name, const char* what, c10::ScalarType dt, Shape shape, int dev) {
  std::string s = std::string(name) + " must be " + what + " " + c10::toString(dt) + " " + text_of(shape) + " on cuda:" +
                  std::to_string(dev) + ", got " + c10::toString(t.scalar_type()) + " " + text_of(t.sizes());
  if (t.layout() == at::kStrided) s += ", strides " + text_of(t.strides()) + ",";
  return refuse(s + " on " + device_of(t));
}

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
  refuse(std::string(name) + " must be a tensor");
  return nullptr;
}
bool fits(const at::Tensor& t, c10::ScalarType dt, Shape shape, int dev) {
  return t.scalar_type() == dt && t.is_cuda() && t.get_device() == dev && t.layout() == at::kStrided && t.sizes() == shape;
}

struct Rows {
  void* p = nullptr;
  int64_t ld = 0;
};
// Token rows [rows, cols] whose columns are neighbours; null for None.
bool rows(PyObject* o, const char* name, c10::ScalarType dt, int64_t r, int64_t c, int dev, Rows& out) {
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  const int64_t shape[2] = {r, c};
  if (!fits(*t, dt, shape, dev) || (t->stride(1) != 1 && c > 1)) return refuse_tensor(*t, name, "rows of", dt, shape, dev);
  out.p = t->data_ptr();
  out.ld = r > 1 ? t->stride(0) : c;
  return true;
}
// A contiguous array; null for None.
template <typename P> bool dense(PyObject* o, const char* name, c10::ScalarType dt, Shape shape, int dev, P*& out) {
  out = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  if (!fits(*t, dt, shape, dev) || !t->is_contiguous()) return refuse_tensor(*t, name, "a contiguous", dt, shape, dev);
  out = static_cast<P*>(t->data_ptr());
  return true;
}
bool vec_f32(PyObject* o, const char* name, int64_t n, int dev, const float*& out) {
  const int64_t shape[1] = {n};
  return dense(o, name, at::kFloat, shape, dev, out);
}
bool mat_f32(PyObject* o, const char* name, int64_t r, int64_t c, int dev, const float*& out) {
  const int64_t shape[2] = {r, c};
  return dense(o, name, at::kFloat, shape, dev, out);
}
bool vec_i32(PyObject* o, const char* name, int64_t n, int dev, int32_t*& out) {
  const int64_t shape[1] = {n};
  return dense(o, name, at::kInt, shape, dev, out);
}

bool code_of(c10::ScalarType dt, const char* name, attamba_dtype_t& out) {
  if (dt != at::kBFloat16 && dt != at::kFloat) return refuse(std::string(name) + ": unsupported dtype " + c10::toString(dt));
  out = dt == at::kBFloat16 ? ATTAMBA_BF16 : ATTAMBA_F32;
  return true;
}

// The tensor that says the call's type, device, rows and columns.
struct Lead {
  c10::ScalarType dt;
  attamba_dtype_t code;
  int dev;
  int64_t rows, cols;
};
bool lead(PyObject* o, const char* name, Lead& l) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  if (!t->is_cuda()) return refuse(std::string(name) + " must be a CUDA tensor (there is no CPU path)");
  if (t->dim() != 2 || t->size(0) < 1)
    return refuse(std::string(name) + " must be [rows >= 1, cols], got " + text_of(t->sizes()));
  if (t->size(0) > INT32_MAX || t->size(1) > INT32_MAX) return refuse(std::string(name) + " is too large");
  l.dt = t->scalar_type();
  l.dev = (int)t->get_device();
  l.rows = t->size(0);
  l.cols = t->size(1);
  return code_of(l.dt, name, l.code);
}
bool last_dim(PyObject* o, const char* name, int64_t& out) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  out = t->dim() ? t->size(-1) : 0;
  return out <= INT32_MAX || refuse(std::string(name) + " is too large");
}

// A contiguous state [slots, rows, cols]; null and 0 for None.
struct State {
  void* p = nullptr;
  int32_t n = 0;
};
bool state(PyObject* o, c10::ScalarType dt, int64_t r, int64_t c, int dev, State& out) {
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o, "state");
  if (!t) return false;
  const int64_t shape[3] = {t->dim() == 3 ? t->size(0) : -1, r, c};
  if (shape[0] == 0) return refuse("state has no slots");   // its address is null, which would mean no state
  if (shape[0] > INT32_MAX) return refuse("state has too many slots");
  out.n = (int32_t)shape[0];
  return dense(o, "state", dt, shape, dev, out.p);
}

bool number(PyObject* o, int64_t& out) {
  out = PyLong_AsLongLong(o);
  return out != -1 || !PyErr_Occurred();
}
bool number32(PyObject* o, const char* name, int32_t& out) {
  int64_t v;
  if (!number(o, v)) return false;
  if (v < INT32_MIN || v > INT32_MAX) return refuse(std::string(name) + " is out of range");
  out = (int32_t)v;
  return true;
}
bool real(PyObject* o, float& out) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) return false;
  out = (float)v;
  return true;
}

// The stream to launch on: the given torch.cuda.Stream, or the current one of the device.
bool stream_of(PyObject* o, int dev, const char* what, attamba_stream_t& out) {
  if (o == Py_None) {
    out = reinterpret_cast<attamba_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
    return true;
  }
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  PyObject* d = h ? PyObject_GetAttrString(o, "device_index") : nullptr;
  const uintptr_t handle = d ? (uintptr_t)PyLong_AsUnsignedLongLong(h) : 0;
  const long index = d ? PyLong_AsLong(d) : -1;
  Py_XDECREF(h);
  Py_XDECREF(d);
  if (PyErr_Occurred()) return false;
  if (index != dev)
    return refuse(std::string(what) + ": the stream is on cuda:" + std::to_string(index) + ", the tensors on cuda:" +
                  std::to_string(dev));
  out = reinterpret_cast<attamba_stream_t>(handle);
  return true;
}

bool check(attamba_status_t st, const char* what) {
  if (st == ATTAMBA_OK) return true;
  std::string text = std::string(what) + ": " + g_status_string(st);
  const char* more = g_last_error();   // every refusal of these entry points says why
  if (more && *more) text += std::string(" (") + more + ")";
  return refuse(text);
}

bool count_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want && g_error) return true;
  PyErr_SetString(PyExc_TypeError, g_error ? "wrong number of arguments" : "_binding.init has not run");
  return false;
}

// The call's device current for as long as this lives (a plain device query where it is already).
struct OnDevice {
  c10::DeviceIndex before = -1;
  bool ok = true;
  explicit OnDevice(int dev) {
    c10::DeviceIndex now = -1;
    ok = c10::cuda::GetDevice(&now) == cudaSuccess;
    if (ok && now != dev) {
      ok = c10::cuda::SetDevice((c10::DeviceIndex)dev) == cudaSuccess;
      before = now;
    }
    if (!ok) refuse("cannot make cuda:" + std::to_string(dev) + " current");
  }
  ~OnDevice() {
    if (before >= 0) (void)c10::cuda::SetDevice(before);
  }
};

bool table(PyObject* addr, PyObject* T, PyObject* dev, const Lead& l, const attamba_seqs_t*& out) {
  int64_t t, d;
  if (!number(T, t) || !number(dev, d)) return false;
  if (t != l.rows || d != l.dev)
    return refuse("the sequence table is for " + std::to_string(t) + " token rows on cuda:" + std::to_string(d) + ", got " +
                  std::to_string(l.rows) + " on cuda:" + std::to_string(l.dev));
  out = static_cast<const attamba_seqs_t*>(PyLong_AsVoidPtr(addr));
  return !PyErr_Occurred();
}

PyObject* done(bool ok) {
  if (!ok) return nullptr;
  Py_RETURN_NONE;
}

struct Conv {
  Lead l;
  int64_t K;
  Rows x, y;
  const float *w, *bias;
  State st;
  bool read(PyObject* x_, PyObject* w_, PyObject* bias_, PyObject* state_, PyObject* y_) {
    return lead(x_, "x", l) && last_dim(w_, "w", K) && rows(x_, "x", l.dt, l.rows, l.cols, l.dev, x) &&
           rows(y_, "y", l.dt, l.rows, l.cols, l.dev, y) && mat_f32(w_, "w", l.cols, K, l.dev, w) &&
           vec_f32(bias_, "bias", l.cols, l.dev, bias) && state(state_, l.dt, K - 1, l.cols, l.dev, st);
  }
};

// x, w, bias, (table address, T, device), y, state, act, status, stream
PyObject* causal_conv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Conv v;
  const attamba_seqs_t* q = nullptr;
  int32_t act, *status;
  attamba_stream_t s;
  if (!count_is(n, 11) || !v.read(a[0], a[1], a[2], a[7], a[6]) || !table(a[3], a[4], a[5], v.l, q) ||
      !number32(a[8], "act", act) || !vec_i32(a[9], "status", 1, v.l.dev, status) ||
      !stream_of(a[10], v.l.dev, "attamba_causal_conv", s))
    return nullptr;
  const OnDevice on(v.l.dev);
  return done(on.ok && check(g_causal_conv(v.l.code, v.x.p, v.x.ld, v.w, v.bias, (int32_t)v.l.cols, (int32_t)v.K,
                                           (attamba_act_t)act, q, v.st.p, v.st.n, v.y.p, v.y.ld, status, s),
                             "attamba_causal_conv"));
}

// x, w, bias, state, y, slots, act, status, stream
PyObject* conv_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Conv v;
  int32_t act, *slots, *status;
  attamba_stream_t s;
  if (!count_is(n, 9) || !v.read(a[0], a[1], a[2], a[3], a[4]) || !vec_i32(a[5], "slots", v.l.rows, v.l.dev, slots) ||
      !number32(a[6], "act", act) || !vec_i32(a[7], "status", 1, v.l.dev, status) ||
      !stream_of(a[8], v.l.dev, "attamba_conv_step", s))
    return nullptr;
  const OnDevice on(v.l.dev);
  return done(on.ok && check(g_conv_step(v.l.code, v.x.p, v.x.ld, v.w, v.bias, (int32_t)v.l.cols, (int32_t)v.K,
                                         (attamba_act_t)act, (int32_t)v.l.rows, slots, v.st.p, v.st.n, v.y.p, v.y.ld,
                                         status, s),
                             "attamba_conv_step"));
}

// x, dt, bias, A, B, C, y, skip, z, state
struct Scan {
  Lead l;
  int64_t N;
  Rows x, dt, B, C, z, y;
  const float *bias, *A, *skip;
  State st;
  bool read(PyObject* const* a) {
    return lead(a[0], "x", l) && last_dim(a[3], "A", N) && rows(a[0], "x", l.dt, l.rows, l.cols, l.dev, x) &&
           rows(a[1], "dt", l.dt, l.rows, l.cols, l.dev, dt) && vec_f32(a[2], "bias", l.cols, l.dev, bias) &&
           mat_f32(a[3], "A", l.cols, N, l.dev, A) && rows(a[4], "B", l.dt, l.rows, N, l.dev, B) &&
           rows(a[5], "C", l.dt, l.rows, N, l.dev, C) && rows(a[6], "y", l.dt, l.rows, l.cols, l.dev, y) &&
           vec_f32(a[7], "skip", l.cols, l.dev, skip) && rows(a[8], "z", l.dt, l.rows, l.cols, l.dev, z) &&
           state(a[9], at::kFloat, N, l.cols, l.dev, st);
  }
};

// the scan's arguments, (table address, T, device), workspace, status, stream
PyObject* selective_scan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Scan v;
  const attamba_seqs_t* q = nullptr;
  void* work = nullptr;
  size_t bytes = 0;
  int32_t* status;
  attamba_stream_t s;
  if (!count_is(n, 16) || !v.read(a) || !table(a[10], a[11], a[12], v.l, q)) return nullptr;
  if (a[13] != Py_None) {
    const at::Tensor* t = tensor(a[13], "workspace");
    if (!t || !dense(a[13], "workspace", t->scalar_type(), t->sizes(), v.l.dev, work)) return nullptr;
    bytes = t->nbytes();
  }
  if (!vec_i32(a[14], "status", 1, v.l.dev, status) || !stream_of(a[15], v.l.dev, "attamba_selective_scan", s)) return nullptr;
  const OnDevice on(v.l.dev);
  return done(on.ok && check(g_selective_scan(v.l.code, v.x.p, v.x.ld, v.dt.p, v.dt.ld, v.bias, v.A, v.B.p, v.B.ld, v.C.p,
                                              v.C.ld, v.skip, v.z.p, v.z.ld, (int32_t)v.l.cols, (int32_t)v.N, q,
                                              static_cast<float*>(v.st.p), v.st.n, v.y.p, v.y.ld, work, bytes, status, s),
                             "attamba_selective_scan"));
}

// the scan's arguments, slots, status, stream
PyObject* scan_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Scan v;
  int32_t *slots, *status;
  attamba_stream_t s;
  if (!count_is(n, 13) || !v.read(a) || !vec_i32(a[10], "slots", v.l.rows, v.l.dev, slots) ||
      !vec_i32(a[11], "status", 1, v.l.dev, status) || !stream_of(a[12], v.l.dev, "attamba_scan_step", s))
    return nullptr;
  const OnDevice on(v.l.dev);
  return done(on.ok && check(g_scan_step(v.l.code, v.x.p, v.x.ld, v.dt.p, v.dt.ld, v.bias, v.A, v.B.p, v.B.ld, v.C.p, v.C.ld,
                                         v.skip, v.z.p, v.z.ld, (int32_t)v.l.cols, (int32_t)v.N, (int32_t)v.l.rows, slots,
                                         static_cast<float*>(v.st.p), v.st.n, v.y.p, v.y.ld, status, s),
                             "attamba_scan_step"));
}

// y, (table address or None, T, device), slots, stream
PyObject* clear_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Lead l;
  Rows y;
  const attamba_seqs_t* q = nullptr;
  int32_t* slots = nullptr;
  attamba_stream_t s;
  if (!count_is(n, 6) || !lead(a[0], "y", l) || !rows(a[0], "y", l.dt, l.rows, l.cols, l.dev, y) ||
      (a[1] != Py_None && !table(a[1], a[2], a[3], l, q)) || !vec_i32(a[4], "slots", l.rows, l.dev, slots) ||
      !stream_of(a[5], l.dev, "attamba_clear_rows", s))
    return nullptr;
  const OnDevice on(l.dev);
  return done(on.ok && check(g_clear_rows(l.code, y.p, y.ld, (int32_t)l.cols, q, q ? 0 : (int32_t)l.rows, slots, s),
                             "attamba_clear_rows"));
}

// y, res, res_out, h, w_post, w_pre, gate, act, gate_first, scale, alpha, eps, stream
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 13)) return nullptr;
  const bool has_y = a[0] != Py_None, has_res = a[1] != Py_None;
  if (!has_y && !has_res) return done(refuse("block_norm needs y or res"));
  Lead l;
  if (!lead(has_y ? a[0] : a[1], has_y ? "y" : "res", l)) return nullptr;
  c10::ScalarType rdt = l.dt;
  attamba_dtype_t rcode = l.code;
  if (has_y) {   // the residual stream has a type of its own
    PyObject* r = has_res ? a[1] : a[2];
    if (r != Py_None) {
      const at::Tensor* t = tensor(r, has_res ? "res" : "res_out");
      if (!t || !code_of(t->scalar_type(), has_res ? "res" : "res_out", rcode)) return nullptr;
      rdt = t->scalar_type();
    }
  } else if (a[3] != Py_None) {   // a norm alone: h has a type of its own
    const at::Tensor* t = tensor(a[3], "h");
    if (!t || !code_of(t->scalar_type(), "h", l.code)) return nullptr;
    l.dt = t->scalar_type();
  }
  const int64_t M = l.rows, D = l.cols;
  const int dev = l.dev;
  Rows y, gate, res, out, h;
  const float *w_post, *w_pre, *scale;
  int32_t act;
  float alpha, eps;
  attamba_stream_t s;
  if (!rows(a[0], "y", l.dt, M, D, dev, y) || !rows(a[6], "gate", l.dt, M, D, dev, gate) ||
      !rows(a[1], "res", rdt, M, D, dev, res) || !rows(a[2], "res_out", rdt, M, D, dev, out) ||
      !rows(a[3], "h", l.dt, M, D, dev, h) || !vec_f32(a[4], "w_post", D, dev, w_post) ||
      !vec_f32(a[5], "w_pre", D, dev, w_pre) || !vec_f32(a[9], "scale", D, dev, scale) || !number32(a[7], "gate_act", act) ||
      !real(a[10], alpha) || !real(a[11], eps) || !stream_of(a[12], dev, "attamba_block_norm", s))
    return nullptr;
  const int first = PyObject_IsTrue(a[8]);
  if (first < 0) return nullptr;
  const OnDevice on(dev);
  return done(on.ok && check(g_block_norm(l.code, rcode, y.p, y.ld, gate.p, gate.ld, (attamba_act_t)act, first, w_post, res.p,
                                          res.ld, scale, alpha, w_pre, eps, M, (int32_t)D, out.p, out.ld, h.p, h.ld, s),
                             "attamba_block_norm"));
}

// (AttambaError, addresses of attamba_status_string, _last_error, _causal_conv, _conv_step, _selective_scan, _scan_step,
// _clear_rows, _block_norm)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9) {
    PyErr_SetString(PyExc_TypeError, "init takes the error class and eight addresses");
    return nullptr;
  }
  void* f[8];
  for (int i = 0; i < 8; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_INCREF(a[0]);
  Py_XSETREF(g_error, a[0]);
  g_status_string = reinterpret_cast<decltype(g_status_string)>(f[0]);
  g_last_error = reinterpret_cast<decltype(g_last_error)>(f[1]);
  g_causal_conv = reinterpret_cast<decltype(g_causal_conv)>(f[2]);
  g_conv_step = reinterpret_cast<decltype(g_conv_step)>(f[3]);
  g_selective_scan = reinterpret_cast<decltype(g_selective_scan)>(f[4]);
  g_scan_step = reinterpret_cast<decltype(g_scan_step)>(f[5]);
  g_clear_rows = reinterpret_cast<decltype(g_clear_rows)>(f[6]);
  g_block_norm = reinterpret_cast<decltype(g_block_norm)>(f[7]);
  Py_RETURN_NONE;
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
template <Fast F> PyObject* entry(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(entry<name>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(init),      FAST(causal_conv), FAST(conv_step), FAST(selective_scan),
                           FAST(scan_step), FAST(clear_rows),  FAST(block_norm),     {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};
}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&g_module); }
