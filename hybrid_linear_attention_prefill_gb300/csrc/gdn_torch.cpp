// The tensor wrappers' common case in C++: checks and the call of the C entry, without a Python call per
// attribute.  A CPython module next to libgdn.so; each function returns the entry's status, or None for
// anything it does not take (the Python wrappers then check for themselves and say what is wrong).
#include <Python.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "gdn.h"

namespace {

using at::Tensor;

struct Call {
  bool ok = true;
  int dev = -1;
  PyObject* const* argv;

  explicit Call(PyObject* const* a) : argv(a) {}

  // Argument i as a tensor, or null for None.
  const Tensor* tensor(int i, bool optional = false) {
    PyObject* o = argv[i];
    if (o == Py_None && optional) return nullptr;
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || (dev >= 0 && t.get_device() != dev)) ok = false;
    if (ok && dev < 0) dev = (int)t.get_device();
    return ok ? &t : nullptr;
  }
  static bool same(const Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape) {
    return t.scalar_type() == type && t.sizes() == at::IntArrayRef(shape.begin(), shape.size());
  }
  // Address of a contiguous tensor of this type and shape; null for None.
  void* plain(int i, at::ScalarType type, std::initializer_list<int64_t> shape, bool optional = false) {
    const Tensor* t = tensor(i, optional);
    if (t == nullptr) return nullptr;
    if (!same(*t, type, shape) || !t->is_contiguous()) ok = false;
    return ok ? t->data_ptr() : nullptr;
  }
  // Address and row stride of a tensor whose rows are contiguous.
  void* rows(int i, at::ScalarType type, std::initializer_list<int64_t> shape, long long& stride,
             bool optional = false) {
    stride = 0;
    const Tensor* t = tensor(i, optional);
    if (t == nullptr) return nullptr;
    if (!same(*t, type, shape)) ok = false;
    long long width = 1;
    for (int64_t d = t->dim() - 1; ok && d > 0; --d) {
      if (t->size(d) != 1 && t->stride(d) != width) ok = false;
      width *= t->size(d);
    }
    if (!ok) return nullptr;
    stride = t->size(0) > 1 ? t->stride(0) : width;
    return t->data_ptr();
  }
  // The stream of a call on the current device (one on another is for the Python way, which makes that current).
  void* stream(int i) {
    PyObject* o = argv[i];
    if (ok && c10::cuda::current_device() != dev) ok = false;
    if (!ok) return nullptr;
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    if (!PyLong_Check(o)) {
      ok = false;
      return nullptr;
    }
    return PyLong_AsVoidPtr(o);
  }
  bool flag(int i) {
    const int yes = PyObject_IsTrue(argv[i]);
    if (yes < 0) ok = false;
    return yes == 1;
  }
};

// Left to the Python checks, which meet the same arguments and raise for themselves.
PyObject* none() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

// A C++ exception does not cross into the interpreter: what it was is for the Python checks to say.
template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return none();
  }
}

constexpr at::ScalarType kBf16 = at::ScalarType::BFloat16, kF32 = at::ScalarType::Float;

// (sequences, tokens) of n rows from the boundaries (argument cu_at) or the count (argument b_at).
bool batch(Call& c, int64_t n, int cu_at, int b_at, const int32_t*& cu, int& B, int& T) {
  cu = nullptr;
  if (c.argv[cu_at] != Py_None) {
    const Tensor* t = c.tensor(cu_at);
    if (t == nullptr || t->scalar_type() != at::ScalarType::Int || t->dim() != 1 || t->numel() < 1 ||
        !t->is_contiguous())
      return false;
    cu = static_cast<const int32_t*>(t->data_ptr());
    B = (int)(t->numel() - 1);
    T = (int)n;
    return true;
  }
  long b = 1;
  if (c.argv[b_at] != Py_None) {
    if (!PyLong_Check(c.argv[b_at])) return false;
    b = PyLong_AsLong(c.argv[b_at]);
  }
  if (b < 1 || b > 0x7fffffff || n % b != 0) return false;
  B = (int)b;
  T = (int)(n / b);
  return true;
}

// causal_conv(x, weight, bias, cu_seqlens, init_state, B, silu, out, final_state, stream)
PyObject* conv(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 10) return none();
    Call c(argv);
    gdn_conv_args a = {};
    const Tensor *x = c.tensor(0), *w = c.tensor(1);
    if (!c.ok || x->dim() != 2 || w->dim() != 2 || x->size(0) > 0x7fffffff) return none();
    const int64_t rows = x->size(0), C = w->size(0), K = w->size(1);
    a.x = c.rows(0, kBf16, {rows, C}, a.x_stride);
    a.weight = c.plain(1, kBf16, {C, K});
    a.bias = c.plain(2, kBf16, {C}, true);
    if (!c.ok || !batch(c, rows, 3, 5, a.cu_seqlens, a.B, a.T)) return none();
    a.init_state = c.plain(4, kBf16, {a.B, K - 1, C}, true);
    a.out = c.plain(7, kBf16, {rows, C});
    a.final_state = c.plain(8, kBf16, {a.B, K - 1, C}, true);
    a.C = (int)C;
    a.K = (int)K;
    a.flags = c.flag(6) ? GDN_CONV_SILU : 0;
    a.stream = c.stream(9);
    return c.ok ? PyLong_FromLong(gdn_conv(&a)) : none();
  });
}

// causal_conv_step(x, weight, state, bias, silu, out, stream)
PyObject* conv_step(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 7) return none();
    Call c(argv);
    gdn_conv_step_args a = {};
    const Tensor *x = c.tensor(0), *w = c.tensor(1);
    if (!c.ok || x->dim() != 2 || w->dim() != 2 || x->size(0) > 0x7fffffff) return none();
    const int64_t B = x->size(0), C = w->size(0), K = w->size(1);
    a.x = c.rows(0, kBf16, {B, C}, a.x_stride);
    a.weight = c.plain(1, kBf16, {C, K});
    a.state = c.plain(2, kBf16, {B, K - 1, C});
    a.bias = c.plain(3, kBf16, {C}, true);
    a.out = c.plain(5, kBf16, {B, C});
    a.B = (int)B;
    a.C = (int)C;
    a.K = (int)K;
    a.flags = c.flag(4) ? GDN_CONV_SILU : 0;
    a.stream = c.stream(6);
    return c.ok ? PyLong_FromLong(gdn_conv_step(&a)) : none();
  });
}

// The operands that the scan and its step share: argv x, dt, A, Bm, Cm at 0..4, D, z, dt_bias at d_at.., out.
template <class A>
bool ssm_operands(Call& c, A& a, int d_at, int out_at, int softplus_at, int64_t& rows) {
  const Tensor *x = c.tensor(0), *dt = c.tensor(1), *bm = c.tensor(3);
  if (!c.ok || x->dim() != 3 || bm->dim() != 3 || x->size(0) > 0x7fffffff) return false;
  rows = x->size(0);
  const int64_t Hv = x->size(1), dv = x->size(2), Hk = bm->size(1), dk = bm->size(2);
  const bool f32 = dt->scalar_type() == kF32;
  a.x = c.rows(0, kBf16, {rows, Hv, dv}, a.x_stride);
  a.dt = c.rows(1, f32 ? kF32 : kBf16, {rows, Hv}, a.dt_stride);
  a.A = static_cast<const float*>(c.plain(2, kF32, {Hv}));
  a.Bm = c.rows(3, kBf16, {rows, Hk, dk}, a.b_stride);
  a.Cm = c.rows(4, kBf16, {rows, Hk, dk}, a.c_stride);
  a.D = static_cast<const float*>(c.plain(d_at, kF32, {Hv}, true));
  a.z = c.rows(d_at + 1, kBf16, {rows, Hv, dv}, a.z_stride, true);
  a.dt_bias = static_cast<const float*>(c.plain(d_at + 2, kF32, {Hv}, true));
  a.out = c.plain(out_at, kBf16, {rows, Hv, dv});
  a.Hk = (int)Hk;
  a.Hv = (int)Hv;
  a.dk = (int)dk;
  a.dv = (int)dv;
  a.flags = (f32 ? GDN_SSM_DT_F32 : 0) | (c.flag(softplus_at) ? GDN_SSM_SOFTPLUS : 0);
  return c.ok;
}

// ssm_scan(x, dt, A, Bm, Cm, D, z, dt_bias, cu_seqlens, init_state, B, softplus, out, final_state, workspace, stream)
PyObject* scan(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 16) return none();
    Call c(argv);
    gdn_ssm_scan_args a = {};
    int64_t rows = 0;
    if (!ssm_operands(c, a, 5, 12, 11, rows) || !batch(c, rows, 8, 10, a.cu_seqlens, a.B, a.T)) return none();
    a.init_state = static_cast<const float*>(c.plain(9, kF32, {a.B, a.Hv, a.dv, a.dk}, true));
    a.final_state = static_cast<float*>(c.plain(13, kF32, {a.B, a.Hv, a.dv, a.dk}, true));
    if (const Tensor* w = c.tensor(14, true)) {
      if (!w->is_contiguous()) return none();
      a.workspace = w->data_ptr();
      a.workspace_bytes = w->nbytes();
    }
    a.stream = c.stream(15);
    return c.ok ? PyLong_FromLong(gdn_ssm_scan(&a)) : none();
  });
}

// ssm_step(x, dt, A, Bm, Cm, state, D, z, dt_bias, softplus, out, stream)
PyObject* step(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 12) return none();
    Call c(argv);
    gdn_ssm_step_args a = {};
    int64_t rows = 0;
    if (!ssm_operands(c, a, 6, 10, 9, rows)) return none();
    a.B = (int)rows;
    a.state = static_cast<float*>(c.plain(5, kF32, {rows, a.Hv, a.dv, a.dk}));
    a.stream = c.stream(11);
    return c.ok ? PyLong_FromLong(gdn_ssm_step(&a)) : none();
  });
}

// add_norm(x, weight, residual, eps, group, out, scales, residual_out, stream)
PyObject* norm(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 9 || !PyFloat_Check(argv[3]) || !PyLong_Check(argv[4])) return none();
    Call c(argv);
    gdn_add_norm_args a = {};
    const Tensor *x = c.tensor(0), *out = c.tensor(5);
    if (!c.ok || x->dim() != 2 || x->size(0) > 0x7fffffff || x->size(1) > 0x7fffffff) return none();
    const int64_t rows = x->size(0), D = x->size(1);
    const long group = PyLong_AsLong(argv[4]);
    if (group < 0 || group > D + 0x10000) return none();
    const bool e4m3 = out->scalar_type() == at::ScalarType::Float8_e4m3fn;
    a.x = c.rows(0, kBf16, {rows, D}, a.x_stride);
    a.weight = c.plain(1, kBf16, {D});
    a.residual = c.plain(2, kBf16, {rows, D}, true);
    a.out = c.plain(5, e4m3 ? at::ScalarType::Float8_e4m3fn : kBf16, {rows, D});
    if (!e4m3 && argv[6] != Py_None) return none();  // scales that the call does not write
    if (e4m3) a.scales = static_cast<float*>(c.plain(6, kF32, {rows, group ? (D + group - 1) / group : 1}));
    a.residual_out = c.plain(7, kBf16, {rows, D}, true);
    a.rows = (int)rows;
    a.D = (int)D;
    a.group = (int)group;
    a.eps = (float)PyFloat_AsDouble(argv[3]);
    a.flags = e4m3 ? GDN_NORM_E4M3 : 0;
    a.stream = c.stream(8);
    return c.ok ? PyLong_FromLong(gdn_add_norm(&a)) : none();
  });
}

#define GDN_METHOD(name, f) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GDN_METHOD("causal_conv", conv), GDN_METHOD("causal_conv_step", conv_step),
                         GDN_METHOD("ssm_scan", scan),    GDN_METHOD("ssm_step", step),
                         GDN_METHOD("add_norm", norm),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "gdn_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gdn_torch(void) { return PyModule_Create(&module); }
