// The tensor wrappers' common case in C++: checks and the call of the C entry, without a Python call per
// attribute.  A CPython module next to libgdn.so; each function returns the entry's status, or None for
// anything it does not take (the Python wrappers then check for themselves and say what is wrong).
#include <Python.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
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

constexpr at::ScalarType kI32 = at::ScalarType::Int, kE4m3 = at::ScalarType::Float8_e4m3fn;

// Argument i as an integer of at least `least`.
int whole(Call& c, int i, long least) {
  long v = -1;
  if (c.ok && !PyLong_Check(c.argv[i])) c.ok = false;
  if (c.ok) v = PyLong_AsLong(c.argv[i]);
  if (v < least || v > 0x7fffffff) c.ok = false;
  return c.ok ? (int)v : 0;
}

// Argument i as the scores' scale, 1 / sqrt(d) for None.
float scale_of(Call& c, int i, int64_t d) {
  if (c.argv[i] == Py_None) return d > 0 ? (float)(1.0 / std::sqrt((double)d)) : 1.f;
  if (!PyFloat_Check(c.argv[i])) c.ok = false;
  return c.ok ? (float)PyFloat_AsDouble(c.argv[i]) : 0.f;
}

// A paged cache: arguments k_at, k_at + 1 and its scales s_at, s_at + 1.
template <class A>
void paged(Call& c, A& a, int k_at, int s_at, int64_t Hkv, int64_t d) {
  const Tensor* k = c.tensor(k_at);
  if (!c.ok || k->dim() != 4 || k->size(0) > 0x7fffffff || k->size(2) > 0x7fffffff) {
    c.ok = false;
    return;
  }
  const at::ScalarType type = k->scalar_type();
  const bool e4m3 = type == kE4m3;
  if (!e4m3 && type != kBf16) c.ok = false;
  const int64_t blocks = k->size(0), page = k->size(2);
  a.k_cache = c.rows(k_at, type, {blocks, Hkv, page, d}, a.k_block_stride);
  a.v_cache = c.rows(k_at + 1, type, {blocks, Hkv, page, d}, a.v_block_stride);
  if (e4m3) {
    a.k_scale = static_cast<const float*>(c.plain(s_at, kF32, {Hkv}));
    a.v_scale = static_cast<const float*>(c.plain(s_at + 1, kF32, {Hkv}));
  } else if (c.argv[s_at] != Py_None || c.argv[s_at + 1] != Py_None) {
    c.ok = false;
  }
  a.blocks = (int)blocks;
  a.page = (int)page;
  a.flags = e4m3 ? GDN_CACHE_E4M3 : 0;
}

template <class A>
void workspace(Call& c, A& a, int i) {
  if (const Tensor* w = c.tensor(i, true)) {
    if (!w->is_contiguous() || w->nbytes() == 0) c.ok = false;
    a.workspace = w->data_ptr();
    a.workspace_bytes = w->nbytes();
  }
}

// cache_plan(lens, block_table, free_blocks, free_count, cu_seqlens, page, T, slots, new_lens, new_count, refused,
// stream)
PyObject* plan(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 12) return none();
    Call c(argv);
    gdn_cache_plan_args a = {};
    const Tensor *lens = c.tensor(0), *table = c.tensor(1), *free_blocks = c.tensor(2), *slots = c.tensor(7);
    if (!c.ok || lens->dim() != 1 || table->dim() != 2 || free_blocks->dim() != 1 || slots->dim() != 1) return none();
    const int64_t B = lens->size(0), W = table->size(1), capacity = free_blocks->size(0), T = slots->size(0);
    if (B > 0x7ffffffe || W > 0x7fffffff || capacity > 0x7fffffff || T > 0x7fffffff) return none();
    if (argv[6] != Py_None && (whole(c, 6, 0) != T || !c.ok)) return none();
    if (argv[4] == Py_None && T != B) return none();
    a.lens = static_cast<const int32_t*>(c.plain(0, kI32, {B}));
    a.block_table = static_cast<int32_t*>(c.rows(1, kI32, {B, W}, a.table_stride));
    a.free_blocks = static_cast<const int32_t*>(c.plain(2, kI32, {capacity}));
    a.free_count = static_cast<const int32_t*>(c.plain(3, kI32, {1}));
    a.cu_seqlens = static_cast<const int32_t*>(c.plain(4, kI32, {B + 1}, true));
    a.slots = static_cast<int32_t*>(c.plain(7, kI32, {T}));
    a.new_lens = static_cast<int32_t*>(c.plain(8, kI32, {B}));
    a.new_count = static_cast<int32_t*>(c.plain(9, kI32, {1}));
    a.refused = static_cast<int32_t*>(c.plain(10, kI32, {1}));
    a.B = (int)B;
    a.T = (int)T;
    a.W = (int)W;
    a.capacity = (int)capacity;
    a.page = whole(c, 5, 1);
    a.stream = c.stream(11);
    return c.ok ? PyLong_FromLong(gdn_cache_plan(&a)) : none();
  });
}

// cache_append(k, v, k_cache, v_cache, slots, k_scale, v_scale, stream)
PyObject* append(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 8) return none();
    Call c(argv);
    gdn_cache_append_args a = {};
    const Tensor* k = c.tensor(0);
    if (!c.ok || k->dim() != 3 || k->size(0) > 0x7fffffff || k->size(1) > 0x7fffffff || k->size(2) > 0x7fffffff)
      return none();
    const int64_t T = k->size(0), Hkv = k->size(1), d = k->size(2);
    a.k = c.rows(0, kBf16, {T, Hkv, d}, a.k_stride);
    a.v = c.rows(1, kBf16, {T, Hkv, d}, a.v_stride);
    paged(c, a, 2, 5, Hkv, d);
    a.slots = static_cast<const int32_t*>(c.plain(4, kI32, {T}));
    a.T = (int)T;
    a.Hkv = (int)Hkv;
    a.d = (int)d;
    a.stream = c.stream(7);
    return c.ok ? PyLong_FromLong(gdn_cache_append(&a)) : none();
  });
}

// attention(q, k, v, cu_seqlens, cu_seqlens_k, B, window, sinks, scale, out, lse, workspace, stream)
PyObject* attn(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 13) return none();
    Call c(argv);
    gdn_attn_args a = {};
    const Tensor *q = c.tensor(0), *k = c.tensor(1);
    if (!c.ok || q->dim() != 3 || k->dim() != 3) return none();
    for (int i = 0; i < 3; ++i)
      if (q->size(i) > 0x7fffffff || k->size(i) > 0x7fffffff) return none();
    const int64_t T = q->size(0), Hq = q->size(1), d = q->size(2), Tk = k->size(0), Hkv = k->size(1);
    a.q = c.rows(0, kBf16, {T, Hq, d}, a.q_stride);
    a.k = c.rows(1, kBf16, {Tk, Hkv, d}, a.k_stride);
    a.v = c.rows(2, kBf16, {Tk, Hkv, d}, a.v_stride);
    if (!c.ok || !batch(c, T, 3, 5, a.cu_seqlens, a.B, a.T)) return none();
    if (a.cu_seqlens == nullptr) {
      if (argv[4] != Py_None || Tk % a.B != 0) return none();
      a.Tk = (int)(Tk / a.B);
    } else {
      if (argv[4] == Py_None && Tk != T) return none();
      a.cu_seqlens_k = static_cast<const int32_t*>(c.plain(4, kI32, {a.B + 1}, true));
      a.Tk = (int)Tk;
    }
    a.window = whole(c, 6, 0);
    a.sinks = whole(c, 7, 0);
    a.scale = scale_of(c, 8, d);
    a.out = c.plain(9, kBf16, {T, Hq, d});
    a.lse = static_cast<float*>(c.plain(10, kF32, {T, Hq}, true));
    workspace(c, a, 11);
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.d = (int)d;
    a.stream = c.stream(12);
    return c.ok ? PyLong_FromLong(gdn_attn(&a)) : none();
  });
}

// attention_step(q, k_cache, v_cache, block_table, lens, k_scale, v_scale, window, sinks, scale, out, lse, workspace,
// stream)
PyObject* attn_step(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 14) return none();
    Call c(argv);
    gdn_attn_step_args a = {};
    const Tensor *q = c.tensor(0), *k = c.tensor(1), *table = c.tensor(3);
    if (!c.ok || q->dim() != 3 || k->dim() != 4 || table->dim() != 2 || table->size(1) > 0x7fffffff) return none();
    for (int i = 0; i < 3; ++i)
      if (q->size(i) > 0x7fffffff || k->size(i) > 0x7fffffff) return none();
    const int64_t B = q->size(0), Hq = q->size(1), d = q->size(2), Hkv = k->size(1), W = table->size(1);
    a.q = c.rows(0, kBf16, {B, Hq, d}, a.q_stride);
    paged(c, a, 1, 5, Hkv, d);
    a.block_table = static_cast<const int32_t*>(c.rows(3, kI32, {B, W}, a.table_stride));
    a.lens = static_cast<const int32_t*>(c.plain(4, kI32, {B}));
    a.window = whole(c, 7, 0);
    a.sinks = whole(c, 8, 0);
    a.scale = scale_of(c, 9, d);
    a.out = c.plain(10, kBf16, {B, Hq, d});
    a.lse = static_cast<float*>(c.plain(11, kF32, {B, Hq}, true));
    workspace(c, a, 12);
    a.B = (int)B;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.d = (int)d;
    a.W = (int)W;
    a.stream = c.stream(13);
    return c.ok ? PyLong_FromLong(gdn_attn_step(&a)) : none();
  });
}

#define GDN_METHOD(name, f) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GDN_METHOD("causal_conv", conv), GDN_METHOD("causal_conv_step", conv_step),
                         GDN_METHOD("ssm_scan", scan),    GDN_METHOD("ssm_step", step),
                         GDN_METHOD("add_norm", norm),    GDN_METHOD("cache_plan", plan),
                         GDN_METHOD("cache_append", append), GDN_METHOD("attention", attn),
                         GDN_METHOD("attention_step", attn_step), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "gdn_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gdn_torch(void) { return PyModule_Create(&module); }
