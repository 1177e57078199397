// The Python side of the batched adapters' and the 8-bit calls in C++: these
// calls are a few kernel launches on tensors that take microseconds, and a dozen
// tensors checked, allocated and passed one by one from Python took longer than
// the kernels (a single-token forward of the adapters: 14 of 20 us).  Argument marshalling only;
// the functions themselves are the C ABI's (include/qlora.h), given by address.
//
// Each call checks its tensors like the binding's checker (type, shape,
// contiguity, one HIP device) and returns None where one fails, for the
// checker to name; else (status, outputs...).  An output that overlaps an input
// or another output raises ValueError here.  Outputs that are not given, and
// scratch memory where no workspace is given, come from torch's allocator on
// the current stream of the tensors' device, on which the call is made.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/qlora.h"

namespace {

decltype(&lora_adapter_tiles) g_tiles;
decltype(&lora_adapter_plan) g_plan;
decltype(&lora_adapters_workspace_bytes) g_ws;
decltype(&lora_adapters_fwd) g_fwd;
decltype(&lora_adapters_bwd) g_bwd;
decltype(&int8_quantize) g_q8;
decltype(&int8_quantize_fp32) g_q8_fp32;
decltype(&int8_dequant) g_dq8;
decltype(&int8_linear_workspace_bytes) g_ws8;
decltype(&int8_linear_fwd) g_fwd8;
decltype(&int8_linear_bwd) g_bwd8;
decltype(&qlora_linear_bwd_int8) g_bwd8_nf4;
decltype(&qlora_linear_bwd_bf16_int8) g_bwd8_bf16;
decltype(&silu_mul_fwd_int8) g_silu8;
decltype(&silu_mul_bwd_int8) g_silu8_bwd;

// Tensors of one call: each must be a contiguous tensor of its type and shape
// on the first one's device.
struct Checked {
  c10::Device device{c10::kCPU};
  bool ok = true, any = false;

  const at::Tensor* one(PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
    if (!THPVariable_Check(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided || t.scalar_type() != type || t.sizes() != shape ||
        !t.is_contiguous() || !t.is_cuda())
      return fail();
    if (!any) device = t.device();
    any = true;
    return t.device() == device ? &t : fail();
  }
  const at::Tensor* opt(PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
    return o == Py_None ? nullptr : one(o, type, shape);
  }
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
};

template <class T>
T* ptr(const at::Tensor* t) {
  return t ? reinterpret_cast<T*>(t->data_ptr()) : nullptr;
}
at::Tensor fresh(const Checked& c, at::ScalarType type, at::IntArrayRef shape) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(c.device));
}
void* stream_of(const Checked& c) {
  return c10::hip::getCurrentHIPStream(c.device.index()).stream();
}
// Sizes of a tensor of `dims` dimensions.
bool sizes(PyObject* o, int dims, int64_t* out) {
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.dim() != dims) return false;
  for (int i = 0; i < dims; ++i) out[i] = t.size(i);
  return true;
}

// X, A, B, scale and the plan (a tuple token_slot, order, start, tiles, S).
struct Batch {
  int64_t M, K, N;
  int r, S;
  const at::Tensor *X, *A, *B, *scale, *order, *start, *tiles;

  bool take(Checked& c, PyObject* x, PyObject* a, PyObject* b, PyObject* s, PyObject* plan) {
    int64_t sx[2], sa[3], sb[3];
    if (!sizes(x, 2, sx) || !sizes(a, 3, sa) || !sizes(b, 3, sb) || !PyTuple_Check(plan) ||
        PyTuple_GET_SIZE(plan) != 5)
      return false;
    M = sx[0]; K = sx[1]; N = sb[1];
    const long ps = PyLong_AsLong(PyTuple_GET_ITEM(plan, 4));
    if (ps == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      return false;
    }
    if (ps != sa[0] || sa[0] > (1 << 30) || sa[1] > (1 << 30)) return false;
    S = (int)sa[0]; r = (int)sa[1];
    X = c.one(x, at::kBFloat16, {M, K});
    A = c.one(a, at::kBFloat16, {sa[0], sa[1], K});
    B = c.one(b, at::kBFloat16, {sa[0], N, sa[1]});
    scale = c.one(s, at::kFloat, {sa[0]});
    order = c.one(PyTuple_GET_ITEM(plan, 1), at::kInt, {M});
    start = c.one(PyTuple_GET_ITEM(plan, 2), at::kInt, {sa[0] + 2});
    tiles = c.one(PyTuple_GET_ITEM(plan, 3), at::kInt, {g_tiles(M, S), 3});
    return c.ok && tiles->size(0) > 0;
  }
};

struct Named {
  const char* name;
  const at::Tensor* t;   // null: not given
};
bool overlap(const at::Tensor& a, const at::Tensor& b) {
  const char* const p = static_cast<const char*>(a.data_ptr());
  const char* const q = static_cast<const char*>(b.data_ptr());
  return p < q + b.nbytes() && q < p + a.nbytes();
}
// False, with Python's ValueError set, where an output given by the caller
// shares memory with an input or another output.  The first output may be
// `base`, the tensor it adds to, itself.
bool apart(std::initializer_list<Named> outs, std::initializer_list<Named> ins, Named base) {
  for (const Named* o = outs.begin(); o != outs.end(); ++o) {
    if (!o->t) continue;
    const bool adds = o == outs.begin() && base.t && o->t->data_ptr() == base.t->data_ptr();
    const Named* with = !adds && base.t && overlap(*o->t, *base.t) ? &base : nullptr;
    for (const Named& i : ins)
      if (i.t && overlap(*o->t, *i.t)) with = &i;
    for (const Named* p = outs.begin(); p != o; ++p)
      if (p->t && overlap(*o->t, *p->t)) with = p;
    if (with) {
      PyErr_Format(PyExc_ValueError, "%s: overlaps %s", o->name, with->name);
      return false;
    }
  }
  return true;
}

// The given workspace's memory, or fresh scratch of `need` bytes (held by
// `own`).  A 1-D byte tensor that is too small is the library's to refuse.
void* scratch(Checked& c, PyObject* o, size_t need, at::Tensor& own, size_t* bytes) {
  if (o != Py_None) {
    int64_t n[1];
    if (!sizes(o, 1, n)) {
      c.fail();
      return nullptr;
    }
    const at::Tensor* t = c.one(o, at::kByte, {n[0]});
    *bytes = (size_t)n[0];
    return ptr<void>(t);
  }
  *bytes = need;
  if (need == 0) return nullptr;
  own = fresh(c, at::kByte, {(int64_t)need});
  return own.data_ptr();
}

PyObject* none() { Py_RETURN_NONE; }

// ATen's errors (out of memory, a lost device) as Python's.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

bool number(PyObject* o, double* out) {
  *out = PyFloat_AsDouble(o);
  return !(*out == -1.0 && PyErr_Occurred());
}

// plan(slots, lengths | None, M, S) -> None or (status, token_slot, order, start, tiles)
PyObject* call_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) return PyErr_Format(PyExc_TypeError, "plan takes 4 arguments");
  return guarded([&]() -> PyObject* {
    Checked c;
    int64_t q[1];
    if (!sizes(a[0], 1, q)) return none();
    const at::Tensor* slots = c.one(a[0], at::kInt, {q[0]});
    const at::Tensor* lengths = c.opt(a[1], at::kInt, {q[0]});
    if (!c.ok) return none();
    const long long M = PyLong_AsLongLong(a[2]), S = PyLong_AsLongLong(a[3]);
    if ((M == -1 || S == -1) && PyErr_Occurred()) return nullptr;
    const int64_t nt = S < 1 || S > (1 << 30) ? 0 : g_tiles(M, (int)S);
    if (nt <= 0) return Py_BuildValue("(i)", QLORA_ERR_SHAPE);
    const c10::DeviceGuard guard(c.device);
    const at::Tensor t0 = fresh(c, at::kInt, {M}), t1 = fresh(c, at::kInt, {M}),
                     t2 = fresh(c, at::kInt, {S + 2}), t3 = fresh(c, at::kInt, {nt, 3});
    const int st = g_plan(ptr<int32_t>(lengths), q[0] ? ptr<int32_t>(slots) : nullptr, q[0], M,
                          (int)S, ptr<int32_t>(&t0), ptr<int32_t>(&t1), ptr<int32_t>(&t2),
                          ptr<int32_t>(&t3), stream_of(c));
    return Py_BuildValue("(iNNNN)", st, THPVariable_Wrap(t0), THPVariable_Wrap(t1),
                         THPVariable_Wrap(t2), THPVariable_Wrap(t3));
  });
}

// fwd(X, Y | None, A, B, scale, plan, p, seed, save_T, out | None, T_out | None, ws | None)
//   -> None or (status, out, T | None)
PyObject* call_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 12) return PyErr_Format(PyExc_TypeError, "fwd takes 12 arguments");
  return guarded([&]() -> PyObject* {
    Checked c;
    Batch b;
    if (!b.take(c, a[0], a[2], a[3], a[4], a[5])) return none();
    const at::Tensor* Y = c.opt(a[1], at::kBFloat16, {b.M, b.N});
    const at::Tensor* out = c.opt(a[9], at::kBFloat16, {b.M, b.N});
    const at::Tensor* T = c.opt(a[10], at::kFloat, {b.M, b.r});
    double p;
    if (!number(a[6], &p)) return nullptr;
    const uint64_t seed = PyLong_AsUnsignedLongLong(a[7]);
    if (seed == (uint64_t)-1 && PyErr_Occurred()) return nullptr;
    const int save = PyObject_IsTrue(a[8]);
    if (save < 0) return nullptr;
    if (!c.ok) return none();
    if (!apart({{"out", out}, {"T_out", T}},
               {{"X", b.X}, {"A", b.A}, {"B", b.B}, {"scale", b.scale}, {"plan", b.order},
                {"plan", b.start}, {"plan", b.tiles}}, {"Y", Y}))
      return nullptr;
    const c10::DeviceGuard guard(c.device);
    at::Tensor own_out, own_T, own_ws;
    if (!out) out = &(own_out = fresh(c, at::kBFloat16, {b.M, b.N}));
    if (!T && save) T = &(own_T = fresh(c, at::kFloat, {b.M, b.r}));
    size_t bytes;
    void* ws = scratch(c, a[11], g_ws(b.M, b.K, b.N, b.r, b.S, 0), own_ws, &bytes);
    if (!c.ok) return none();
    const int st = g_fwd(ptr<uint16_t>(b.X), b.M, b.K, b.N, ptr<uint16_t>(b.A), ptr<uint16_t>(b.B),
                         ptr<float>(b.scale), b.r, b.S, ptr<int32_t>(b.order),
                         ptr<int32_t>(b.start), ptr<int32_t>(b.tiles), ptr<uint16_t>(Y), p, seed,
                         ptr<uint16_t>(out), ptr<float>(T), ws, bytes, stream_of(c));
    return Py_BuildValue("(iNN)", st, THPVariable_Wrap(*out), T ? THPVariable_Wrap(*T) : none());
  });
}

// bwd(dY, X, A, B, scale, plan, T | None, dX0 | None, p, seed, need_dX, dX_out | None,
//     dA_out | None, dB_out | None, ws | None) -> None or (status, dX | None, dA, dB)
PyObject* call_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 15) return PyErr_Format(PyExc_TypeError, "bwd takes 15 arguments");
  return guarded([&]() -> PyObject* {
    Checked c;
    Batch b;
    if (!b.take(c, a[1], a[2], a[3], a[4], a[5])) return none();
    const at::Tensor* dY = c.one(a[0], at::kBFloat16, {b.M, b.N});
    const at::Tensor* T = c.opt(a[6], at::kFloat, {b.M, b.r});
    const at::Tensor* dX0 = c.opt(a[7], at::kBFloat16, {b.M, b.K});
    const at::Tensor* dX = c.opt(a[11], at::kBFloat16, {b.M, b.K});
    const at::Tensor* dA = c.opt(a[12], at::kFloat, {b.S, b.r, b.K});
    const at::Tensor* dB = c.opt(a[13], at::kFloat, {b.S, b.N, b.r});
    double p;
    if (!number(a[8], &p)) return nullptr;
    const uint64_t seed = PyLong_AsUnsignedLongLong(a[9]);
    if (seed == (uint64_t)-1 && PyErr_Occurred()) return nullptr;
    const int need = PyObject_IsTrue(a[10]);
    if (need < 0) return nullptr;
    if (!c.ok) return none();
    if (!apart({{"dX_out", dX}, {"dA", dA}, {"dB", dB}},
               {{"dY", dY}, {"X", b.X}, {"A", b.A}, {"B", b.B}, {"scale", b.scale}, {"T", T},
                {"plan", b.order}, {"plan", b.start}, {"plan", b.tiles}}, {"dX", dX0}))
      return nullptr;
    const c10::DeviceGuard guard(c.device);
    at::Tensor own_dX, own_dA, own_dB, own_ws;
    if (!dX && need) dX = &(own_dX = fresh(c, at::kBFloat16, {b.M, b.K}));
    if (!dA) dA = &(own_dA = fresh(c, at::kFloat, {b.S, b.r, b.K}));
    if (!dB) dB = &(own_dB = fresh(c, at::kFloat, {b.S, b.N, b.r}));
    size_t bytes;
    void* ws = scratch(c, a[14], g_ws(b.M, b.K, b.N, b.r, b.S, 1), own_ws, &bytes);
    if (!c.ok) return none();
    const int st = g_bwd(ptr<uint16_t>(dY), ptr<uint16_t>(b.X), b.M, b.K, b.N, ptr<uint16_t>(b.A),
                         ptr<uint16_t>(b.B), ptr<float>(b.scale), b.r, b.S, ptr<int32_t>(b.order),
                         ptr<int32_t>(b.start), ptr<int32_t>(b.tiles), ptr<float>(T),
                         ptr<uint16_t>(dX0), p, seed, ptr<uint16_t>(dX), ptr<float>(dA),
                         ptr<float>(dB), ws, bytes, stream_of(c));
    return Py_BuildValue("(iNNN)", st, dX ? THPVariable_Wrap(*dX) : none(), THPVariable_Wrap(*dA),
                         THPVariable_Wrap(*dB));
  });
}

// bind(tiles, plan, workspace_bytes, fwd, bwd): addresses of the C ABI's functions.
PyObject* call_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) return PyErr_Format(PyExc_TypeError, "bind takes 5 addresses");
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "null address");
  }
  g_tiles = reinterpret_cast<decltype(g_tiles)>(p[0]);
  g_plan = reinterpret_cast<decltype(g_plan)>(p[1]);
  g_ws = reinterpret_cast<decltype(g_ws)>(p[2]);
  g_fwd = reinterpret_cast<decltype(g_fwd)>(p[3]);
  g_bwd = reinterpret_cast<decltype(g_bwd)>(p[4]);
  return none();
}

// ---- activations and weights in 8 bits --------------------------------------

// Codes [rows, cols] and scales: one per row, or one per 64 columns.
struct Codes {
  const at::Tensor *codes = nullptr, *scale = nullptr;
  int64_t rows = 0, cols = 0;
  bool block = false;

  bool take(Checked& c, PyObject* o) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) return false;
    return take(c, PyTuple_GET_ITEM(o, 0), PyTuple_GET_ITEM(o, 1));
  }
  bool take(Checked& c, PyObject* oc, PyObject* os) {
    int64_t s[2];
    if (!sizes(oc, 2, s) || !THPVariable_Check(os)) return false;
    rows = s[0]; cols = s[1];
    block = THPVariable_Unpack(os).dim() == 2;
    codes = c.one(oc, at::kChar, {rows, cols});
    scale = block ? c.one(os, at::kFloat, {rows, cols / 64}) : c.one(os, at::kFloat, {rows});
    return c.ok && (!block || cols % 64 == 0);
  }
};

// quantize(X, codes_out | None, scale_out | None) -> None or (status, codes, scale)
PyObject* call_quantize8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3) return PyErr_Format(PyExc_TypeError, "quantize8 takes 3 arguments");
  return guarded([&]() -> PyObject* {
    Checked c;
    int64_t s[2];
    if (!sizes(a[0], 2, s)) return none();
    const bool wide = THPVariable_Unpack(a[0]).scalar_type() == at::kFloat;
    const at::Tensor* X = c.one(a[0], wide ? at::kFloat : at::kBFloat16, {s[0], s[1]});
    const at::Tensor* codes = c.opt(a[1], at::kChar, {s[0], s[1]});
    const at::Tensor* scale = c.opt(a[2], at::kFloat, {s[0]});
    if (!c.ok) return none();
    if (!apart({{"codes_out", codes}, {"scale_out", scale}}, {{"X", X}}, {})) return nullptr;
    const c10::DeviceGuard guard(c.device);
    at::Tensor own_c, own_s;
    if (!codes) codes = &(own_c = fresh(c, at::kChar, {s[0], s[1]}));
    if (!scale) scale = &(own_s = fresh(c, at::kFloat, {s[0]}));
    const int st = wide ? g_q8_fp32(ptr<float>(X), s[0], s[1], ptr<int8_t>(codes), ptr<float>(scale),
                                    stream_of(c))
                        : g_q8(ptr<uint16_t>(X), s[0], s[1], ptr<int8_t>(codes), ptr<float>(scale),
                               stream_of(c));
    return Py_BuildValue("(iNN)", st, THPVariable_Wrap(*codes), THPVariable_Wrap(*scale));
  });
}

// dequant(codes, scale, out | None) -> None or (status, out)
PyObject* call_dequant8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3) return PyErr_Format(PyExc_TypeError, "dequant8 takes 3 arguments");
  return guarded([&]() -> PyObject* {
    Checked c;
    Codes x;
    if (!x.take(c, a[0], a[1])) return none();
    const at::Tensor* out = c.opt(a[2], at::kBFloat16, {x.rows, x.cols});
    if (!c.ok) return none();
    if (!apart({{"out", out}}, {{"codes", x.codes}, {"scale", x.scale}}, {})) return nullptr;
    const c10::DeviceGuard guard(c.device);
    at::Tensor own;
    if (!out) out = &(own = fresh(c, at::kBFloat16, {x.rows, x.cols}));
    const int st = g_dq8(ptr<int8_t>(x.codes), ptr<float>(x.scale), x.rows, x.cols, x.block ? 64 : 0,
                         ptr<uint16_t>(out), stream_of(c));
    return Py_BuildValue("(iN)", st, THPVariable_Wrap(*out));
  });
}

// fwd8(X, W, A | None, B | None, alpha, save_T, out | None, T_out | None, ws | None)
//   -> None or (status, Y, T | None)
PyObject* call_fwd8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9) return PyErr_Format(PyExc_TypeError, "fwd8 takes 9 arguments");
  return guarded([&]() -> PyObject* {
    Checked c;
    Codes X, W;
    if (!X.take(c, a[0]) || !W.take(c, a[1]) || X.block || W.block || X.cols != W.cols) return none();
    const int64_t M = X.rows, K = X.cols, N = W.rows;
    int64_t sa[2] = {0, 0};
    const bool bare = a[2] == Py_None && a[3] == Py_None;
    if (!bare && (!sizes(a[2], 2, sa) || sa[0] < 1 || sa[0] > (1 << 30))) return none();
    const int r = (int)sa[0];
    const at::Tensor* A = bare ? nullptr : c.one(a[2], at::kBFloat16, {r, K});
    const at::Tensor* B = bare ? nullptr : c.one(a[3], at::kBFloat16, {N, r});
    double alpha;
    if (!number(a[4], &alpha)) return nullptr;
    const int save = PyObject_IsTrue(a[5]);
    if (save < 0) return nullptr;
    const at::Tensor* Y = c.opt(a[6], at::kBFloat16, {M, N});
    const at::Tensor* T = c.opt(a[7], at::kFloat, {M, r});
    if (!c.ok || (bare && T)) return none();
    if (!apart({{"out", Y}, {"T_out", T}},
               {{"X", X.codes}, {"X", X.scale}, {"W", W.codes}, {"W", W.scale}, {"A", A}, {"B", B}}, {}))
      return nullptr;
    const c10::DeviceGuard guard(c.device);
    at::Tensor own_Y, own_T, own_ws;
    if (!Y) Y = &(own_Y = fresh(c, at::kBFloat16, {M, N}));
    if (!T && save && !bare) T = &(own_T = fresh(c, at::kFloat, {M, r}));
    size_t bytes;
    void* ws = scratch(c, a[8], g_ws8(M, K, N, r, QLORA_BASE_INT8, 0), own_ws, &bytes);
    if (!c.ok) return none();
    const int st = g_fwd8(ptr<int8_t>(X.codes), ptr<float>(X.scale), M, K, N, ptr<int8_t>(W.codes),
                          ptr<float>(W.scale), ptr<uint16_t>(A), ptr<uint16_t>(B), r, (float)alpha,
                          ptr<uint16_t>(Y), ptr<float>(T), ws, bytes, stream_of(c));
    return Py_BuildValue("(iNN)", st, THPVariable_Wrap(*Y), T ? THPVariable_Wrap(*T) : none());
  });
}

// The base of a backward: (codes, scale), (packed, codes, scales, mean, N, K) or a
// bf16 tensor.
struct Base {
  int kind = -1;
  int64_t N = 0;
  Codes w8;
  const at::Tensor *t[4] = {nullptr, nullptr, nullptr, nullptr};

  bool take(Checked& c, PyObject* o, int64_t K) {
    if (PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 2) {
      kind = QLORA_BASE_INT8;
      if (!w8.take(c, o) || w8.block || w8.cols != K) return false;
      N = w8.rows;
      t[0] = w8.codes; t[1] = w8.scale;
      return true;
    }
    if (PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 6) {
      kind = QLORA_BASE_NF4;
      N = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 4));
      const int64_t k = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 5));
      if (PyErr_Occurred()) {
        PyErr_Clear();
        return false;
      }
      if (k != K || N < 1 || N > (1 << 30) || K > (1 << 30)) return false;
      const int64_t nb = N * K / 64;
      t[0] = c.one(PyTuple_GET_ITEM(o, 0), at::kByte, {N * K / 2});
      t[1] = c.one(PyTuple_GET_ITEM(o, 1), at::kByte, {nb});
      t[2] = c.one(PyTuple_GET_ITEM(o, 2), at::kFloat, {(nb + 255) / 256});
      t[3] = c.one(PyTuple_GET_ITEM(o, 3), at::kFloat, {1});
      return c.ok;
    }
    int64_t s[2];
    if (!sizes(o, 2, s)) return false;
    kind = QLORA_BASE_BF16;
    N = s[0];
    t[0] = c.one(o, at::kBFloat16, {N, K});
    return c.ok;
  }
};

// bwd8(dY, X, base, A, B, alpha, T | None, need_dX, accumulate_into | None, dX_out | None,
//      dA_out | None, dB_out | None, ws | None) -> None or (status, dX | None, dA, dB)
PyObject* call_bwd8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 13) return PyErr_Format(PyExc_TypeError, "bwd8 takes 13 arguments");
  return guarded([&]() -> PyObject* {
    Checked c;
    Codes X;
    Base base;
    int64_t sa[2];
    if (!X.take(c, a[1]) || X.block || !base.take(c, a[2], X.cols) || !sizes(a[3], 2, sa) ||
        sa[0] < 1 || sa[0] > (1 << 30))
      return none();
    const int64_t M = X.rows, K = X.cols, N = base.N;
    const int r = (int)sa[0];
    const at::Tensor* dY = c.one(a[0], at::kBFloat16, {M, N});
    const at::Tensor* A = c.one(a[3], at::kBFloat16, {r, K});
    const at::Tensor* B = c.one(a[4], at::kBFloat16, {N, r});
    double alpha;
    if (!number(a[5], &alpha)) return nullptr;
    const at::Tensor* T = c.opt(a[6], base.kind == QLORA_BASE_INT8 ? at::kFloat : at::kBFloat16, {M, r});
    const int need = PyObject_IsTrue(a[7]);
    if (need < 0) return nullptr;
    const bool add = a[8] != Py_None;
    const at::Tensor* dX = c.opt(add ? a[8] : a[9], at::kBFloat16, {M, K});
    const at::Tensor* dA = c.opt(a[10], at::kFloat, {r, K});
    const at::Tensor* dB = c.opt(a[11], at::kFloat, {N, r});
    if (!c.ok) return none();
    if (!apart({{"dX", dX}, {"dA", dA}, {"dB", dB}},
               {{"dY", dY}, {"X", X.codes}, {"X", X.scale}, {"base weight", base.t[0]},
                {"base weight", base.t[1]}, {"base weight", base.t[2]}, {"base weight", base.t[3]},
                {"A", A}, {"B", B}, {"T", T}}, {}))
      return nullptr;
    const c10::DeviceGuard guard(c.device);
    at::Tensor own_dX, own_dA, own_dB, own_ws;
    if (!dX && need) dX = &(own_dX = fresh(c, at::kBFloat16, {M, K}));
    if (!dA) dA = &(own_dA = fresh(c, at::kFloat, {r, K}));
    if (!dB) dB = &(own_dB = fresh(c, at::kFloat, {N, r}));
    size_t bytes;
    void* ws = scratch(c, a[12], g_ws8(M, K, N, r, base.kind, 1), own_ws, &bytes);
    if (!c.ok) return none();
    const int flags = add ? QLORA_BWD_ACCUMULATE_DX : 0;
    int st;
    if (base.kind == QLORA_BASE_INT8)
      st = g_bwd8(ptr<uint16_t>(dY), ptr<int8_t>(X.codes), ptr<float>(X.scale), M, K, N,
                  ptr<int8_t>(base.t[0]), ptr<float>(base.t[1]), ptr<uint16_t>(A), ptr<uint16_t>(B), r,
                  (float)alpha, ptr<float>(T), ptr<uint16_t>(dX), ptr<float>(dA), ptr<float>(dB), flags,
                  ws, bytes, stream_of(c));
    else if (base.kind == QLORA_BASE_NF4)
      st = g_bwd8_nf4(ptr<uint16_t>(dY), ptr<int8_t>(X.codes), ptr<float>(X.scale), M, K, N,
                      ptr<uint8_t>(base.t[0]), ptr<uint8_t>(base.t[1]), ptr<float>(base.t[2]),
                      ptr<float>(base.t[3]), ptr<uint16_t>(A), ptr<uint16_t>(B), r, (float)alpha,
                      ptr<uint16_t>(T), ptr<uint16_t>(dX), ptr<float>(dA), ptr<float>(dB), flags, ws,
                      bytes, stream_of(c));
    else
      st = g_bwd8_bf16(ptr<uint16_t>(dY), ptr<int8_t>(X.codes), ptr<float>(X.scale), M, K, N,
                       ptr<uint16_t>(base.t[0]), ptr<uint16_t>(A), ptr<uint16_t>(B), r, (float)alpha,
                       ptr<uint16_t>(T), ptr<uint16_t>(dX), ptr<float>(dA), ptr<float>(dB), flags, ws,
                       bytes, stream_of(c));
    return Py_BuildValue("(iNNN)", st, dX ? THPVariable_Wrap(*dX) : none(), THPVariable_Wrap(*dA),
                         THPVariable_Wrap(*dB));
  });
}

// silu8(G, Up, keep, out | None) -> None or (status, Hcodes, Hscale, Gcodes, Gscale, Ucodes,
//                                           Uscale), the last four None unless kept
PyObject* call_silu8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) return PyErr_Format(PyExc_TypeError, "silu8 takes 4 arguments");
  return guarded([&]() -> PyObject* {
    Checked c;
    int64_t s[2];
    if (!sizes(a[0], 2, s)) return none();
    const int64_t M = s[0], I = s[1];
    const at::Tensor* G = c.one(a[0], at::kBFloat16, {M, I});
    const at::Tensor* U = c.one(a[1], at::kBFloat16, {M, I});
    const int keep = PyObject_IsTrue(a[2]);
    if (keep < 0) return nullptr;
    const at::Tensor* H = c.opt(a[3], at::kBFloat16, {M, I});
    if (!c.ok) return none();
    if (!apart({{"out", H}}, {{"G", G}, {"Up", U}}, {})) return nullptr;
    const c10::DeviceGuard guard(c.device);
    at::Tensor t[6];
    for (int i = 0; i < (keep ? 6 : 2); i += 2) {
      t[i] = fresh(c, at::kChar, {M, I});
      t[i + 1] = i ? fresh(c, at::kFloat, {M, I / 64}) : fresh(c, at::kFloat, {M});
    }
    auto at = [&](int i) { return keep || i < 2 ? &t[i] : nullptr; };
    const int st = g_silu8(ptr<uint16_t>(G), ptr<uint16_t>(U), M, I, ptr<uint16_t>(H),
                           ptr<int8_t>(at(0)), ptr<float>(at(1)), ptr<int8_t>(at(2)),
                           ptr<float>(at(3)), ptr<int8_t>(at(4)), ptr<float>(at(5)), stream_of(c));
    auto py = [&](int i) { return at(i) ? THPVariable_Wrap(t[i]) : none(); };
    return Py_BuildValue("(iNNNNNN)", st, py(0), py(1), py(2), py(3), py(4), py(5));
  });
}

// silu8_bwd(dH, G, Up) (blocks) -> None or (status, dG, dUp)
PyObject* call_silu8_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) return PyErr_Format(PyExc_TypeError, "silu8_bwd takes 5 arguments");
  return guarded([&]() -> PyObject* {
    Checked c;
    Codes G, U;
    if (!G.take(c, a[1]) || !U.take(c, a[2]) || !G.block || !U.block || G.rows != U.rows ||
        G.cols != U.cols)
      return none();
    const int64_t M = G.rows, I = G.cols;
    const at::Tensor* dH = c.one(a[0], at::kBFloat16, {M, I});
    const at::Tensor* dG = c.opt(a[3], at::kBFloat16, {M, I});
    const at::Tensor* dU = c.opt(a[4], at::kBFloat16, {M, I});
    if (!c.ok) return none();
    if (!apart({{"dG_out", dG}, {"dUp_out", dU}},
               {{"dH", dH}, {"G", G.codes}, {"G", G.scale}, {"Up", U.codes}, {"Up", U.scale}}, {}))
      return nullptr;
    const c10::DeviceGuard guard(c.device);
    at::Tensor own_G, own_U;
    if (!dG) dG = &(own_G = fresh(c, at::kBFloat16, {M, I}));
    if (!dU) dU = &(own_U = fresh(c, at::kBFloat16, {M, I}));
    const int st = g_silu8_bwd(ptr<uint16_t>(dH), ptr<int8_t>(G.codes), ptr<float>(G.scale),
                               ptr<int8_t>(U.codes), ptr<float>(U.scale), M, I, ptr<uint16_t>(dG),
                               ptr<uint16_t>(dU), stream_of(c));
    return Py_BuildValue("(iNN)", st, THPVariable_Wrap(*dG), THPVariable_Wrap(*dU));
  });
}

// bind8(addresses of the C ABI's ten 8-bit functions, in the order below)
PyObject* call_bind8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10) return PyErr_Format(PyExc_TypeError, "bind8 takes 10 addresses");
  void* p[10];
  for (int i = 0; i < 10; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "null address");
  }
  g_q8 = reinterpret_cast<decltype(g_q8)>(p[0]);
  g_q8_fp32 = reinterpret_cast<decltype(g_q8_fp32)>(p[1]);
  g_dq8 = reinterpret_cast<decltype(g_dq8)>(p[2]);
  g_ws8 = reinterpret_cast<decltype(g_ws8)>(p[3]);
  g_fwd8 = reinterpret_cast<decltype(g_fwd8)>(p[4]);
  g_bwd8 = reinterpret_cast<decltype(g_bwd8)>(p[5]);
  g_bwd8_nf4 = reinterpret_cast<decltype(g_bwd8_nf4)>(p[6]);
  g_bwd8_bf16 = reinterpret_cast<decltype(g_bwd8_bf16)>(p[7]);
  g_silu8 = reinterpret_cast<decltype(g_silu8)>(p[8]);
  g_silu8_bwd = reinterpret_cast<decltype(g_silu8_bwd)>(p[9]);
  return none();
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef kMethods[] = {
    {"bind", fast(call_bind), METH_FASTCALL, nullptr},
    {"plan", fast(call_plan), METH_FASTCALL, nullptr},
    {"fwd", fast(call_fwd), METH_FASTCALL, nullptr},
    {"bwd", fast(call_bwd), METH_FASTCALL, nullptr},
    {"bind8", fast(call_bind8), METH_FASTCALL, nullptr},
    {"quantize8", fast(call_quantize8), METH_FASTCALL, nullptr},
    {"dequant8", fast(call_dequant8), METH_FASTCALL, nullptr},
    {"fwd8", fast(call_fwd8), METH_FASTCALL, nullptr},
    {"bwd8", fast(call_bwd8), METH_FASTCALL, nullptr},
    {"silu8", fast(call_silu8), METH_FASTCALL, nullptr},
    {"silu8_bwd", fast(call_silu8_bwd), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&kModule); }
