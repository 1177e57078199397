// The Python side of the batched adapters' calls in C++: these calls are a few
// kernel launches on tensors that take microseconds, and a dozen tensors
// checked, allocated and passed one by one from Python took longer than the
// kernels (a single-token forward: 14 of 20 us).  Argument marshalling only;
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

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef kMethods[] = {
    {"bind", fast(call_bind), METH_FASTCALL, nullptr},
    {"plan", fast(call_plan), METH_FASTCALL, nullptr},
    {"fwd", fast(call_fwd), METH_FASTCALL, nullptr},
    {"bwd", fast(call_bwd), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&kModule); }
