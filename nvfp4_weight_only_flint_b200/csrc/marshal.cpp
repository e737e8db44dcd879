// marshal.cpp -- Python marshalling of the serving calls that run once per
// layer and step (append to the paged cache, paged attention, sampling): each
// function takes the positional arguments of its namesake in __init__.py,
// turns tensors into device pointers and calls the C entry point of
// libflint_moe.so on the current stream.
//
// Why not ctypes, as for the other calls: a decode step's kernels of these
// calls take 4 to 10 us, and 20 to 27 arguments with their checks through
// ctypes cost the host 20 us a call.
//
// Every tensor is checked for what a kernel would read wrongly: it has to be a
// contiguous CUDA tensor on the current device (whose stream the call takes)
// of the element type the call takes and of at least the bytes it reads or
// writes. A plain int passes as a device address, but for the workspace, whose
// size only a tensor tells.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdio>
#include <exception>

#include "flint_moe.h"

namespace {

PyObject* g_error = nullptr;  // FlintError

void raise(int code, const char* msg) {
  PyObject* a = Py_BuildValue("(is)", code, msg);
  if (a != nullptr) {
    PyErr_SetObject(g_error != nullptr ? g_error : PyExc_RuntimeError, a);
    Py_DECREF(a);
  }
}

// Element types. 16-bit and 8-bit integers pass as the bits of bf16 and E4M3.
enum class Kind { kAny, kI32, kF32, kBf16, kE4M3 };

bool is_kind(at::ScalarType t, Kind k) {
  switch (k) {
    case Kind::kAny: return true;
    case Kind::kI32: return t == at::kInt;
    case Kind::kF32: return t == at::kFloat;
    case Kind::kBf16: return t == at::kBFloat16 || t == at::kShort || t == at::kUInt16;
    case Kind::kE4M3: return t == at::kFloat8_e4m3fn || t == at::kByte || t == at::kChar;
  }
  return false;
}
const char* kind_name(Kind k) {
  return k == Kind::kI32 ? "int32" : k == Kind::kF32 ? "float32" : k == Kind::kBf16 ? "bfloat16" : "float8_e4m3fn";
}
Kind cache_kind(int32_t dtype) {
  return dtype == FLINT_KV_BF16 ? Kind::kBf16 : dtype == FLINT_KV_E4M3 ? Kind::kE4M3 : Kind::kAny;
}
Kind logits_kind(int32_t dtype) {
  return dtype == FLINT_LOGITS_F32 ? Kind::kF32 : dtype == FLINT_LOGITS_BF16 ? Kind::kBf16 : Kind::kAny;
}

struct Args {
  PyObject* const* v;
  int device;
  bool bad = false;

  int64_t i(int k) {
    if (bad) return 0;
    const long long x = PyLong_AsLongLong(v[k]);
    if (x == -1 && PyErr_Occurred()) bad = true;
    return x;
  }
  // an int32 argument of the C call; one that does not fit is refused
  int32_t i32(int k) {
    const int64_t x = i(k);
    if (!bad && x != static_cast<int32_t>(x)) {
      bad = true;
      raise(FLINT_ERR_INVALID_ARG, "an integer argument does not fit 32 bits");
    }
    return static_cast<int32_t>(x);
  }
  double f(int k) {
    if (bad) return 0.0;
    const double x = PyFloat_AsDouble(v[k]);
    if (x == -1.0 && PyErr_Occurred()) bad = true;
    return x;
  }
  int32_t truth(int k) {
    if (bad) return 0;
    const int t = PyObject_IsTrue(v[k]);
    if (t < 0) bad = true;
    return t > 0;
  }
  // device address of argument k, which the call takes `need` bytes of
  void* p(int k, const char* name, Kind kind, int64_t need, int64_t* bytes = nullptr) {
    if (bad || v[k] == Py_None) return nullptr;
    if (PyLong_Check(v[k]) && !PyBool_Check(v[k])) {
      void* a = PyLong_AsVoidPtr(v[k]);
      if (PyErr_Occurred()) bad = true;
      return a;
    }
    char msg[160];
    if (!THPVariable_Check(v[k])) {
      std::snprintf(msg, sizeof msg, "%s: expected a CUDA tensor", name);
    } else {
      const at::Tensor& t = THPVariable_Unpack(v[k]);
      const int64_t have = static_cast<int64_t>(t.nbytes());
      if (!is_kind(t.scalar_type(), kind)) {
        std::snprintf(msg, sizeof msg, "%s: element type %s, %s expected", name, c10::toString(t.scalar_type()),
                      kind_name(kind));
      } else if (!t.is_contiguous()) {
        std::snprintf(msg, sizeof msg, "%s: not contiguous", name);
      } else if (have < need) {
        std::snprintf(msg, sizeof msg, "%s: %lld bytes, %lld needed", name, static_cast<long long>(have),
                      static_cast<long long>(need));
      } else if (!t.is_cuda()) {
        std::snprintf(msg, sizeof msg, "%s: expected a CUDA tensor", name);
      } else if (t.get_device() != device) {
        std::snprintf(msg, sizeof msg, "%s: on device %d, the current one is %d", name,
                      static_cast<int>(t.get_device()), device);
      } else {
        if (bytes != nullptr) *bytes = have;
        return t.data_ptr();
      }
    }
    bad = true;
    raise(FLINT_ERR_INVALID_ARG, msg);
    return nullptr;
  }
  void* stream(int k) {
    if (bad) return nullptr;
    if (v[k] == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    if (PyLong_Check(v[k])) return PyLong_AsVoidPtr(v[k]);
    PyObject* s = PyObject_GetAttrString(v[k], "cuda_stream");
    if (s == nullptr) {
      bad = true;
      return nullptr;
    }
    void* a = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (PyErr_Occurred()) bad = true;
    return a;
  }
};

// The current device, or -1 on a machine without one (then every tensor is refused).
int device_now() {
  try {
    return static_cast<int>(c10::cuda::current_device());
  } catch (...) {
    return -1;
  }
}

// Makes the C call without the interpreter lock: a launch waits where the stream's queue is full, and other threads (a
// host function that the stream waits for, even) go on meanwhile. The caller holds the tensors.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F>
PyObject* launch(F call) {
  int rc;
  {
    const Unlocked u;
    rc = call();
  }
  if (rc != FLINT_OK) {
    raise(rc, flint_last_error());
    return nullptr;
  }
  Py_RETURN_NONE;
}

// Torch's checks throw (a sparse tensor has no strides, say); nothing may leave a C function.
template <PyObject* (*kCall)(PyObject* const*)>
PyObject* guarded(PyObject*, PyObject* const* v, Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return kCall(v);
  } catch (const std::exception& e) {
    raise(FLINT_ERR_INVALID_ARG, e.what());
  } catch (...) {
    raise(FLINT_ERR_INVALID_ARG, "unknown exception");
  }
  return nullptr;
}

// a * b and a + b of sizes, INT64_MAX where they do not fit (no tensor has as many bytes); factors below 1 are left to
// the C call's checks
int64_t mul(int64_t a, int64_t b) {
  if (a <= 0 || b <= 0) return 0;
  int64_t r;
  return __builtin_mul_overflow(a, b, &r) ? INT64_MAX : r;
}

int64_t add(int64_t a, int64_t b) {
  int64_t r;
  return __builtin_add_overflow(a, b, &r) ? INT64_MAX : r;
}

// qkv T Hq Hkv qw kw cos_sin max_pos rope eps | q_start kv_len B table max_pages page n_pages dtype ks vs | q_out k v
// status head_dim stream
PyObject* paged_kv_call(PyObject* const* v) {
  Args a{v, device_now()};
  const int32_t T = a.i32(1), hq = a.i32(2), hkv = a.i32(3), max_pos = a.i32(7), rope = a.truth(8), B = a.i32(12),
                mp = a.i32(14), ps = a.i32(15), dt = a.i32(17), dh = a.i32(24);
  const int64_t np = a.i(16), row = mul(2 * static_cast<int64_t>(T), dh);
  const float eps = static_cast<float>(a.f(9));
  const bool live = T > 0 && B > 0;
  const int64_t pool = mul(mul(mul(np, ps), mul(hkv, dh)), dt == FLINT_KV_E4M3 ? 1 : 2);
  const int64_t sc = dt == FLINT_KV_E4M3 ? 4 * static_cast<int64_t>(hkv) : 0;
  const Kind sk = dt == FLINT_KV_E4M3 ? Kind::kF32 : Kind::kAny;  // ignored for a bf16 cache
  auto qkv = static_cast<const uint16_t*>(a.p(0, "qkv", Kind::kBf16, mul(row, hq + 2 * static_cast<int64_t>(hkv))));
  auto qw = static_cast<const uint16_t*>(a.p(4, "q_norm_w", Kind::kBf16, 2 * static_cast<int64_t>(dh)));
  auto kw = static_cast<const uint16_t*>(a.p(5, "k_norm_w", Kind::kBf16, 2 * static_cast<int64_t>(dh)));
  auto cs = static_cast<const float*>(
      a.p(6, "cos_sin", Kind::kF32, rope ? mul(4 * static_cast<int64_t>(dh), max_pos) : 0));
  auto qs = static_cast<const int32_t*>(a.p(10, "q_start", Kind::kI32, live ? 4 * (static_cast<int64_t>(B) + 1) : 0));
  auto kl = static_cast<const int32_t*>(a.p(11, "kv_len", Kind::kI32, live ? 4 * static_cast<int64_t>(B) : 0));
  auto bt = static_cast<const int32_t*>(
      a.p(13, "block_table", Kind::kI32, live ? mul(4 * static_cast<int64_t>(B), mp) : 0));
  auto ks = static_cast<const float*>(a.p(18, "k_scale", sk, sc));
  auto vs = static_cast<const float*>(a.p(19, "v_scale", sk, sc));
  auto q_out = static_cast<uint16_t*>(a.p(20, "q_out", Kind::kBf16, mul(row, hq)));
  void* k = a.p(21, "k_cache", cache_kind(dt), pool);
  void* vv = a.p(22, "v_cache", cache_kind(dt), pool);
  auto st = static_cast<int32_t*>(a.p(23, "status", Kind::kI32, 4));
  void* stream = a.stream(25);
  if (a.bad) return nullptr;
  return launch([&] {
    return flint_qk_norm_rope_paged_kv(qkv, T, hq, hkv, dh, qw, kw, cs, max_pos, rope, eps, qs, kl, B, bt, mp, ps, np,
                                       dt, ks, vs, q_out, k, vv, st, stream);
  });
}

// q T | q_start kv_len B table max_pages page n_pages | k v dtype ks vs | Hq Hkv max_q window scale out ws status
// head_dim stream
PyObject* paged_attention_call(PyObject* const* v) {
  Args a{v, device_now()};
  const int32_t T = a.i32(1), B = a.i32(4), mp = a.i32(6), ps = a.i32(7), dt = a.i32(11), hq = a.i32(14),
                hkv = a.i32(15), max_q = a.i32(16), window = a.i32(17), dh = a.i32(22);
  const int64_t np = a.i(8), row = mul(mul(2 * static_cast<int64_t>(T), dh), hq);
  const float scale = static_cast<float>(a.f(18));
  const bool live = T > 0 && B > 0;
  const int64_t pool = mul(mul(mul(np, ps), mul(hkv, dh)), dt == FLINT_KV_E4M3 ? 1 : 2);
  const int64_t sc = dt == FLINT_KV_E4M3 ? 4 * static_cast<int64_t>(hkv) : 0;
  const Kind sk = dt == FLINT_KV_E4M3 ? Kind::kF32 : Kind::kAny;  // ignored for a bf16 cache
  int64_t ws_bytes = 0;
  auto q = static_cast<const uint16_t*>(a.p(0, "q", Kind::kBf16, row));
  auto qs = static_cast<const int32_t*>(a.p(2, "q_start", Kind::kI32, live ? 4 * (static_cast<int64_t>(B) + 1) : 0));
  auto kl = static_cast<const int32_t*>(a.p(3, "kv_len", Kind::kI32, live ? 4 * static_cast<int64_t>(B) : 0));
  auto bt = static_cast<const int32_t*>(
      a.p(5, "block_table", Kind::kI32, live ? mul(4 * static_cast<int64_t>(B), mp) : 0));
  void* k = a.p(9, "k_cache", cache_kind(dt), pool);
  void* vv = a.p(10, "v_cache", cache_kind(dt), pool);
  auto ks = static_cast<const float*>(a.p(12, "k_scale", sk, sc));
  auto vs = static_cast<const float*>(a.p(13, "v_scale", sk, sc));
  auto out = static_cast<uint16_t*>(a.p(19, "out", Kind::kBf16, row));
  void* ws = a.p(20, "workspace", Kind::kAny, 0, &ws_bytes);
  auto st = static_cast<int32_t*>(a.p(21, "status", Kind::kI32, 4));
  void* stream = a.stream(23);
  if (!a.bad && PyLong_Check(v[20])) {
    a.bad = true;
    raise(FLINT_ERR_INVALID_ARG, "workspace: a tensor, for its size; the C call takes an address with its bytes");
  }
  if (a.bad) return nullptr;
  return launch([&] {
    return flint_paged_attention(q, T, qs, kl, B, bt, mp, ps, np, k, vv, dt, ks, vs, hq, hkv, dh, max_q, window,
                                 scale, out, ws, static_cast<size_t>(ws_bytes), st, stream);
  });
}

// logits rows vocab row_stride dtype temperature top_k top_p min_p u tokens logprobs status stream
PyObject* sample_call(PyObject* const* v) {
  Args a{v, device_now()};
  const int32_t rows = a.i32(1), vocab = a.i32(2), dt = a.i32(4);
  const int64_t stride = a.i(3), per_row = rows > 0 ? 4 * static_cast<int64_t>(rows) : 0;
  const int64_t elems = rows > 0 ? add(mul(rows - 1, stride), vocab > 0 ? vocab : 0) : 0;
  const void* x = a.p(0, "logits", logits_kind(dt), mul(elems, dt == FLINT_LOGITS_F32 ? 4 : 2));
  auto t = static_cast<const float*>(a.p(5, "temperature", Kind::kF32, per_row));
  auto k = static_cast<const int32_t*>(a.p(6, "top_k", Kind::kI32, per_row));
  auto p = static_cast<const float*>(a.p(7, "top_p", Kind::kF32, per_row));
  auto m = static_cast<const float*>(a.p(8, "min_p", Kind::kF32, per_row));
  auto u = static_cast<const float*>(a.p(9, "u", Kind::kF32, per_row));
  auto tok = static_cast<int32_t*>(a.p(10, "tokens", Kind::kI32, per_row));
  auto lp = static_cast<float*>(a.p(11, "logprobs", Kind::kF32, per_row));
  auto st = static_cast<int32_t*>(a.p(12, "status", Kind::kI32, 4));
  void* stream = a.stream(13);
  if (a.bad) return nullptr;
  return launch([&] {
    return flint_sample(x, rows, vocab, stride, dt, t, k, p, m, u, tok, lp, st, stream);
  });
}

PyObject* paged_kv(PyObject* m, PyObject* const* v, Py_ssize_t n) { return guarded<paged_kv_call>(m, v, n, 26); }
PyObject* paged_attention(PyObject* m, PyObject* const* v, Py_ssize_t n) {
  return guarded<paged_attention_call>(m, v, n, 24);
}
PyObject* sample(PyObject* m, PyObject* const* v, Py_ssize_t n) { return guarded<sample_call>(m, v, n, 14); }

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XDECREF(g_error);
  g_error = Py_NewRef(cls);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"paged_kv", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_kv)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_attention)), METH_FASTCALL,
     nullptr},
    {"sample", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(sample)), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
