// cache_calls.cpp -- the ordinary form of the cache's calls from Python: every
// tensor as the C ABI wants it, on the current device, on the current stream.
//
// A decode step's kernels take 2 to 6 us, and so does a call whose dozen tensors
// are looked at attribute by attribute from Python: a plan took 8.3 us on the
// host, an attention call 7.9, a read 5.8.  Here the same checks are made on the
// tensors themselves.  A function returns the C ABI's status, or None for any
// call that is not ordinary; cache.py then makes the call, or says what is wrong
// with it.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "dsa_select.h"

namespace {

constexpr int64_t kDim = 128;

struct Library {
  decltype(&dsa_cache_bytes) bytes;
  decltype(&dsa_cache_plan) plan;
  decltype(&dsa_cache_write) write;
  decltype(&dsa_cache_read) read;
  decltype(&dsa_cache_attention) attention;
  decltype(&dsa_cache_attention_prompt) prompt;
};
Library lib;
PyObject* cfg_type;  // cache.py's dsa_cache_cfg
bool host_tensors;   // tensors of the host stand in for a device's (the tests' stubs)

// The arguments of one call.
class Call {
 public:
  explicit Call(PyObject* cfg) {
    ok_ = (PyObject*)Py_TYPE(cfg) == cfg_type && PyObject_GetBuffer(cfg, &view_, PyBUF_SIMPLE) == 0;
    held_ = ok_;
    if (!ok_) PyErr_Clear();
    ok_ = ok_ && view_.len == (Py_ssize_t)sizeof(dsa_cache_cfg);
  }
  ~Call() {
    if (held_) PyBuffer_Release(&view_);
  }
  Call(const Call&) = delete;
  Call& operator=(const Call&) = delete;

  explicit operator bool() const { return ok_; }
  const dsa_cache_cfg* cfg() const { return static_cast<const dsa_cache_cfg*>(view_.buf); }

  // A tensor without surprises, on the device of the others.
  const at::Tensor* tensor(PyObject* o) {
    if (!ok_ || !THPVariable_Check(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != at::kStrided || t.unsafeGetTensorImpl()->is_python_dispatch()) return fail();
    if (!host_tensors && !t.is_cuda()) return fail();
    if (host_tensors && !t.is_cpu()) return fail();
    if (!device_known_) {
      device_known_ = true;
      device_ = t.get_device();
    }
    return t.get_device() == device_ ? &t : fail();
  }
  // Its memory: contiguous, of `type`, at least n elements.
  template <typename T>
  T* data(PyObject* o, at::ScalarType type, int64_t n) {
    const at::Tensor* t = tensor(o);
    if (!t || t->scalar_type() != type || t->numel() < n || !t->is_contiguous()) {
      ok_ = false;
      return nullptr;
    }
    return static_cast<T*>(t->data_ptr());
  }
  int32_t* ints(PyObject* o, int64_t n) { return data<int32_t>(o, at::kInt, n); }
  uint8_t* cache(PyObject* o) {
    size_t n = 0;
    if (ok_ && (lib.bytes(cfg(), &n) != DSA_OK || n > (size_t)INT64_MAX)) ok_ = false;
    return data<uint8_t>(o, at::kByte, (int64_t)n);
  }
  // A number of the C ABI's.
  int32_t number(int64_t n) {
    if (n < 0 || n > INT32_MAX) ok_ = false;
    return (int32_t)n;
  }
  float real(PyObject* o) {
    const double x = PyFloat_Check(o) ? PyFloat_AS_DOUBLE(o) : 0.0;
    ok_ = ok_ && PyFloat_Check(o);
    return (float)x;
  }
  // The stream to launch on, when the tensors' device is the current one.
  CUstream_st* stream() {
    if (!ok_ || host_tensors) return nullptr;
    if (c10::cuda::current_device() != device_) {
      ok_ = false;
      return nullptr;
    }
    return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device_).stream();
  }

 private:
  const at::Tensor* fail() {
    ok_ = false;
    return nullptr;
  }
  Py_buffer view_;
  bool ok_ = false, held_ = false, device_known_ = false;
  int64_t device_ = -1;
};

int32_t type_code(at::ScalarType t, int32_t types) {
  const int32_t c = t == at::kBFloat16 ? DSA_BF16 : t == at::kHalf ? DSA_F16 : t == at::kFloat ? DSA_F32 : types;
  return c < types ? c : -1;
}

template <typename F>
PyObject* launch(Call& c, F&& f) {
  if (!c) Py_RETURN_NONE;
  int rc;
  Py_BEGIN_ALLOW_THREADS rc = f();
  Py_END_ALLOW_THREADS return PyLong_FromLong(rc);
}

// Every entry point: no C++ exception leaves it.
template <PyObject* (*kBody)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != kArgs || !lib.bytes) Py_RETURN_NONE;
  try {
    return kBody(a);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

// cfg, lens, fresh, tables, held, free_pages, free_count, first, token_req, ends, slots, status
PyObject* plan(PyObject* const* a) {
  Call c(a[0]);
  const at::Tensor* lens = c.tensor(a[1]);
  const at::Tensor* tables = c.tensor(a[3]);
  const at::Tensor* free = c.tensor(a[5]);
  const at::Tensor* token_req = c.tensor(a[8]);
  if (!c || tables->dim() != 2 || tables->size(0) != lens->numel()) Py_RETURN_NONE;
  const int32_t R = c.number(lens->numel()), P = c.number(tables->size(1)), T = c.number(token_req->numel()),
                cap = c.number(free->numel());
  int32_t* p[11];
  const int64_t need[11] = {R, R, 0, R, 0, 1, (int64_t)R + 1, T, T, T, 4};
  for (int i = 0; i < 11; ++i) p[i] = c.ints(a[1 + i], need[i]);
  CUstream_st* s = c.stream();
  return launch(c, [&] {
    return lib.plan(c.cfg(), R, P, T, cap, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], p[10], s);
  });
}

// The token stride of rows [T, H, 128] whose heads and dims are packed, or -1.
int64_t token_stride(const at::Tensor& t, int64_t T, int64_t H) {
  if (t.dim() != 3 || t.size(0) != T || t.size(1) != H || t.size(2) != kDim) return -1;
  if (T && (t.stride(2) != 1 || (H > 1 && t.stride(1) != kDim))) return -1;
  return T <= 1 ? H * kDim : t.stride(0) < H * kDim ? -1 : t.stride(0);
}

// cfg, k, v, slots, cache
PyObject* write(PyObject* const* a) {
  Call c(a[0]);
  const at::Tensor* k = c.tensor(a[1]);
  const at::Tensor* v = c.tensor(a[2]);
  const at::Tensor* slots = c.tensor(a[3]);
  if (!c) Py_RETURN_NONE;
  const int32_t T = c.number(slots->numel()), code = type_code(k->scalar_type(), 3);
  const int64_t ks = token_stride(*k, T, c.cfg()->kv_heads), vs = token_stride(*v, T, c.cfg()->kv_heads);
  const int32_t* rows = c.ints(a[3], 0);
  uint8_t* cache = c.cache(a[4]);
  CUstream_st* s = c.stream();
  if (code < 0 || v->scalar_type() != k->scalar_type() || ks < 0 || vs < 0 || !c) Py_RETURN_NONE;
  const void *kp = k->data_ptr(), *vp = v->data_ptr();
  return launch(c, [&] { return lib.write(c.cfg(), T, code, kp, vp, ks, vs, rows, cache, s); });
}

// cfg, cache, slots, k, v
PyObject* read(PyObject* const* a) {
  Call c(a[0]);
  const at::Tensor* slots = c.tensor(a[2]);
  const at::Tensor* k = c.tensor(a[3]);
  if (!c) Py_RETURN_NONE;
  const int32_t T = c.number(slots->numel()), code = type_code(k->scalar_type(), 3);
  const uint8_t* cache = c.cache(a[1]);
  if (!c || code < 0) Py_RETURN_NONE;
  const int64_t n = (int64_t)T * c.cfg()->kv_heads * kDim;  // kv_heads <= 64: cache() has checked cfg
  const int32_t* rows = c.ints(a[2], 0);
  void *kp = c.data<void>(a[3], k->scalar_type(), n), *vp = c.data<void>(a[4], k->scalar_type(), n);
  CUstream_st* s = c.stream();
  return launch(c, [&] { return lib.read(c.cfg(), T, code, cache, rows, kp, vp, s); });
}

// What both attention calls take.
struct Attention {
  int32_t code, T, H, Kc;
  const uint8_t* cache;
  const void* q;
  const int32_t* idx;
  void* o;
  float* lse;
};

bool attention_args(Call& c, PyObject* cache, PyObject* q, PyObject* idx, PyObject* o, PyObject* lse, Attention* out) {
  const at::Tensor* tq = c.tensor(q);
  const at::Tensor* ti = c.tensor(idx);
  if (!c || tq->dim() != 3 || tq->size(2) != kDim || ti->dim() != 2 || ti->size(0) != tq->size(0)) return false;
  const at::ScalarType type = tq->scalar_type();
  out->code = type_code(type, 2);
  out->T = c.number(tq->size(0));
  out->H = c.number(tq->size(1));
  out->Kc = c.number(ti->size(1));
  if (!c || out->code < 0) return false;
  const int64_t rows = (int64_t)out->T * out->H;
  if (rows > INT32_MAX) return false;
  out->cache = c.cache(cache);
  out->q = c.data<void>(q, type, 0);
  out->idx = c.ints(idx, 0);
  out->o = c.data<void>(o, type, rows * kDim);
  out->lse = c.data<float>(lse, at::kFloat, rows);
  return (bool)c;
}

// cfg, cache, q, idx, token_req, tables, scale, o, lse
PyObject* attention(PyObject* const* a) {
  Call c(a[0]);
  Attention x;
  if (!attention_args(c, a[1], a[2], a[3], a[7], a[8], &x)) Py_RETURN_NONE;
  const at::Tensor* tables = c.tensor(a[5]);
  if (!c || tables->dim() != 2) Py_RETURN_NONE;
  const int32_t R = c.number(tables->size(0)), P = c.number(tables->size(1));
  const int32_t *req = c.ints(a[4], x.T), *table = c.ints(a[5], 0);
  const float scale = c.real(a[6]);
  CUstream_st* s = c.stream();
  return launch(c, [&] {
    return lib.attention(c.cfg(), x.T, x.H, x.Kc, R, P, x.code, x.cache, x.q, x.idx, req, table, scale, x.o, x.lse, s);
  });
}

// cfg, cache, q, idx, table, scale, workspace, o, lse
PyObject* prompt(PyObject* const* a) {
  Call c(a[0]);
  Attention x;
  if (!attention_args(c, a[1], a[2], a[3], a[7], a[8], &x)) Py_RETURN_NONE;
  const at::Tensor* table = c.tensor(a[4]);
  const at::Tensor* ws = c.tensor(a[6]);
  if (!c) Py_RETURN_NONE;
  const int32_t P = c.number(table->numel());
  const size_t ws_bytes = (size_t)ws->numel();
  const int32_t* pages = c.ints(a[4], 0);
  const float scale = c.real(a[5]);
  uint8_t* w = c.data<uint8_t>(a[6], at::kByte, 0);
  CUstream_st* s = c.stream();
  return launch(c, [&] {
    return lib.prompt(c.cfg(), x.T, x.H, x.Kc, P, x.code, x.cache, x.q, x.idx, pages, scale, w, ws_bytes, x.o, x.lse,
                      s);
  });
}

// bind(cfg type, host tensors, addresses of the six functions in Library's order)
PyObject* bind(PyObject*, PyObject* args) {
  PyObject* type;
  int host;
  unsigned long long p[6];
  if (!PyArg_ParseTuple(args, "OpKKKKKK", &type, &host, &p[0], &p[1], &p[2], &p[3], &p[4], &p[5])) return nullptr;
  Py_INCREF(type);
  Py_XSETREF(cfg_type, type);
  host_tensors = host != 0;
  lib.bytes = reinterpret_cast<decltype(lib.bytes)>((uintptr_t)p[0]);
  lib.plan = reinterpret_cast<decltype(lib.plan)>((uintptr_t)p[1]);
  lib.write = reinterpret_cast<decltype(lib.write)>((uintptr_t)p[2]);
  lib.read = reinterpret_cast<decltype(lib.read)>((uintptr_t)p[3]);
  lib.attention = reinterpret_cast<decltype(lib.attention)>((uintptr_t)p[4]);
  lib.prompt = reinterpret_cast<decltype(lib.prompt)>((uintptr_t)p[5]);
  Py_RETURN_NONE;
}

template <PyObject* (*kBody)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
  const auto f = reinterpret_cast<void (*)()>(entry<kBody, kArgs>);
  return {name, reinterpret_cast<PyCFunction>(f), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    method<plan, 12>("plan"),
    method<write, 5>("write"),
    method<read, 5>("read"),
    method<attention, 9>("attention"),
    method<prompt, 9>("prompt"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "cache_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_cache_calls() { return PyModule_Create(&module); }
