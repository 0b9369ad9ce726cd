// The streaming calls of the Python binding for arguments that are in order.
//
// They are made per layer and token, and their checks, allocations and
// conversions in Python take 5 to 10 us, longer than the kernels of a single
// token (2.6 to 8 us). Here the same checks take under 1 us. A call that finds
// anything out of order (or anything rare: a stream of its own, a subclass, a
// gradient that is asked for), or that the library refuses, returns None, and
// the binding's Python code, which accepts every case and names every fault,
// makes it again.
//
// Measured: one token's rotation 10.8 -> 6.0 us a call, its cache write 8.9 ->
// 4.1, its attention over 333 tokens 13.8 -> 10.2 (of which 8.2 were the kernel's).
#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <exception>

#include "calibatt.h"

namespace {

decltype(&calibatt_rope_fwd) rope_fwd;
decltype(&calibatt_rope_bwd) rope_bwd;
decltype(&calibatt_cache_write) write_fn;
decltype(&calibatt_cache_attn_fwd) attn_fn;
decltype(&calibatt_cache_attn_workspace_size) attn_ws;  // all or none: see bind

constexpr int64_t kPage = 128;

struct NotPlain {};  // left to the Python code
void want(bool ok) {
  if (!ok) throw NotPlain();
}

const at::Tensor& tensor(PyObject* o) {
  want(THPVariable_CheckExact(o));
  const at::Tensor& t = THPVariable_Unpack(o);
  want(t.is_cuda() && t.layout() == at::kStrided);
  return t;
}

// A contiguous tensor of this type on the device.
const at::Tensor& plain(PyObject* o, at::ScalarType type, c10::DeviceIndex device) {
  const at::Tensor& t = tensor(o);
  want(t.scalar_type() == type && t.get_device() == device && t.is_contiguous());
  return t;
}

// bf16 with three dimensions and 128 contiguous channels.
const at::Tensor& rows(PyObject* o, c10::DeviceIndex device) {
  const at::Tensor& t = tensor(o);
  want(t.scalar_type() == at::kBFloat16 && t.get_device() == device && t.dim() == 3 &&
       t.size(2) == CALIBATT_HEAD_DIM && t.stride(2) == 1);
  return t;
}

bool asks_gradient(const at::Tensor& t) { return t.requires_grad() && at::GradMode::is_enabled(); }

int small(int64_t x) {
  want(x >= INT_MIN && x <= INT_MAX);
  return static_cast<int>(x);
}

int number(PyObject* o) {
  want(PyLong_CheckExact(o));
  int over = 0;
  const long long x = PyLong_AsLongLongAndOverflow(o, &over);
  want(over == 0);
  return small(x);
}

template <typename T>
T* data(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, c10::DeviceIndex device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, device)));
}

calibatt_stream_t stream_of(c10::DeviceIndex device) { return c10::cuda::getCurrentCUDAStream(device).stream(); }

// A C call without the interpreter's lock.
template <typename F>
bool ok(F&& call) {
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = call();
  Py_END_ALLOW_THREADS;
  return rc == CALIBATT_OK;
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t need, F&& body) {
  try {
    want(n == need && attn_fn != nullptr);
    return body();
  } catch (const NotPlain&) {
  } catch (const std::exception&) {  // what the Python code meets too, and reports
  }
  if (PyErr_Occurred()) PyErr_Clear();
  Py_RETURN_NONE;
}

struct Cache {
  const at::Tensor &k8, &v8, &ks, &vs, &start, &len, &table;
  int pages, heads, batch, width;
};

// k8, v8, k_scale, v_scale, tok_start, kv_len, table
Cache cache(PyObject* const* a, c10::DeviceIndex device) {
  const auto pool = [&](PyObject* o) -> const at::Tensor& {
    const at::Tensor& t = tensor(o);
    want((t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte) && t.get_device() == device &&
         t.is_contiguous());
    return t;
  };
  const Cache c{pool(a[0]),
                pool(a[1]),
                plain(a[2], at::kFloat, device),
                plain(a[3], at::kFloat, device),
                plain(a[4], at::kInt, device),
                plain(a[5], at::kInt, device),
                plain(a[6], at::kInt, device),
                0, 0, 0, 0};
  want(c.k8.dim() == 4 && c.k8.size(2) == kPage && c.k8.size(3) == CALIBATT_HEAD_DIM && c.v8.sizes() == c.k8.sizes());
  want(c.ks.sizes() == c.k8.sizes().slice(0, 2) && c.vs.sizes() == c.ks.sizes());
  want(c.table.dim() == 2 && c.table.size(0) == c.len.numel() && c.start.numel() == c.len.numel() + 1);
  return {c.k8, c.v8, c.ks, c.vs, c.start, c.len, c.table,
          small(c.k8.size(0)), small(c.k8.size(1)), small(c.len.numel()), small(c.table.size(1))};
}

// forward, q, k, plan's address, grid, start, pos, q_out, k_out -> (q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t argc) {
  return guarded(argc, 9, [&]() -> PyObject* {
    const bool forward = a[0] == Py_True;
    const int tok = forward ? 0 : 1, hd = 1 - tok;
    const c10::DeviceIndex device = c10::cuda::current_device();
    const at::Tensor& q = rows(a[1], device);
    want(!asks_gradient(q));
    const int64_t n = q.size(tok);
    const auto place = [&](PyObject* given, int64_t heads) {
      const int64_t shape[3] = {forward ? heads : n, forward ? n : heads, CALIBATT_HEAD_DIM};
      if (given == Py_None) return fresh(shape, at::kBFloat16, device);
      const at::Tensor& t = rows(given, device);
      want(t.size(0) == shape[0] && t.size(1) == shape[1]);
      return t;
    };
    at::Tensor qo = place(a[7], q.size(hd)), ko;
    const at::Tensor* k = nullptr;
    if (a[2] != Py_None) {
      k = &rows(a[2], device);
      want(k->size(tok) == n && !asks_gradient(*k));
      ko = place(a[8], k->size(hd));
    } else {
      want(a[8] == Py_None);
    }
    int H = 0, W = 0;
    const int32_t* pos = nullptr;
    if (a[6] == Py_None) {
      want(PyTuple_CheckExact(a[4]) && PyTuple_GET_SIZE(a[4]) == 2);
      H = number(PyTuple_GET_ITEM(a[4], 0));
      W = number(PyTuple_GET_ITEM(a[4], 1));
    } else {
      const at::Tensor& t = plain(a[6], at::kInt, device);
      want(a[4] == Py_None && t.dim() == 2 && t.size(0) == n && t.size(1) == 3);
      pos = data<const int32_t>(t);
    }
    want(PyTuple_CheckExact(a[5]) && PyTuple_GET_SIZE(a[5]) == 3);
    int32_t start[3];
    for (int i = 0; i < 3; ++i) start[i] = number(PyTuple_GET_ITEM(a[5], i));
    const auto* plan = static_cast<const calibatt_rope_plan*>(PyLong_AsVoidPtr(a[3]));
    want(plan != nullptr);
    const auto fn = forward ? rope_fwd : rope_bwd;
    const auto* qp = data<const calibatt_bf16>(q);
    const auto* kp = k ? data<const calibatt_bf16>(*k) : nullptr;
    auto* qop = data<calibatt_bf16>(qo);
    auto* kop = k ? data<calibatt_bf16>(ko) : nullptr;
    const int heads = small(q.size(hd)), heads_k = k ? small(k->size(hd)) : 0;
    const auto stream = stream_of(device);
    want(ok([&] {
      return fn(plan, qp, q.stride(tok), q.stride(hd), heads, kp, k ? k->stride(tok) : 0, k ? k->stride(hd) : 0, heads_k,
                n, CALIBATT_HEAD_DIM, pos, H, W, start, qop, qo.stride(hd), qo.stride(tok), kop, k ? ko.stride(hd) : 0,
                k ? ko.stride(tok) : 0, stream);
    }));
    PyObject* first = THPVariable_Wrap(std::move(qo));
    PyObject* second = Py_NewRef(Py_None);
    if (k) {
      Py_DECREF(second);
      second = THPVariable_Wrap(std::move(ko));
    }
    PyObject* both = PyTuple_New(2);
    PyTuple_SET_ITEM(both, 0, first);
    PyTuple_SET_ITEM(both, 1, second);
    return both;
  });
}

// k, v, the cache's seven, max_new -> True
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t argc) {
  return guarded(argc, 10, [&]() -> PyObject* {
    const c10::DeviceIndex device = c10::cuda::current_device();
    const at::Tensor &k = rows(a[0], device), &v = rows(a[1], device);
    want(k.sizes() == v.sizes());
    const Cache c = cache(a + 2, device);
    const int n = small(k.size(0)), heads = small(k.size(1));
    want(heads == c.heads);
    const int max_new = a[9] == Py_None ? n : number(a[9]);
    const auto *kp = data<const calibatt_bf16>(k), *vp = data<const calibatt_bf16>(v);
    const auto *start = data<const int32_t>(c.start), *len = data<const int32_t>(c.len),
               *table = data<const int32_t>(c.table);
    auto *k8 = data<uint8_t>(c.k8), *v8 = data<uint8_t>(c.v8);
    auto *ks = data<float>(c.ks), *vs = data<float>(c.vs);
    const auto stream = stream_of(device);
    want(ok([&] {
      return write_fn(kp, k.stride(0), k.stride(1), vp, v.stride(0), v.stride(1), heads, n, CALIBATT_HEAD_DIM, start, len,
                      c.batch, max_new, table, c.width, c.pages, k8, v8, ks, vs, stream);
    }));
    Py_RETURN_TRUE;
  });
}

// q, the cache's seven, max_new, max_kv, causal_unit, o, lse, ws, scale, want_lse -> (o, lse)
PyObject* cache_attn(PyObject*, PyObject* const* a, Py_ssize_t argc) {
  return guarded(argc, 16, [&]() -> PyObject* {
    const c10::DeviceIndex device = c10::cuda::current_device();
    const at::Tensor& q = plain(a[0], at::kBFloat16, device);
    want(q.dim() == 3 && q.size(2) == CALIBATT_HEAD_DIM);
    const int heads = small(q.size(0)), n = small(q.size(1));
    const Cache c = cache(a + 1, device);
    const int max_new = a[8] == Py_None ? n : number(a[8]);
    const int max_kv = a[9] == Py_None ? static_cast<int>(std::min<int64_t>(c.width * kPage, INT_MAX)) : number(a[9]);
    const int unit = number(a[10]);
    float scale = 1.f / std::sqrt(static_cast<float>(CALIBATT_HEAD_DIM));
    if (a[14] != Py_None) {
      want(PyFloat_CheckExact(a[14]));
      scale = static_cast<float>(PyFloat_AS_DOUBLE(a[14]));
    }
    at::Tensor o, lse, ws;
    if (a[11] == Py_None) {
      o = fresh(q.sizes(), at::kBFloat16, device);
    } else {
      o = plain(a[11], at::kBFloat16, device);
      want(o.sizes() == q.sizes());
    }
    if (a[12] != Py_None) {
      lse = plain(a[12], at::kFloat, device);
      want(lse.dim() == 2 && lse.size(0) == heads && lse.size(1) == n);
    } else if (a[15] == Py_True) {
      lse = fresh({heads, n}, at::kFloat, device);
    }
    size_t bytes = 0;
    if (a[13] != Py_None) {
      ws = plain(a[13], at::kByte, device);
      bytes = static_cast<size_t>(ws.numel());
    } else {
      bytes = attn_ws(c.batch, heads, c.heads, n, max_new, max_kv);
      if (bytes > 0) ws = fresh({static_cast<int64_t>(bytes)}, at::kByte, device);
    }
    const auto* qp = data<const calibatt_bf16>(q);
    const auto *start = data<const int32_t>(c.start), *len = data<const int32_t>(c.len),
               *table = data<const int32_t>(c.table);
    const auto *k8 = data<const uint8_t>(c.k8), *v8 = data<const uint8_t>(c.v8);
    const auto *ks = data<const float>(c.ks), *vs = data<const float>(c.vs);
    auto* op = data<calibatt_bf16>(o);
    auto* lp = lse.defined() ? data<float>(lse) : nullptr;
    void* wp = ws.defined() ? ws.data_ptr() : nullptr;
    const auto stream = stream_of(device);
    want(ok([&] {
      return attn_fn(qp, heads, c.heads, n, CALIBATT_HEAD_DIM, scale, unit, start, len, c.batch, max_new, max_kv, table,
                     c.width, c.pages, k8, v8, ks, vs, op, lp, wp, bytes, stream);
    }));
    PyObject* second = lse.defined() ? THPVariable_Wrap(std::move(lse)) : Py_NewRef(Py_None);
    PyObject* both = PyTuple_New(2);
    PyTuple_SET_ITEM(both, 0, THPVariable_Wrap(std::move(o)));
    PyTuple_SET_ITEM(both, 1, second);
    return both;
  });
}

// The addresses of the loaded library's functions, in the order of the
// variables above, then of calibatt_version. A library of another version may
// want other arguments: False, and every call is left to the Python code.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* at[6] = {};
  for (Py_ssize_t i = 0; i < n && i < 6; ++i) at[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  const auto version = reinterpret_cast<decltype(&calibatt_version)>(at[5]);
  const bool fits = version != nullptr && version() == CALIBATT_VERSION;
  if (!fits)
    for (void*& x : at) x = nullptr;
  rope_fwd = reinterpret_cast<decltype(rope_fwd)>(at[0]);
  rope_bwd = reinterpret_cast<decltype(rope_bwd)>(at[1]);
  write_fn = reinterpret_cast<decltype(write_fn)>(at[2]);
  attn_fn = reinterpret_cast<decltype(attn_fn)>(at[3]);
  attn_ws = reinterpret_cast<decltype(attn_ws)>(at[4]);
  return PyBool_FromLong(fits);
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name, const char* doc) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, doc};
}

PyMethodDef methods[] = {method<rope>("rope", "calibatt_rope_fwd or _bwd, or None"),
                         method<cache_write>("cache_write", "calibatt_cache_write, or None"),
                         method<cache_attn>("cache_attn", "calibatt_cache_attn_fwd, or None"),
                         method<bind>("bind", "addresses of the library's functions; whether they fit"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycalls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pycalls() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch", CALIBATT_TORCH) != 0) Py_CLEAR(m);  // what it was built against
  return m;
}
