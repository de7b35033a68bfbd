// hca_py.cpp -- the serving calls of hca.py without its Python
//
// A decode step's kernels take 6 to 25 us; checking a dozen tensors, allocating
// three and passing thirty arguments takes Python 18 to 22 us a call.  Here the
// same takes 2, and 2 more for each tensor that is made; a workspace that nobody
// asks for is not made a tensor.  A function takes hca.py's arguments and answers
//   a tuple   the call was made: the results and the workspace (None: its own)
//   an int    the C function's status, not HCA_OK
//   None      something is not as in an ordinary call (a tensor that does not
//             fit, a subclass, another device than the current one, no memory):
//             nothing was done, and hca.py's own code says what is wrong or does it
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>
#include <memory>

#include "../../include/hca.h"

namespace {

struct {
  decltype(&hca_cache_plan_workspace_size) plan_ws;
  decltype(&hca_cache_plan) plan;
  decltype(&hca_cache_append_workspace_size) append_ws;
  decltype(&hca_cache_append) append;
  decltype(&hca_cache_attn_workspace_size) attn_ws;
  decltype(&hca_cache_attn) attn;
} lib;

constexpr at::ScalarType kI32 = at::kInt, kF32 = at::kFloat, kU8 = at::kByte, kE4m3 = at::kFloat8_e4m3fn;

struct Declined {};

void need(bool ok) {
  if (!ok) throw Declined();
}

const at::Tensor &tensor(PyObject *o) {
  need(THPVariable_CheckExact(o));
  return THPVariable_Unpack(o);
}

int integer(PyObject *o) {
  need(PyLong_CheckExact(o));
  int overflow;
  const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
  need(!overflow && v >= INT_MIN && v <= INT_MAX);
  return (int)v;
}

struct Call {
  c10::DeviceIndex dev;

  explicit Call(const at::Tensor &t) {
    need(t.is_cuda());
    dev = t.get_device();
    need(dev == c10::cuda::current_device());
  }
  void *stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
  void *fits(const at::Tensor &t, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    need(t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.sizes() == at::IntArrayRef(shape) && t.is_contiguous());
    return t.data_ptr();
  }
  void *fits(PyObject *o, at::ScalarType type, std::initializer_list<int64_t> shape) const { return fits(tensor(o), type, shape); }
  // the caller's tensor, or a new one
  at::Tensor result(PyObject *o, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    if (o != Py_None) {
      const at::Tensor &t = tensor(o);
      fits(t, type, shape);
      return t;
    }
    return at::empty(at::IntArrayRef(shape), at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, dev)));
  }
};

// The caller's workspace (any bytes: what there is of them is for the C function
// to check), a tensor if its status will be looked at, or plain memory that goes
// back to the allocator behind the launch, in the order of the stream.
struct Workspace {
  at::Tensor tensor_;
  c10::DataPtr own;
  void *ptr;
  size_t bytes;

  Workspace(const Call &c, PyObject *o, bool keep, size_t need_bytes) : bytes(need_bytes) {
    if (o != Py_None) {
      tensor_ = tensor(o);
      need(tensor_.is_cuda() && tensor_.get_device() == c.dev && tensor_.scalar_type() == kU8 && tensor_.is_contiguous());
      bytes = tensor_.numel();
    } else if (keep) {
      tensor_ = at::empty({(int64_t)bytes}, at::TensorOptions().dtype(kU8).device(at::Device(at::kCUDA, c.dev)));
    } else {
      own = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
    }
    ptr = tensor_.defined() ? tensor_.data_ptr() : own.get();
  }
};

int dtype_code(at::ScalarType t) {
  need(t == at::kBFloat16 || t == at::kFloat);
  return t == at::kFloat ? HCA_F32 : HCA_BF16;
}

struct Release {
  void operator()(PyObject *o) const { Py_DECREF(o); }
};
using Tuple = std::unique_ptr<PyObject, Release>;

// The answer is made in front of the launch, so that nothing is left to fail behind
// it: a call that has been made is never answered as one that has not.
template <typename... T>
Tuple results(const T &...t) {
  Tuple r(PyTuple_New(sizeof...(t)));
  need(r != nullptr);
  Py_ssize_t i = 0;
  ([&](const at::Tensor &x) {
    PyObject *o = THPVariable_Wrap(x);  // None for an undefined one
    need(o);
    PyTuple_SET_ITEM(r.get(), i++, o);
  }(t), ...);
  return r;
}

PyObject *answer(int rc, Tuple &r) { return rc ? PyLong_FromLong(rc) : r.release(); }

template <typename F>
PyObject *guarded(F f) {
  try {
    return f();
  } catch (...) {  // Declined, or torch's: hca.py meets it again and reports it
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

// held, added, table, free_blocks, free_count, nblocks, bs, nslots, m, start, slots, free_left, ws, check
PyObject *cache_plan(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    need(n == 14);
    const at::Tensor &held = tensor(a[0]), &table = tensor(a[2]), &free_blocks = tensor(a[3]);
    need(held.dim() == 1 && table.dim() == 2 && free_blocks.dim() == 1);
    const int64_t R = table.size(0), cols = table.size(1), nfree = free_blocks.size(0);
    const int nblocks = integer(a[5]), bs = integer(a[6]), nslots = integer(a[7]), m = integer(a[8]);
    need(R < INT_MAX && cols <= INT_MAX && nfree <= INT_MAX && nslots >= 0);
    const Call c(held);
    void *h = c.fits(held, kI32, {R}), *ad = c.fits(a[1], kI32, {R}), *t = c.fits(table, kI32, {R, cols});
    void *fb = c.fits(free_blocks, kI32, {nfree}), *fc = c.fits(a[4], kI32, {1});
    const at::Tensor start = c.result(a[9], kI32, {R + 1}), slots = c.result(a[10], kI32, {nslots}), left = c.result(a[11], kI32, {1});
    const Workspace ws(c, a[12], a[13] != Py_False, lib.plan_ws((int)R));
    Tuple r = results(start, slots, left, ws.tensor_);
    void *const stream = c.stream();
    const int rc = lib.plan(static_cast<int32_t *>(h), static_cast<int32_t *>(ad), static_cast<int32_t *>(t), static_cast<int32_t *>(fb),
                            static_cast<int32_t *>(fc), static_cast<int32_t *>(left.data_ptr()), static_cast<int32_t *>(start.data_ptr()),
                            static_cast<int32_t *>(slots.data_ptr()), (int)R, (int)cols, bs, m, nblocks, (int)nfree, nslots,
                            ws.ptr, ws.bytes, stream);
    return answer(rc, r);
  });
}

// x, slots, pool, scale, ws, check
PyObject *cache_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    need(n == 6);
    const at::Tensor &x = tensor(a[0]), &pool = tensor(a[2]);
    need(x.dim() == 2 && pool.dim() == 3);
    const int64_t N = x.size(0), D = x.size(1), nblocks = pool.size(0), bs = pool.size(1);
    need(N <= INT_MAX && D <= INT_MAX && nblocks <= INT_MAX && bs <= INT_MAX);
    const int dt = dtype_code(x.scalar_type());
    const Call c(x);
    void *px = c.fits(x, x.scalar_type(), {N, D}), *ps = c.fits(a[1], kI32, {N});
    void *pp = c.fits(pool, kE4m3, {nblocks, bs, D}), *pc = c.fits(a[3], kF32, {nblocks});
    const Workspace ws(c, a[4], a[5] != Py_False, lib.append_ws((int)nblocks));
    Tuple r = results(ws.tensor_);
    void *const stream = c.stream();
    const int rc = lib.append(px, static_cast<int32_t *>(ps), pp, static_cast<float *>(pc), (int)N, (int)D, (int)bs, (int)nblocks, dt,
                              ws.ptr, ws.bytes, stream);
    return answer(rc, r);
  });
}

struct Cache {
  void *pool = nullptr, *scale = nullptr, *table = nullptr;
  int nblocks = 0, cols = 0;
};

Cache cache_of(const Call &c, PyObject *o, int64_t R, int64_t bs, int64_t D) {
  Cache r;
  if (o == Py_None) return r;
  need(PyTuple_CheckExact(o) && PyTuple_GET_SIZE(o) == 3);
  const at::Tensor &pool = tensor(PyTuple_GET_ITEM(o, 0)), &table = tensor(PyTuple_GET_ITEM(o, 2));
  need(pool.dim() == 3 && table.dim() == 2);
  const int64_t nblocks = pool.size(0), cols = table.size(1);
  need(nblocks <= INT_MAX && cols <= INT_MAX);
  r.pool = c.fits(pool, kE4m3, {nblocks, bs, D});
  r.scale = c.fits(PyTuple_GET_ITEM(o, 1), kF32, {nblocks});
  r.table = c.fits(table, kI32, {R, cols});
  r.nblocks = (int)nblocks;
  r.cols = (int)cols;
  return r;
}

// q, start, held, raw, comp, W, m, scale, out, lse, ws, check
PyObject *cache_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    need(n == 12);
    const at::Tensor &q = tensor(a[0]), &held = tensor(a[2]);
    need(q.dim() == 3 && held.dim() == 1 && PyTuple_CheckExact(a[3]) && PyTuple_GET_SIZE(a[3]) == 3);
    const at::Tensor &raw_pool = tensor(PyTuple_GET_ITEM(a[3], 0));
    need(raw_pool.dim() == 3);
    const int64_t N = q.size(0), H = q.size(1), D = q.size(2), R = held.size(0), bs = raw_pool.size(1);
    need(N <= INT_MAX && H <= INT_MAX && D <= INT_MAX && R < INT_MAX && bs <= INT_MAX);
    const int W = integer(a[5]), m = integer(a[6]), dt = dtype_code(q.scalar_type());
    need(PyFloat_CheckExact(a[7]));
    const float scale = (float)PyFloat_AS_DOUBLE(a[7]);
    const Call c(q);
    const Cache raw = cache_of(c, a[3], R, bs, D), comp = cache_of(c, a[4], R, bs, D);
    void *pq = c.fits(q, q.scalar_type(), {N, H, D}), *ps = c.fits(a[1], kI32, {R + 1}), *ph = c.fits(held, kI32, {R});
    const size_t bytes = lib.attn_ws((int)N, (int)R, (int)H, (int)D, dt);
    need(bytes > 0);
    const at::Tensor out = c.result(a[8], q.scalar_type(), {N, H, D}), lse = c.result(a[9], kF32, {N, H});
    const Workspace ws(c, a[10], a[11] != Py_False, bytes);
    Tuple r = results(out, lse, ws.tensor_);
    void *const stream = c.stream();
    const int rc = lib.attn(pq, static_cast<int32_t *>(ps), static_cast<int32_t *>(ph), raw.pool, static_cast<float *>(raw.scale),
                            static_cast<int32_t *>(raw.table), raw.nblocks, raw.cols, comp.pool, static_cast<float *>(comp.scale),
                            static_cast<int32_t *>(comp.table), comp.nblocks, comp.cols, out.data_ptr(),
                            static_cast<float *>(lse.data_ptr()), (int)N, (int)R, (int)H, (int)D, W, m, (int)bs, scale, dt,
                            ws.ptr, ws.bytes, stream);
    return answer(rc, r);
  });
}

// addresses of the C functions, in the order of `lib`
PyObject *bind(PyObject *, PyObject *args) {
  unsigned long long f[6];
  if (!PyArg_ParseTuple(args, "KKKKKK", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5])) return nullptr;
  lib.plan_ws = reinterpret_cast<decltype(lib.plan_ws)>(f[0]);
  lib.plan = reinterpret_cast<decltype(lib.plan)>(f[1]);
  lib.append_ws = reinterpret_cast<decltype(lib.append_ws)>(f[2]);
  lib.append = reinterpret_cast<decltype(lib.append)>(f[3]);
  lib.attn_ws = reinterpret_cast<decltype(lib.attn_ws)>(f[4]);
  lib.attn = reinterpret_cast<decltype(lib.attn)>(f[5]);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"cache_plan", fast(cache_plan), METH_FASTCALL, nullptr},
    {"cache_append", fast(cache_append), METH_FASTCALL, nullptr},
    {"cache_attn", fast(cache_attn), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hca_py", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__hca_py() {
  PyObject *m = PyModule_Create(&module);
  // what torch's headers were: hca.py uses the module with that torch only
  if (m && PyModule_AddStringConstant(m, "torch_version", HCA_TORCH) != 0) Py_CLEAR(m);
  return m;
}
