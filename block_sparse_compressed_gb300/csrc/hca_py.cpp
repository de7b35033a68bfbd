// hca_py.cpp -- the serving calls of hca.py, and those of the norms with positions,
// without their Python
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
#include <ATen/ops/empty_like.h>
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
  decltype(&hca_cache_attn_shared_workspace_size) shared_ws;
  decltype(&hca_cache_attn_shared) shared;
  decltype(&hca_norm_rope_fwd) norm_rope_fwd;
  decltype(&hca_norm_rope_workspace_size) norm_rope_ws;
  decltype(&hca_norm_rope_bwd) norm_rope_bwd;
  decltype(&hca_rope) rope;
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

// q, start, held, raw, comp, first, shared_cols, W, m, scale, out, lse, ws, check
PyObject *cache_attn_shared(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    need(n == 14);
    const at::Tensor &q = tensor(a[0]), &held = tensor(a[2]), &cols = tensor(a[6]);
    need(q.dim() == 3 && held.dim() == 1 && cols.dim() == 1 && PyTuple_CheckExact(a[3]) && PyTuple_GET_SIZE(a[3]) == 3 && a[4] != Py_None);
    const at::Tensor &raw_pool = tensor(PyTuple_GET_ITEM(a[3], 0));
    need(raw_pool.dim() == 3);
    const int64_t N = q.size(0), H = q.size(1), D = q.size(2), R = held.size(0), bs = raw_pool.size(1), G = cols.size(0);
    need(N <= INT_MAX && H <= INT_MAX && D <= INT_MAX && R < INT_MAX && bs <= INT_MAX && G < INT_MAX);
    const int W = integer(a[7]), m = integer(a[8]), dt = dtype_code(q.scalar_type());
    need(PyFloat_CheckExact(a[9]));
    const float scale = (float)PyFloat_AS_DOUBLE(a[9]);
    const Call c(q);
    const Cache raw = cache_of(c, a[3], R, bs, D), comp = cache_of(c, a[4], R, bs, D);
    void *pq = c.fits(q, q.scalar_type(), {N, H, D}), *ps = c.fits(a[1], kI32, {R + 1}), *ph = c.fits(held, kI32, {R});
    void *pf = c.fits(a[5], kI32, {G + 1}), *pc = c.fits(cols, kI32, {G});
    const size_t bytes = lib.shared_ws((int)N, (int)R, (int)H, (int)D, (int)G, dt);
    need(bytes > 0);
    const at::Tensor out = c.result(a[10], q.scalar_type(), {N, H, D}), lse = c.result(a[11], kF32, {N, H});
    const Workspace ws(c, a[12], a[13] != Py_False, bytes);
    Tuple r = results(out, lse, ws.tensor_);
    void *const stream = c.stream();
    const int rc = lib.shared(pq, static_cast<int32_t *>(ps), static_cast<int32_t *>(ph), raw.pool, static_cast<float *>(raw.scale),
                              static_cast<int32_t *>(raw.table), raw.nblocks, raw.cols, comp.pool, static_cast<float *>(comp.scale),
                              static_cast<int32_t *>(comp.table), comp.nblocks, comp.cols, static_cast<int32_t *>(pf),
                              static_cast<int32_t *>(pc), out.data_ptr(), static_cast<float *>(lse.data_ptr()), (int)N, (int)R, (int)H,
                              (int)D, (int)G, W, m, (int)bs, scale, dt, ws.ptr, ws.bytes, stream);
    return answer(rc, r);
  });
}

// Rows with adjacent columns: their pointer, and the strides of the other
// dimensions where they are not contiguous.
struct Rows {
  void *ptr = nullptr;
  int64_t v[3];
  const int64_t *strides = nullptr;

  Rows() = default;
  // packed: [N,H,D] or [N,D] as batch rows of one, heads and positions
  Rows(const Call &c, const at::Tensor &t, at::ScalarType type, at::IntArrayRef shape, bool packed) {
    need(t.is_cuda() && t.get_device() == c.dev && t.scalar_type() == type && t.sizes() == shape);
    ptr = t.data_ptr();
    if (t.is_contiguous()) return;
    const auto st = t.strides();
    need(st.back() == 1);
    if (packed) {
      v[0] = 0;
      if (shape.size() == 3) v[1] = st[1], v[2] = st[0];
      else v[1] = st[0];
    } else {
      for (size_t i = 0; i + 1 < shape.size(); ++i) v[i] = st[i];
    }
    strides = v;
  }
  Rows(const Rows &) = delete;
  Rows &operator=(const Rows &o) {
    ptr = o.ptr;
    for (int i = 0; i < 3; ++i) v[i] = o.v[i];
    strides = o.strides ? v : nullptr;
    return *this;
  }
};

// Coordinates of tokens (a batch of them, or packed ones) and frequencies
struct Angles {
  int32_t *pos = nullptr;
  float *freq;
  int axes, rot, first;

  Angles(const Call &c, PyObject *pos_, PyObject *freq_, PyObject *first_, at::IntArrayRef lead, int64_t D) {
    const at::Tensor &f = tensor(freq_);
    need(f.is_cuda() && f.get_device() == c.dev && f.scalar_type() == kF32 && f.is_contiguous() && (f.dim() == 1 || f.dim() == 2));
    need(f.size(-1) <= INT_MAX / 2);
    freq = static_cast<float *>(f.data_ptr());
    axes = f.dim() == 2 ? (int)f.size(0) : 1;
    rot = 2 * (int)f.size(-1);
    first = first_ == Py_None ? (int)D - rot : integer(first_);
    if (pos_ == Py_None) {
      need(axes == 1);
      return;
    }
    const at::Tensor &p = tensor(pos_);
    need(p.is_cuda() && p.get_device() == c.dev && p.scalar_type() == kI32 && p.is_contiguous());
    if (!(axes == 1 && p.sizes() == lead)) {
      need(p.dim() == (int64_t)lead.size() + 1 && p.size(0) == axes && p.sizes().slice(1) == lead);
    }
    pos = static_cast<int32_t *>(p.data_ptr());
  }
};

float number(PyObject *o) {
  need(PyFloat_CheckExact(o));
  return (float)PyFloat_AS_DOUBLE(o);
}

int flag(PyObject *o) {
  need(PyBool_Check(o));
  return o == Py_True;
}

const float *weight(const Call &c, PyObject *o, int64_t D) { return o == Py_None ? nullptr : static_cast<float *>(c.fits(o, kF32, {D})); }

// Sizes of q [B,H,S,D] and kv [B,S,D], or packed q [N,H,D] and kv [N,D]; one may be None
struct Pair {
  const at::Tensor *q = nullptr, *kv = nullptr, *any;
  int64_t B = 1, H = 0, S, D;
  at::ScalarType type;
  at::DimVector qshape, kvshape, lead;

  Pair(PyObject *q_, PyObject *kv_, bool packed) {
    if (q_ != Py_None) q = &tensor(q_);
    if (kv_ != Py_None) kv = &tensor(kv_);
    need(q || kv);
    any = q ? q : kv;
    const int64_t lead_dims = packed ? 1 : 2;
    need((!q || q->dim() == lead_dims + 2) && (!kv || kv->dim() == lead_dims + 1));
    D = any->size(-1);
    S = packed ? any->size(0) : any->size(-2);
    if (!packed) B = any->size(0);
    if (q) H = q->size(1);
    need(B <= INT_MAX && H <= INT_MAX && S <= INT_MAX && D <= INT_MAX);
    type = any->scalar_type();
    if (packed) {
      qshape = {S, H, D};
      kvshape = {S, D};
      lead = {S};
    } else {
      qshape = {B, H, S, D};
      kvshape = {B, S, D};
      lead = {B, S};
    }
  }
};

at::Tensor result_like(const Call &c, PyObject *o, at::ScalarType type, at::IntArrayRef shape) {
  if (o != Py_None) {
    const at::Tensor &t = tensor(o);
    need(t.is_cuda() && t.get_device() == c.dev && t.scalar_type() == type && t.sizes() == shape && t.is_contiguous());
    return t;
  }
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, c.dev)));
}

// q, kv, start, held, wq, wkv, pos, freq, eps, first, halves, qo, kvo (start None: a batch; else packed)
PyObject *norm_rope_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    need(n == 13);
    const bool packed = a[2] != Py_None;
    const Pair s(a[0], a[1], packed);
    const int dt = dtype_code(s.type);
    const Call c(*s.any);
    const float eps = number(a[8]);
    const Angles an(c, a[6], a[7], a[9], s.lead, s.D);
    const int halves = flag(a[10]);
    void *ps = nullptr, *ph = nullptr;
    int64_t R = 0;
    if (packed) {
      const at::Tensor &start = tensor(a[2]);
      need(start.dim() == 1 && start.size(0) >= 1 && start.size(0) <= INT_MAX && (a[3] != Py_None || an.pos));
      R = start.size(0) - 1;
      ps = c.fits(start, kI32, {R + 1});
      if (a[3] != Py_None) ph = c.fits(a[3], kI32, {R});
    }
    const float *wq = nullptr, *wkv = nullptr;
    Rows xq, xkv;
    at::Tensor qo, kvo;
    if (s.q) {
      xq = Rows(c, *s.q, s.type, s.qshape, packed);
      wq = weight(c, a[4], s.D);
      qo = result_like(c, a[11], s.type, s.qshape);
    }
    if (s.kv) {
      xkv = Rows(c, *s.kv, s.type, s.kvshape, packed);
      wkv = weight(c, a[5], s.D);
      kvo = result_like(c, a[12], s.type, s.kvshape);
    }
    Tuple r = results(qo, kvo);
    void *const stream = c.stream();
    const int rc = lib.norm_rope_fwd(xq.ptr, xq.strides, wq, s.q ? qo.data_ptr() : nullptr, xkv.ptr, xkv.strides, wkv,
                                     s.kv ? kvo.data_ptr() : nullptr, an.pos, an.freq, static_cast<int32_t *>(ps),
                                     static_cast<int32_t *>(ph), (int)s.B, (int)s.H, (int)s.S, (int)s.D, (int)R, an.axes, an.first, an.rot,
                                     halves, eps, dt, stream);
    return answer(rc, r);
  });
}

// The gradient of x: the caller's, or one laid out as x is.
at::Tensor gradient(const Call &c, PyObject *o, const at::Tensor &x) {
  if (o != Py_None) return tensor(o);
  for (const int64_t st : x.strides()) need(st != 0);
  return at::empty_like(x);
}

// q, kv, wq, wkv, pos, freq, eps, dqo, dkvo, first, halves, dq, dkv, dwq, dwkv, ws
PyObject *norm_rope_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    need(n == 16);
    const Pair s(a[0], a[1], false);
    const int dt = dtype_code(s.type);
    const Call c(*s.any);
    const float eps = number(a[6]);
    const Angles an(c, a[4], a[5], a[9], s.lead, s.D);
    const int halves = flag(a[10]);
    const float *w[2] = {nullptr, nullptr};
    void *g[2] = {nullptr, nullptr};
    Rows x[2], dx[2];
    at::Tensor gx[2], dw[2];
    for (int i = 0; i < 2; ++i) {
      const at::Tensor *t = i ? s.kv : s.q;
      if (!t) continue;
      const at::IntArrayRef shape = i ? s.kvshape : s.qshape;
      x[i] = Rows(c, *t, s.type, shape, false);
      const at::Tensor &cot = tensor(a[7 + i]);
      need(cot.is_cuda() && cot.get_device() == c.dev && cot.scalar_type() == s.type && cot.sizes() == shape && cot.is_contiguous());
      g[i] = cot.data_ptr();
      gx[i] = gradient(c, a[11 + i], *t);
      dx[i] = Rows(c, gx[i], s.type, shape, false);
      w[i] = weight(c, a[2 + i], s.D);
      need(w[i] || a[13 + i] == Py_None);
      if (w[i]) dw[i] = result_like(c, a[13 + i], kF32, {s.D});
    }
    const Workspace ws(c, a[15], false, lib.norm_rope_ws((int)s.D));
    Tuple r = results(gx[0], gx[1], dw[0], dw[1]);
    void *const stream = c.stream();
    auto ptr = [](const at::Tensor &t) { return t.defined() ? static_cast<float *>(t.data_ptr()) : nullptr; };
    const int rc = lib.norm_rope_bwd(x[0].ptr, x[0].strides, w[0], g[0], dx[0].ptr, dx[0].strides, ptr(dw[0]), x[1].ptr, x[1].strides, w[1],
                                     g[1], dx[1].ptr, dx[1].strides, ptr(dw[1]), an.pos, an.freq, (int)s.B, (int)s.H, (int)s.S, (int)s.D,
                                     an.axes, an.first, an.rot, halves, eps, dt, ws.ptr, ws.bytes, stream);
    return answer(rc, r);
  });
}

// x, start, held, pos, freq, inverse, first, halves, y (start None: a batch; else packed)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    need(n == 9);
    const bool packed = a[1] != Py_None;
    const Pair s(a[0], Py_None, packed);
    const int dt = dtype_code(s.type);
    const Call c(*s.any);
    const Angles an(c, a[3], a[4], a[6], s.lead, s.D);
    const int inverse = flag(a[5]), halves = flag(a[7]);
    void *ps = nullptr, *ph = nullptr;
    int64_t R = 0;
    if (packed) {
      const at::Tensor &start = tensor(a[1]);
      need(start.dim() == 1 && start.size(0) >= 1 && start.size(0) <= INT_MAX && (a[2] != Py_None || an.pos));
      R = start.size(0) - 1;
      ps = c.fits(start, kI32, {R + 1});
      if (a[2] != Py_None) ph = c.fits(a[2], kI32, {R});
    }
    const Rows x(c, *s.q, s.type, s.qshape, packed);
    const at::Tensor out = a[8] != Py_None ? tensor(a[8]) : result_like(c, Py_None, s.type, s.qshape);
    const Rows y(c, out, s.type, s.qshape, packed);
    Tuple r = results(out);
    void *const stream = c.stream();
    const int rc = lib.rope(x.ptr, x.strides, y.ptr, y.strides, an.pos, an.freq, static_cast<int32_t *>(ps), static_cast<int32_t *>(ph),
                            (int)s.B, (int)s.H, (int)s.S, (int)s.D, (int)R, an.axes, an.first, an.rot, halves, inverse, dt, stream);
    return answer(rc, r);
  });
}

// addresses of the C functions, in the order of `lib`
PyObject *bind(PyObject *, PyObject *args) {
  unsigned long long f[12];
  if (!PyArg_ParseTuple(args, "KKKKKKKKKKKK", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &f[7], &f[8], &f[9], &f[10], &f[11]))
    return nullptr;
  lib.plan_ws = reinterpret_cast<decltype(lib.plan_ws)>(f[0]);
  lib.plan = reinterpret_cast<decltype(lib.plan)>(f[1]);
  lib.append_ws = reinterpret_cast<decltype(lib.append_ws)>(f[2]);
  lib.append = reinterpret_cast<decltype(lib.append)>(f[3]);
  lib.attn_ws = reinterpret_cast<decltype(lib.attn_ws)>(f[4]);
  lib.attn = reinterpret_cast<decltype(lib.attn)>(f[5]);
  lib.shared_ws = reinterpret_cast<decltype(lib.shared_ws)>(f[6]);
  lib.shared = reinterpret_cast<decltype(lib.shared)>(f[7]);
  lib.norm_rope_fwd = reinterpret_cast<decltype(lib.norm_rope_fwd)>(f[8]);
  lib.norm_rope_ws = reinterpret_cast<decltype(lib.norm_rope_ws)>(f[9]);
  lib.norm_rope_bwd = reinterpret_cast<decltype(lib.norm_rope_bwd)>(f[10]);
  lib.rope = reinterpret_cast<decltype(lib.rope)>(f[11]);
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
    {"cache_attn_shared", fast(cache_attn_shared), METH_FASTCALL, nullptr},
    {"norm_rope_fwd", fast(norm_rope_fwd), METH_FASTCALL, nullptr},
    {"norm_rope_bwd", fast(norm_rope_bwd), METH_FASTCALL, nullptr},
    {"rope", fast(rope), METH_FASTCALL, nullptr},
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
