// marshal.cpp -- the Python side of the token mixers' entry points: reads
// sizes, strides and addresses off torch tensors, checks that they fit
// together, and calls the C ABI on the tensors' device and the given (or that
// device's current) stream.  A call costs about 2 us of host time here where
// the same checks written in Python cost 18 us: single-token calls run for 3
// to 12 us on the device.  Nothing is kept between calls.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "redlite_moe.h"

// What this file was built against (the build gives it); read from the binary
// before it is loaded.
extern "C" __attribute__((used, visibility("default"))) const char redlite_marshal_abi[];
const char redlite_marshal_abi[] = "redlite_marshal_abi:" REDLITE_MARSHAL_ABI ";";

namespace {

struct Bad {};      // arguments that do not fit together: REDLITE_EINVAL
struct Raised {};   // a Python error is set

using at::Tensor;

const Tensor &tensor(PyObject *o) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "expected a tensor, got %s", Py_TYPE(o)->tp_name);
    throw Raised();
  }
  return THPVariable_Unpack(o);
}
const Tensor *maybe(PyObject *o) { return o == Py_None ? nullptr : &tensor(o); }

double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}
int32_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (v < INT32_MIN || v > INT32_MAX) throw Bad();
  return (int32_t)v;
}
int32_t count(int64_t n) {
  if (n > INT32_MAX) throw Bad();
  return (int32_t)n;
}

int32_t dtype_of(const Tensor &t) {
  switch (t.scalar_type()) {
    case at::kFloat: return REDLITE_T_F32;
    case at::kBFloat16: return REDLITE_T_BF16;
    case at::kHalf: return REDLITE_T_F16;
    default: throw Bad();
  }
}

// The activations of a call: [rows, heads, head_dim] with dense heads, of one
// type and device; only the row stride is free.
struct Call {
  c10::Device device;
  at::ScalarType type;
  int32_t dtype;

  explicit Call(const Tensor &first) : device(first.device()), type(first.scalar_type()), dtype(dtype_of(first)) {
    if (!first.is_cuda()) throw Bad();
  }
  int64_t heads(const Tensor &t) const {  // its row stride
    if (t.dim() != 3 || t.device() != device || t.scalar_type() != type) throw Bad();
    const auto size = t.sizes();
    const auto stride = t.strides();
    if ((size[2] > 1 && stride[2] != 1) || (size[1] > 1 && stride[1] != size[2])) throw Bad();
    // the stride of a dimension of one element says nothing
    return size[0] > 1 ? stride[0] : size[1] * size[2];
  }
  template <typename T>
  T *dense(const Tensor &t, at::ScalarType want) const {
    if (t.scalar_type() != want || t.device() != device || !t.is_contiguous()) throw Bad();
    return (T *)t.data_ptr();
  }
  template <typename T>
  T *dense(const Tensor *t, at::ScalarType want) const {
    return t ? dense<T>(*t, want) : nullptr;
  }
  void *bytes(const Tensor &t, size_t &n) const {
    if (t.device() != device || !t.is_contiguous()) throw Bad();
    n = (size_t)t.numel() * t.element_size();
    return t.data_ptr();
  }
  void *stream(PyObject *o) const {
    if (o == Py_None) return (void *)c10::cuda::getCurrentCUDAStream(device.index()).stream();
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raised();
    return p;
  }
};

void need(bool ok) {
  if (!ok) throw Bad();
}

// q, k, v, cu_q, cu_k, out, scale, status, stream
int attn_prefill(PyObject *const *a) {
  const Tensor &q = tensor(a[0]), &k = tensor(a[1]), &v = tensor(a[2]), &cu_q = tensor(a[3]), &cu_k = tensor(a[4]),
               &out = tensor(a[5]);
  const Call c(q);
  const int64_t qs = c.heads(q), ks = c.heads(k), vs = c.heads(v), os = c.heads(out);
  const auto *pq = c.dense<int32_t>(cu_q, at::kInt), *pk = c.dense<int32_t>(cu_k, at::kInt);
  const int64_t n = cu_q.numel() - 1;
  need(n >= 0 && cu_k.numel() == n + 1 && q.sizes() == out.sizes() && k.sizes() == v.sizes() && q.size(2) == k.size(2));
  auto *status = c.dense<int32_t>(maybe(a[7]), at::kInt);
  const float scale = (float)number(a[6]);
  const c10::cuda::CUDAGuard guard(c.device);
  return redlite_attn_prefill(c.dtype, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, pq, pk, count(n),
                              count(q.size(0)), count(k.size(0)), count(q.size(1)), count(k.size(1)), count(q.size(2)),
                              scale, out.data_ptr(), os, status, c.stream(a[8]));
}

// Pages that a cache holds; a cache that is not one of whole pages is refused
// with the code in `rc`.
bool pages(const Tensor &cache, int32_t heads, int32_t D, int32_t page, int64_t &n, int &rc) {
  const size_t b = redlite_kv4_page_bytes(heads, D, page);
  rc = b ? REDLITE_EINVAL : REDLITE_EUNSUPPORTED;
  if (!b || cache.numel() % (int64_t)b) return false;
  n = cache.numel() / (int64_t)b;
  return true;
}

// k, v, cu_tokens, start, block_table, cache, page_size, status, stream; load: k and v are written
template <bool APPEND>
int kv4_rows(PyObject *const *a) {
  const Tensor &k = tensor(a[0]), &v = tensor(a[1]), &cu = tensor(a[2]), &start = tensor(a[3]), &table = tensor(a[4]),
               &cache = tensor(a[5]);
  const Call c(k);
  const int64_t ks = c.heads(k), vs = c.heads(v), n = start.numel();
  const auto *pcu = c.dense<int32_t>(cu, at::kInt), *pstart = c.dense<int32_t>(start, at::kInt),
             *ptable = c.dense<int32_t>(table, at::kInt);
  auto *pcache = c.dense<uint8_t>(cache, at::kByte);
  auto *status = c.dense<int32_t>(maybe(a[7]), at::kInt);
  need(k.sizes() == v.sizes() && cu.numel() == n + 1 && table.dim() == 2 && table.size(0) == n);
  const int32_t T = count(k.size(0)), H = count(k.size(1)), D = count(k.size(2)), page = integer(a[6]);
  int64_t n_pages = 0;
  int rc;
  if (!pages(cache, H, D, page, n_pages, rc)) return rc;
  const c10::cuda::CUDAGuard guard(c.device);
  void *s = c.stream(a[8]);
  if (APPEND)
    return redlite_kv4_append(c.dtype, k.data_ptr(), v.data_ptr(), ks, vs, pcu, pstart, count(n), T, H, D, page, ptable,
                              count(table.size(1)), n_pages, pcache, status, s);
  return redlite_kv4_load(c.dtype, pcache, H, D, page, ptable, count(table.size(1)), n_pages, pcu, pstart, count(n), T,
                          k.data_ptr(), v.data_ptr(), ks, vs, status, s);
}

// q, cache, page_size, block_table, lens, out, workspace, scale, status, stream, n_kv_heads
int kv4_decode(PyObject *const *a) {
  const Tensor &q = tensor(a[0]), &cache = tensor(a[1]), &table = tensor(a[3]), &lens = tensor(a[4]),
               &out = tensor(a[5]), &ws = tensor(a[6]);
  const Call c(q);
  const int64_t qs = c.heads(q), os = c.heads(out), B = q.size(0);
  auto *pcache = c.dense<uint8_t>(cache, at::kByte);
  const auto *ptable = c.dense<int32_t>(table, at::kInt), *plens = c.dense<int32_t>(lens, at::kInt);
  auto *status = c.dense<int32_t>(maybe(a[8]), at::kInt);
  size_t wb;
  void *pws = c.bytes(ws, wb);
  need(q.sizes() == out.sizes() && lens.numel() == B && table.dim() == 2 && table.size(0) == B);
  need(a[10] != Py_None || cache.dim() >= 2);
  const int32_t hk = a[10] != Py_None ? integer(a[10]) : count(cache.size(1)), D = count(q.size(2)),
                page = integer(a[2]);
  int64_t n_pages = 0;
  int rc;
  if (!pages(cache, hk, D, page, n_pages, rc)) return rc;
  const float scale = (float)number(a[7]);
  const c10::cuda::CUDAGuard guard(c.device);
  return redlite_kv4_decode(c.dtype, q.data_ptr(), qs, count(B), count(q.size(1)), hk, D, pcache, page, ptable,
                            count(table.size(1)), n_pages, plens, scale, out.data_ptr(), os, pws, wb, status,
                            c.stream(a[9]));
}

struct Delta {
  const Tensor &q, &k, &v, &g, &beta, &state_out, &out;
  const Call c;
  int64_t qs, ks, vs, os, n_slots;
  const float *pg, *pb, *si;
  float *so;
  const int32_t *slots;
  int32_t *status, rows, hk, hv, dk, dv;

  // q, k, v, g, beta, then state_in, state_out, slots, out from `s`, and the status
  Delta(PyObject *const *a, PyObject *const *s, PyObject *st, int64_t n_seqs)
      : q(tensor(a[0])), k(tensor(a[1])), v(tensor(a[2])), g(tensor(a[3])), beta(tensor(a[4])), state_out(tensor(s[1])),
        out(tensor(s[3])), c(q) {
    const Tensor *in = maybe(s[0]), *sl = maybe(s[2]);
    qs = c.heads(q), ks = c.heads(k), vs = c.heads(v), os = c.heads(out);
    pg = c.dense<float>(g, at::kFloat), pb = c.dense<float>(beta, at::kFloat);
    si = c.dense<float>(in, at::kFloat), so = c.dense<float>(state_out, at::kFloat);
    slots = c.dense<int32_t>(sl, at::kInt), status = c.dense<int32_t>(maybe(st), at::kInt);
    rows = count(v.size(0)), hv = count(v.size(1)), dv = count(v.size(2)), hk = count(q.size(1)), dk = count(q.size(2));
    need(q.sizes() == k.sizes() && q.size(0) == rows && out.sizes() == v.sizes());
    need(g.dim() == 2 && g.size(0) == rows && g.size(1) == hv && beta.sizes() == g.sizes());
    need(state_out.dim() == 4 && state_out.size(1) == hv && state_out.size(2) == dk && state_out.size(3) == dv);
    need(!in || in->sizes() == state_out.sizes());
    need(!sl || sl->numel() == n_seqs);
    n_slots = state_out.size(0);
  }
};

// q, k, v, g, beta, cu, state_in, state_out, slots, out, workspace, scale, qk_eps, status, stream
int delta_prefill(PyObject *const *a) {
  const Tensor &cu = tensor(a[5]), &ws = tensor(a[10]);
  const int64_t n = cu.numel() - 1;
  need(n >= 0);
  const Delta d(a, a + 6, a[13], n);
  const auto *pcu = d.c.dense<int32_t>(cu, at::kInt);
  size_t wb;
  void *pws = d.c.bytes(ws, wb);
  const float scale = (float)number(a[11]), eps = (float)number(a[12]);
  const c10::cuda::CUDAGuard guard(d.c.device);
  return redlite_delta_prefill(d.c.dtype, d.q.data_ptr(), d.qs, d.k.data_ptr(), d.ks, d.v.data_ptr(), d.vs, d.pg, d.pb,
                               pcu, count(n), d.rows, d.hk, d.hv, d.dk, d.dv, scale, eps, d.si, d.so, d.slots,
                               d.n_slots, d.out.data_ptr(), d.os, pws, wb, d.status, d.c.stream(a[14]));
}

// q, k, v, g, beta, state_in, state_out, slots, out, scale, qk_eps, status, stream
int delta_step(PyObject *const *a) {
  const Tensor &q = tensor(a[0]);
  need(q.dim() == 3);
  const Delta d(a, a + 5, a[11], q.size(0));
  const float scale = (float)number(a[9]), eps = (float)number(a[10]);
  const c10::cuda::CUDAGuard guard(d.c.device);
  return redlite_delta_step(d.c.dtype, d.q.data_ptr(), d.qs, d.k.data_ptr(), d.ks, d.v.data_ptr(), d.vs, d.pg, d.pb,
                            d.rows, d.hk, d.hv, d.dk, d.dv, scale, eps, d.si, d.so, d.slots, d.n_slots,
                            d.out.data_ptr(), d.os, d.status, d.c.stream(a[12]));
}

template <int (*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  int rc = REDLITE_EINVAL;
  try {
    rc = F(args);
  } catch (const Bad &) {
  } catch (const Raised &) {
    return nullptr;
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  return PyLong_FromLong(rc);
}

PyMethodDef methods[] = {
    {"attn_prefill", (PyCFunction)(void *)entry<attn_prefill, 9>, METH_FASTCALL, nullptr},
    {"kv4_append", (PyCFunction)(void *)entry<kv4_rows<true>, 9>, METH_FASTCALL, nullptr},
    {"kv4_load", (PyCFunction)(void *)entry<kv4_rows<false>, 9>, METH_FASTCALL, nullptr},
    {"kv4_decode", (PyCFunction)(void *)entry<kv4_decode, 11>, METH_FASTCALL, nullptr},
    {"delta_prefill", (PyCFunction)(void *)entry<delta_prefill, 15>, METH_FASTCALL, nullptr},
    {"delta_step", (PyCFunction)(void *)entry<delta_step, 13>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
