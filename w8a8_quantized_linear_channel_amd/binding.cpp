// The argument checks, allocations and C-ABI calls of the binding's
// latency-bound functions (ops.py) without the interpreter: a decode step's
// kernels take a few microseconds, and the same work in Python takes longer
// than they do (host time of a call: append of one token 14.0 us in Python, 5.4
// here; attention 16.5 and 5.2; linear of one token 12.5 and 4.7).  Every function returns its result, an int status of the
// C call that failed, or NotImplemented where an argument is not exactly what
// the call takes; ops.py then repeats its checks to say what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "q8.h"

namespace {

PyObject* g_raw_stream = nullptr;   // torch's current raw stream of a device index

bool tensor(PyObject* o, const at::Tensor** t) {
  if (!THPVariable_Check(o)) return false;
  *t = &THPVariable_Unpack(o);
  return true;
}
// null for None
bool optional_tensor(PyObject* o, const at::Tensor** t) {
  *t = nullptr;
  return o == Py_None || tensor(o, t);
}
bool dense(const at::Tensor& t, at::ScalarType dt, at::IntArrayRef shape, int64_t dev) {
  return t.is_cuda() && t.get_device() == dev && t.scalar_type() == dt && t.sizes() == shape && t.is_contiguous();
}
// [tokens, heads, dim], heads and features dense
bool rows(const at::Tensor& t, at::ScalarType dt, int64_t heads, int64_t dim, int64_t dev) {
  return t.is_cuda() && t.get_device() == dev && t.scalar_type() == dt && t.dim() == 3 && t.size(1) == heads &&
         t.size(2) == dim && (t.numel() == 0 || (t.stride(2) == 1 && (heads == 1 || t.stride(1) == dim)));
}
int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return Q8_F32;
    case at::kHalf: return Q8_F16;
    case at::kBFloat16: return Q8_BF16;
    default: return -1;
  }
}
void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

bool number(PyObject* o, int64_t* v) {
  if (!PyLong_Check(o)) return false;          // bool too
  *v = PyLong_AsLongLong(o);
  if (*v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}
// The current stream of the device; null and a Python error on failure.
bool stream_of(int64_t dev, void** st) {
  PyObject* i = PyLong_FromLongLong(dev);
  PyObject* r = i ? PyObject_CallOneArg(g_raw_stream, i) : nullptr;
  Py_XDECREF(i);
  if (!r) return false;
  *st = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return !PyErr_Occurred();
}

PyObject* not_ours() { Py_RETURN_NOTIMPLEMENTED; }
PyObject* finish(q8_status s, at::Tensor y) {
  if (s != Q8_OK) return PyLong_FromLong(s);
  return THPVariable_Wrap(std::move(y));
}

struct Kv {
  const at::Tensor *k, *ke, *v, *ve, *start, *len, *table;
  int64_t pages, heads, page, dim, seqs, max_pages, max_q, max_kv;
};
bool one_byte(at::ScalarType t, at::ScalarType other) { return t == at::kByte || t == other; }
bool unpack_kv(PyObject* cache, PyObject* batch, int64_t dev, Kv* o) {
  if (!PyTuple_Check(cache) || PyTuple_GET_SIZE(cache) != 4 || !PyTuple_Check(batch) || PyTuple_GET_SIZE(batch) != 5)
    return false;
  if (!tensor(PyTuple_GET_ITEM(cache, 0), &o->k) || !tensor(PyTuple_GET_ITEM(cache, 1), &o->ke) ||
      !tensor(PyTuple_GET_ITEM(cache, 2), &o->v) || !tensor(PyTuple_GET_ITEM(cache, 3), &o->ve) ||
      !tensor(PyTuple_GET_ITEM(batch, 0), &o->start) || !tensor(PyTuple_GET_ITEM(batch, 1), &o->len) ||
      !tensor(PyTuple_GET_ITEM(batch, 2), &o->table) || !number(PyTuple_GET_ITEM(batch, 3), &o->max_q) ||
      !number(PyTuple_GET_ITEM(batch, 4), &o->max_kv))
    return false;
  if (o->k->dim() != 4 || o->table->dim() != 2) return false;
  o->pages = o->k->size(0);
  o->heads = o->k->size(1);
  o->page = o->k->size(2);
  o->dim = o->k->size(3);
  o->seqs = o->table->size(0);
  o->max_pages = o->table->size(1);
  const at::ScalarType c = o->k->scalar_type(), e = o->ke->scalar_type();
  return one_byte(c, at::kFloat8_e4m3fn) && one_byte(e, at::kFloat8_e8m0fnu) &&
         dense(*o->k, c, {o->pages, o->heads, o->page, o->dim}, dev) &&
         dense(*o->v, c, {o->pages, o->heads, o->dim, o->page}, dev) && dense(*o->ke, e, {o->pages, o->heads}, dev) &&
         dense(*o->ve, e, {o->pages, o->heads}, dev) && dense(*o->table, at::kInt, {o->seqs, o->max_pages}, dev) &&
         dense(*o->start, at::kInt, {o->seqs + 1}, dev) && dense(*o->len, at::kInt, {o->seqs}, dev);
}

// (k, v, cache, batch, q, cos, sin, interleaved, out)
PyObject* kv_append(PyObject* const* a) {
  const at::Tensor *k, *v, *q, *cos, *sin, *out;
  Kv kv;
  if (!tensor(a[0], &k) || !tensor(a[1], &v) || !k->is_cuda()) return not_ours();
  const int64_t dev = k->get_device();
  if (!unpack_kv(a[2], a[3], dev, &kv) || !optional_tensor(a[4], &q) || !optional_tensor(a[5], &cos) ||
      !optional_tensor(a[6], &sin) || !optional_tensor(a[8], &out))
    return not_ours();
  const int turn = PyObject_IsTrue(a[7]);
  const at::ScalarType dt = k->scalar_type();
  const int code = dtype_code(dt);
  if (turn < 0 || code < 0 || !rows(*k, dt, kv.heads, kv.dim, dev) || !rows(*v, dt, kv.heads, kv.dim, dev) ||
      v->size(0) != k->size(0))
    return PyErr_Clear(), not_ours();
  const int64_t T = k->size(0);
  int64_t heads = 0, step = 0, positions = 0, rot = 0;
  at::Tensor y;
  if (q) {
    if (q->dim() != 3 || !rows(*q, dt, q->size(1), kv.dim, dev) || q->size(0) != T) return not_ours();
    heads = q->size(1);
    step = q->stride(0);
    if (out && !dense(*out, dt, {T, heads, kv.dim}, dev)) return not_ours();
    y = out ? *out : at::empty({T, heads, kv.dim}, q->options());
  } else if (out) {
    return not_ours();
  }
  if ((cos == nullptr) != (sin == nullptr)) return not_ours();
  if (cos) {
    if (cos->dim() != 2 || !dense(*cos, at::kFloat, cos->sizes(), dev) || !dense(*sin, at::kFloat, cos->sizes(), dev))
      return not_ours();
    positions = cos->size(0);
    rot = 2 * cos->size(1);
  }
  void* st;
  if (!stream_of(dev, &st)) return nullptr;
  const q8_status s = q8_kv_append(
      ptr(q), step, ptr(k), k->stride(0), ptr(v), v->stride(0), (q8_dtype)code, T, heads, kv.heads, kv.dim,
      (const float*)ptr(cos), (const float*)ptr(sin), positions, rot, turn, (const int32_t*)ptr(kv.start),
      (const int32_t*)ptr(kv.len), (const int32_t*)ptr(kv.table), kv.seqs, kv.max_pages, kv.max_q, (uint8_t*)ptr(kv.k),
      (uint8_t*)ptr(kv.ke), (uint8_t*)ptr(kv.v), (uint8_t*)ptr(kv.ve), kv.pages, kv.page, q ? y.data_ptr() : nullptr, st);
  if (s == Q8_OK && !q) Py_RETURN_NONE;
  return finish(s, std::move(y));
}

// (q, cache, batch, scale, causal, window, out): without lse and a caller's workspace
PyObject* attention_kv8(PyObject* const* a) {
  const at::Tensor *q, *out;
  Kv kv;
  int64_t window;
  if (!tensor(a[0], &q) || !q->is_cuda() || q->dim() != 3) return not_ours();
  const int64_t dev = q->get_device();
  if (!unpack_kv(a[1], a[2], dev, &kv) || !number(a[5], &window) || !optional_tensor(a[6], &out)) return not_ours();
  const at::ScalarType dt = q->scalar_type();
  const int causal = PyObject_IsTrue(a[4]);
  const double scale = a[3] == Py_None ? 1.0 / std::sqrt((double)kv.dim) : PyFloat_AsDouble(a[3]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return not_ours();
  }
  const int64_t T = q->size(0), heads = q->size(1);
  if ((dt != at::kHalf && dt != at::kBFloat16) || !rows(*q, dt, heads, kv.dim, dev) ||
      (out && !dense(*out, dt, {T, heads, kv.dim}, dev)))
    return not_ours();
  at::Tensor y = out ? *out : at::empty({T, heads, kv.dim}, q->options()), ws;
  const size_t need = q8_attention_workspace_bytes(T, heads, kv.heads, kv.dim, kv.seqs, kv.max_q, kv.max_kv, window);
  if (need) ws = at::empty({(int64_t)need}, kv.table->options().dtype(at::kByte));
  void* st;
  if (!stream_of(dev, &st)) return nullptr;
  const q8_status s = q8_attention_kv8(
      ptr(q), q->stride(0), (q8_dtype)dtype_code(dt), T, heads, kv.heads, kv.dim, (const int32_t*)ptr(kv.start),
      (const int32_t*)ptr(kv.len), (const int32_t*)ptr(kv.table), kv.seqs, kv.max_pages, kv.max_q, kv.max_kv,
      (const uint8_t*)ptr(kv.k), (const uint8_t*)ptr(kv.ke), (const uint8_t*)ptr(kv.v), (const uint8_t*)ptr(kv.ve),
      kv.pages, kv.page, (float)scale, causal, window, y.data_ptr(), nullptr, need ? ws.data_ptr() : nullptr, need, st);
  return finish(s, std::move(y));
}

// (k, v, cache, batch, q, q_weight, k_weight, eps, cos, sin, interleaved, positions, out)
PyObject* kv_append_norm(PyObject* const* a) {
  const at::Tensor *k, *v, *q, *qw, *kw, *cos, *sin, *pos, *out;
  Kv kv;
  if (!tensor(a[0], &k) || !tensor(a[1], &v) || !k->is_cuda()) return not_ours();
  const int64_t dev = k->get_device();
  if (!unpack_kv(a[2], a[3], dev, &kv) || !optional_tensor(a[4], &q) || !optional_tensor(a[5], &qw) ||
      !optional_tensor(a[6], &kw) || !optional_tensor(a[8], &cos) || !optional_tensor(a[9], &sin) ||
      !optional_tensor(a[11], &pos) || !optional_tensor(a[12], &out))
    return not_ours();
  const double eps = PyFloat_AsDouble(a[7]);
  const int turn = PyObject_IsTrue(a[10]);
  if (PyErr_Occurred()) return PyErr_Clear(), not_ours();
  const at::ScalarType dt = k->scalar_type();
  const int code = dtype_code(dt);
  if (turn < 0 || code < 0 || !rows(*k, dt, kv.heads, kv.dim, dev) || !rows(*v, dt, kv.heads, kv.dim, dev) ||
      v->size(0) != k->size(0))
    return not_ours();
  const int64_t T = k->size(0);
  const at::Tensor* const some = qw ? qw : kw;
  const at::ScalarType wd = some ? some->scalar_type() : at::kFloat;
  const int wcode = dtype_code(wd);
  if (wcode < 0 || (qw && !dense(*qw, wd, {kv.dim}, dev)) || (kw && !dense(*kw, wd, {kv.dim}, dev)) ||
      (pos && !dense(*pos, at::kInt, {T}, dev)) || (qw && !q))
    return not_ours();
  int64_t heads = 0, step = 0, positions = 0, rot = 0;
  c10::DeviceGuard guard(k->device());
  at::Tensor y;
  if (q) {
    if (q->dim() != 3 || !rows(*q, dt, q->size(1), kv.dim, dev) || q->size(0) != T) return not_ours();
    heads = q->size(1);
    step = q->stride(0);
    if (out && !dense(*out, dt, {T, heads, kv.dim}, dev)) return not_ours();
    y = out ? *out : at::empty({T, heads, kv.dim}, q->options());
  } else if (out) {
    return not_ours();
  }
  if ((cos == nullptr) != (sin == nullptr)) return not_ours();
  if (cos) {
    if (cos->dim() != 2 || !dense(*cos, at::kFloat, cos->sizes(), dev) || !dense(*sin, at::kFloat, cos->sizes(), dev))
      return not_ours();
    positions = cos->size(0);
    rot = 2 * cos->size(1);
  }
  void* st;
  if (!stream_of(dev, &st)) return nullptr;
  const q8_status s = q8_kv_append_norm(
      ptr(q), step, ptr(k), k->stride(0), ptr(v), v->stride(0), (q8_dtype)code, T, heads, kv.heads, kv.dim, ptr(qw),
      ptr(kw), (q8_dtype)wcode, (float)eps, (const float*)ptr(cos), (const float*)ptr(sin), positions, rot, turn,
      (const int32_t*)ptr(pos), (const int32_t*)ptr(kv.start), (const int32_t*)ptr(kv.len), (const int32_t*)ptr(kv.table),
      kv.seqs, kv.max_pages, kv.max_q, (uint8_t*)ptr(kv.k), (uint8_t*)ptr(kv.ke), (uint8_t*)ptr(kv.v),
      (uint8_t*)ptr(kv.ve), kv.pages, kv.page, q ? y.data_ptr() : nullptr, st);
  if (s == Q8_OK && !q) Py_RETURN_NONE;
  return finish(s, std::move(y));
}

// (q, cache, batch, mask, positions, scale, window, out): without lse and a caller's workspace
PyObject* attention_kv8_tree(PyObject* const* a) {
  const at::Tensor *q, *mask, *pos, *out;
  Kv kv;
  int64_t window;
  if (!tensor(a[0], &q) || !q->is_cuda() || q->dim() != 3) return not_ours();
  const int64_t dev = q->get_device();
  if (!unpack_kv(a[1], a[2], dev, &kv) || !tensor(a[3], &mask) || !optional_tensor(a[4], &pos) || !number(a[6], &window) ||
      !optional_tensor(a[7], &out))
    return not_ours();
  const at::ScalarType dt = q->scalar_type(), md = mask->scalar_type();
  const double scale = a[5] == Py_None ? 1.0 / std::sqrt((double)kv.dim) : PyFloat_AsDouble(a[5]);
  if (PyErr_Occurred()) return PyErr_Clear(), not_ours();
  const int64_t T = q->size(0), heads = q->size(1);
  if ((dt != at::kHalf && dt != at::kBFloat16) || !rows(*q, dt, heads, kv.dim, dev) || mask->dim() != 2 ||
      (md != at::kLong && md != at::kUInt64) || !dense(*mask, md, {T, mask->size(1)}, dev) ||
      (pos && !dense(*pos, at::kInt, {T}, dev)) || (out && !dense(*out, dt, {T, heads, kv.dim}, dev)))
    return not_ours();
  c10::DeviceGuard guard(q->device());
  at::Tensor y = out ? *out : at::empty({T, heads, kv.dim}, q->options()), ws;
  const size_t need = q8_attention_tree_workspace_bytes(T, heads, kv.heads, kv.dim, kv.seqs, kv.max_q, kv.max_kv, window);
  if (need) ws = at::empty({(int64_t)need}, kv.table->options().dtype(at::kByte));
  void* st;
  if (!stream_of(dev, &st)) return nullptr;
  const q8_status s = q8_attention_kv8_tree(
      ptr(q), q->stride(0), (q8_dtype)dtype_code(dt), T, heads, kv.heads, kv.dim, (const int32_t*)ptr(kv.start),
      (const int32_t*)ptr(kv.len), (const int32_t*)ptr(kv.table), kv.seqs, kv.max_pages, kv.max_q, kv.max_kv,
      (const uint8_t*)ptr(kv.k), (const uint8_t*)ptr(kv.ke), (const uint8_t*)ptr(kv.v), (const uint8_t*)ptr(kv.ve),
      kv.pages, kv.page, (const uint64_t*)ptr(mask), mask->size(1), (const int32_t*)ptr(pos), (float)scale, window,
      y.data_ptr(), nullptr, need ? ws.data_ptr() : nullptr, need, st);
  return finish(s, std::move(y));
}

// The caches of all layers: one cache (a tuple of four tensors) or a list or tuple of them, all alike.
struct Layers {
  static constexpr int kMost = 512;
  uint8_t *k[kMost], *ke[kMost], *v[kMost], *ve[kMost];
  int64_t n, pages, heads, page, dim, dev;
  c10::Device device = c10::Device(c10::kCPU);
};
bool unpack_layers(PyObject* o, Layers* l) {
  const at::Tensor* t;
  const bool one = PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 4 && tensor(PyTuple_GET_ITEM(o, 0), &t);
  if (!one && !PyTuple_Check(o) && !PyList_Check(o)) return false;
  l->n = one ? 1 : PySequence_Fast_GET_SIZE(o);
  if (l->n < 1 || l->n > Layers::kMost) return false;
  for (int64_t i = 0; i < l->n; ++i) {
    PyObject* const c = one ? o : PySequence_Fast_GET_ITEM(o, i);
    const at::Tensor *k, *ke, *v, *ve;
    if (!PyTuple_Check(c) || PyTuple_GET_SIZE(c) != 4 || !tensor(PyTuple_GET_ITEM(c, 0), &k) ||
        !tensor(PyTuple_GET_ITEM(c, 1), &ke) || !tensor(PyTuple_GET_ITEM(c, 2), &v) || !tensor(PyTuple_GET_ITEM(c, 3), &ve))
      return false;
    if (i == 0) {
      if (k->dim() != 4 || !k->is_cuda()) return false;
      l->pages = k->size(0);
      l->heads = k->size(1);
      l->page = k->size(2);
      l->dim = k->size(3);
      l->device = k->device();
      l->dev = k->get_device();
    }
    if (!one_byte(k->scalar_type(), at::kFloat8_e4m3fn) || !one_byte(v->scalar_type(), at::kFloat8_e4m3fn) ||
        !one_byte(ke->scalar_type(), at::kFloat8_e8m0fnu) || !one_byte(ve->scalar_type(), at::kFloat8_e8m0fnu) ||
        !dense(*k, k->scalar_type(), {l->pages, l->heads, l->page, l->dim}, l->dev) ||
        !dense(*v, v->scalar_type(), {l->pages, l->heads, l->dim, l->page}, l->dev) ||
        !dense(*ke, ke->scalar_type(), {l->pages, l->heads}, l->dev) ||
        !dense(*ve, ve->scalar_type(), {l->pages, l->heads}, l->dev))
      return false;
    l->k[i] = (uint8_t*)ptr(k);
    l->ke[i] = (uint8_t*)ptr(ke);
    l->v[i] = (uint8_t*)ptr(v);
    l->ve[i] = (uint8_t*)ptr(ve);
  }
  return true;
}

// (caches, batch, keep, n_keep, out)
PyObject* kv_compact(PyObject* const* a) {
  Layers l;
  const at::Tensor *start, *len, *table, *keep, *kept, *out;
  PyObject* const b = a[1];
  if (!unpack_layers(a[0], &l) || !PyTuple_Check(b) || PyTuple_GET_SIZE(b) != 5 || !tensor(PyTuple_GET_ITEM(b, 0), &start) ||
      !tensor(PyTuple_GET_ITEM(b, 1), &len) || !tensor(PyTuple_GET_ITEM(b, 2), &table) || !tensor(a[2], &keep) ||
      !tensor(a[3], &kept) || !optional_tensor(a[4], &out) || table->dim() != 2 || keep->dim() != 2)
    return not_ours();
  const int64_t S = table->size(0);
  if (!dense(*table, at::kInt, {S, table->size(1)}, l.dev) || !dense(*start, at::kInt, {S + 1}, l.dev) ||
      !dense(*len, at::kInt, {S}, l.dev) || !dense(*keep, at::kInt, {S, keep->size(1)}, l.dev) ||
      !dense(*kept, at::kInt, {S}, l.dev) || (out && !dense(*out, at::kInt, {S}, l.dev)))
    return not_ours();
  c10::DeviceGuard guard(l.device);
  at::Tensor y = out ? *out : at::empty({S}, len->options());
  void* st;
  if (!stream_of(l.dev, &st)) return nullptr;
  const q8_status s = q8_kv_compact(l.k, l.ke, l.v, l.ve, l.n, l.heads, l.dim, (const int32_t*)ptr(start),
                                    (const int32_t*)ptr(len), (const int32_t*)ptr(table), S, table->size(1), l.pages, l.page,
                                    (const int32_t*)ptr(keep), keep->size(1), (const int32_t*)ptr(kept),
                                    (int32_t*)y.data_ptr(), st);
  return finish(s, std::move(y));
}

// (caches, block_table, kv_len, refs, parent, room, out, workspace); a tuple of four tensors
PyObject* kv_fork(PyObject* const* a) {
  Layers l;
  const at::Tensor *table, *len, *refs, *parent, *given, *outs[4] = {};
  int64_t room;
  if (!unpack_layers(a[0], &l) || !tensor(a[1], &table) || !tensor(a[2], &len) || !tensor(a[3], &refs) ||
      !tensor(a[4], &parent) || !number(a[5], &room) || !optional_tensor(a[7], &given) || table->dim() != 2 ||
      parent->dim() != 1)
    return not_ours();
  const int64_t S = table->size(0), width = table->size(1), n = parent->size(0);
  if (!dense(*table, at::kInt, {S, width}, l.dev) || !dense(*len, at::kInt, {S}, l.dev) ||
      !dense(*refs, at::kInt, {l.pages}, l.dev) || !dense(*parent, at::kInt, {n}, l.dev) ||
      (given && (!given->is_cuda() || given->get_device() != l.dev || !given->is_contiguous())))
    return not_ours();
  c10::DeviceGuard guard(l.device);
  at::Tensor y[4], ws;
  if (a[6] != Py_None) {
    if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 4) return not_ours();
    for (int i = 0; i < 4; ++i)
      if (!tensor(PyTuple_GET_ITEM(a[6], i), &outs[i])) return not_ours();
    if (!dense(*outs[0], at::kInt, {n, width}, l.dev) || !dense(*outs[1], at::kInt, {n}, l.dev) ||
        !dense(*outs[2], at::kInt, {l.pages}, l.dev) || !dense(*outs[3], at::kInt, {1}, l.dev))
      return not_ours();
    for (int i = 0; i < 4; ++i) y[i] = *outs[i];
  } else {
    y[0] = at::empty({n, width}, table->options());
    y[1] = at::empty({n}, table->options());
    y[2] = at::empty({l.pages}, table->options());
    y[3] = at::empty({1}, table->options());
  }
  if (given) ws = *given;
  else ws = at::empty({(int64_t)q8_kv_fork_workspace_bytes(S, n, l.pages)}, table->options().dtype(at::kByte));
  void* st;
  if (!stream_of(l.dev, &st)) return nullptr;
  const q8_status s = q8_kv_fork(l.k, l.ke, l.v, l.ve, l.n, l.heads, l.dim, l.pages, l.page, (const int32_t*)ptr(table),
                                 (const int32_t*)ptr(len), (const int32_t*)ptr(refs), S, width, (const int32_t*)ptr(parent),
                                 n, room, (int32_t*)y[0].data_ptr(), (int32_t*)y[1].data_ptr(), (int32_t*)y[2].data_ptr(),
                                 (int32_t*)y[3].data_ptr(), ws.data_ptr(), ws.nbytes(), st);
  if (s != Q8_OK) return PyLong_FromLong(s);
  PyObject* const r = PyTuple_New(4);
  if (!r) return nullptr;
  for (int i = 0; i < 4; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(std::move(y[i])));
  return r;
}

// (x, wq, w_scale, bias, out_dtype, out): without a caller's workspace
PyObject* linear_fp8_block(PyObject* const* a) {
  const at::Tensor *x, *wq, *ws, *bias, *out;
  if (!tensor(a[0], &x) || !tensor(a[1], &wq) || !tensor(a[2], &ws) || !optional_tensor(a[3], &bias) ||
      !optional_tensor(a[5], &out) || !x->is_cuda() || x->dim() != 2 || wq->dim() != 2)
    return not_ours();
  const int64_t dev = x->get_device(), M = x->size(0), K = x->size(1), N = wq->size(0);
  const at::ScalarType xd = x->scalar_type();
  at::ScalarType yd = xd == at::kFloat ? at::kBFloat16 : xd;
  if (a[4] != Py_None) {
    if (!THPDtype_Check(a[4])) return not_ours();
    yd = reinterpret_cast<THPDtype*>(a[4])->scalar_type;
  }
  const int xc = dtype_code(xd), yc = dtype_code(yd);
  if (xc < 0 || yc < 0 || !x->is_contiguous() || !one_byte(wq->scalar_type(), at::kFloat8_e4m3fn) ||
      !dense(*wq, wq->scalar_type(), {N, K}, dev) ||
      !dense(*ws, at::kFloat, {(N + 127) / 128, (K + 127) / 128}, dev) || (bias && !dense(*bias, at::kFloat, {N}, dev)) ||
      (out && !dense(*out, yd, {M, N}, dev)))
    return not_ours();
  at::Tensor y = out ? *out : at::empty({M, N}, x->options().dtype(yd)), scratch;
  const size_t need = q8_workspace_bytes(Q8_OP_FP8_BLOCK, M, N, K);
  if (need) scratch = at::empty({(int64_t)need}, wq->options().dtype(at::kByte));
  void* st;
  if (!stream_of(dev, &st)) return nullptr;
  const q8_status s = q8_linear_fp8_block(ptr(x), (q8_dtype)xc, M, K, (const uint8_t*)ptr(wq), (const float*)ptr(ws), N,
                                          (const float*)ptr(bias), y.data_ptr(), (q8_dtype)yc,
                                          need ? scratch.data_ptr() : nullptr, need, st);
  return finish(s, std::move(y));
}

// A fixed number of positional arguments, and C++ exceptions (an allocation that fails) as Python's.
template <PyObject* (*F)(PyObject* const*), int ARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != ARGS) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", ARGS, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <PyObject* (*F)(PyObject* const*), int ARGS>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, ARGS>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<kv_append, 9>("kv_append"), method<attention_kv8, 7>("attention_kv8"),
                           method<kv_append_norm, 13>("kv_append_norm"), method<attention_kv8_tree, 8>("attention_kv8_tree"),
                           method<kv_compact, 5>("kv_compact"), method<kv_fork, 8>("kv_fork"),
                           method<linear_fp8_block, 6>("linear_fp8_block"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* c = PyImport_ImportModule("torch._C");
  if (!c) return nullptr;
  g_raw_stream = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
  Py_DECREF(c);
  if (!g_raw_stream) return nullptr;
  return PyModule_Create(&g_module);
}
