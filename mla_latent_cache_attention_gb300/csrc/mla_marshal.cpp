// mla_marshal.cpp -- the Python side of the selector's calls, in C: reads the tensors' addresses, shapes and
// strides, allocates the outputs and calls the C ABI.
//
// The calls of a decode step are short on the device (2 to 25 us); written in Python over ctypes their
// marshalling takes longer than that (insert 19.5 us, gather 14, selection 13 to 18, selected decode 30).
// Every function here serves the plain call only: exact types, tensors on the current device, shapes that
// fit.  Anything else, wrong arguments too, returns None, and the Python form of the call looks at it
// again, serves it or words the refusal.  It uses Python's C API and the tensors' own methods, no other
// library's headers.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>

#include "mla.h"

namespace {

struct Ref {                    // owns a reference
  PyObject* p;
  explicit Ref(PyObject* o = nullptr) : p(o) {}
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  ~Ref() { Py_XDECREF(p); }
  PyObject* release() {
    PyObject* o = p;
    p = nullptr;
    return o;
  }
};

// Given by init(), kept for the life of the process.
PyObject *g_tensor, *g_empty, *g_get_device, *g_stream, *g_check, *g_bf16, *g_u8, *g_i8, *g_f32, *g_i32, *g_i64;
PyObject *s_dtype, *s_shape, *s_stride, *s_ptr, *s_dev, *s_device, *g_empty_kw;

PyObject* not_plain() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

bool as_i64(PyObject* o, int64_t* v) {
  if (!PyLong_CheckExact(o)) return false;
  *v = PyLong_AsLongLong(o);
  return !(*v == -1 && PyErr_Occurred());
}
bool as_i32(PyObject* o, int32_t* v) {
  int64_t w;
  if (!as_i64(o, &w) || w < INT32_MIN || w > INT32_MAX) return false;
  *v = static_cast<int32_t>(w);
  return true;
}
bool as_float(PyObject* o, float* v) {
  if (!PyFloat_CheckExact(o)) return false;
  *v = static_cast<float>(PyFloat_AS_DOUBLE(o));
  return true;
}

struct Tensor {
  char* ptr;
  int64_t size[3], stride[3];
  int type;                     // which of the accepted types it has
};

// A plain tensor of device `dev` with `ndim` dimensions, unit innermost stride and one of the types.
bool read(PyObject* o, long dev, int ndim, Tensor* t, PyObject* t0, PyObject* t1 = nullptr, PyObject* t2 = nullptr) {
  if (reinterpret_cast<PyObject*>(Py_TYPE(o)) != g_tensor) return false;
  Ref dt(PyObject_GetAttr(o, s_dtype));
  if (!dt.p) return false;
  if (dt.p == t0)
    t->type = 0;
  else if (t1 && dt.p == t1)
    t->type = 1;
  else if (t2 && dt.p == t2)
    t->type = 2;
  else
    return false;
  Ref d(PyObject_CallMethodNoArgs(o, s_dev));
  if (!d.p || PyLong_AsLong(d.p) != dev) return false;
  Ref st(PyObject_CallMethodNoArgs(o, s_stride)), sh(PyObject_GetAttr(o, s_shape));
  if (!st.p || !sh.p || !PyTuple_Check(st.p) || !PyTuple_Check(sh.p) || PyTuple_GET_SIZE(st.p) != ndim ||
      PyTuple_GET_SIZE(sh.p) != ndim)
    return false;
  for (int i = 0; i < ndim; ++i)
    if (!as_i64(PyTuple_GET_ITEM(st.p, i), &t->stride[i]) || !as_i64(PyTuple_GET_ITEM(sh.p, i), &t->size[i])) return false;
  if (t->stride[ndim - 1] != 1) return false;
  // the C entries refuse rows that overlap; the stride of a dimension of one entry means nothing
  for (int i = ndim - 2; i >= 0; --i) {
    const int64_t span = t->size[i + 1] * t->stride[i + 1];
    if (t->size[i] <= 1 && t->stride[i] < span) t->stride[i] = span;
  }
  Ref p(PyObject_CallMethodNoArgs(o, s_ptr));
  if (!p.p) return false;
  t->ptr = static_cast<char*>(PyLong_AsVoidPtr(p.p));
  return !PyErr_Occurred();
}

bool packed(const Tensor& t, int ndim) {
  int64_t n = 1;
  for (int i = ndim - 1; i >= 0; --i) {
    if (t.stride[i] != n) return false;
    n *= t.size[i];
  }
  return true;
}

// The current device, if it is the tensor's.
bool current(PyObject* first, long* dev, Ref* device) {
  if (reinterpret_cast<PyObject*>(Py_TYPE(first)) != g_tensor) return false;
  Ref d(PyObject_CallMethodNoArgs(first, s_dev));
  if (!d.p) return false;
  *dev = PyLong_AsLong(d.p);
  if (*dev < 0) return false;
  Ref c(PyObject_CallNoArgs(g_get_device));
  if (!c.p || PyLong_AsLong(c.p) != *dev) return false;
  device->p = PyObject_GetAttr(first, s_device);
  return device->p != nullptr;
}

bool stream_of(long dev, cudaStream_t* stream) {
  Ref d(PyLong_FromLong(dev));
  if (!d.p) return false;
  Ref s(PyObject_CallOneArg(g_stream, d.p));
  if (!s.p) return false;
  *stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(s.p));
  return !PyErr_Occurred();
}

PyObject* make_empty(int ndim, const int64_t* size, PyObject* type, PyObject* device) {
  Ref shape(PyTuple_New(ndim));
  if (!shape.p) return nullptr;
  for (int i = 0; i < ndim; ++i) {
    PyObject* v = PyLong_FromLongLong(size[i]);
    if (!v) return nullptr;
    PyTuple_SET_ITEM(shape.p, i, v);
  }
  PyObject* args[3] = {shape.p, type, device};
  return PyObject_Vectorcall(g_empty, args, 1, g_empty_kw);
}

// An output: `given`, or a new packed tensor.  *out gets a reference; false: not plain.
bool output(PyObject* given, long dev, int ndim, const int64_t* size, PyObject* type, PyObject* other, PyObject* device, Tensor* t,
            Ref* out) {
  if (given == Py_None) {
    out->p = make_empty(ndim, size, type, device);
    if (!out->p) return false;
    Ref p(PyObject_CallMethodNoArgs(out->p, s_ptr));
    if (!p.p) return false;
    t->ptr = static_cast<char*>(PyLong_AsVoidPtr(p.p));
    int64_t n = 1;
    for (int i = ndim - 1; i >= 0; --i) t->size[i] = size[i], t->stride[i] = n, n *= size[i];
    return !PyErr_Occurred();
  }
  if (!read(given, dev, ndim, t, type, other)) return false;
  for (int i = 0; i < ndim; ++i)
    if (t->size[i] != size[i]) return false;
  Py_INCREF(given);
  out->p = given;
  return true;
}

// Raises what the C entry reported (an allocation that failed has raised already).
PyObject* refused(int rc) {
  Ref code(PyLong_FromLong(rc));
  if (!code.p) return nullptr;
  Ref r(PyObject_CallOneArg(g_check, code.p));
  if (r.p) PyErr_SetString(PyExc_RuntimeError, "the call failed");
  return nullptr;
}

struct IndexCache {
  Tensor keys, scales;
  int64_t nb, block, entry;
  const float* sc;
  int64_t sc_stride;
  int32_t bs;
};

bool read_index_cache(PyObject* cache, PyObject* scales, int fmt, long dev, IndexCache* c) {
  const bool bf16 = fmt == MLA_CACHE_BF16;
  if (!(bf16 ? read(cache, dev, 3, &c->keys, g_bf16) : read(cache, dev, 3, &c->keys, g_u8, g_i8))) return false;
  const int64_t e = bf16 ? 2 : 1;
  if (c->keys.size[2] != 128 || c->keys.size[1] > INT32_MAX) return false;
  c->nb = c->keys.size[0];
  c->bs = static_cast<int32_t>(c->keys.size[1]);
  c->block = e * c->keys.stride[0];
  c->entry = e * c->keys.stride[1];
  c->sc = nullptr;
  c->sc_stride = 0;
  if (bf16) return scales == Py_None;
  if (!read(scales, dev, 2, &c->scales, g_f32) || c->scales.size[0] != c->nb || c->scales.size[1] != c->bs) return false;
  c->sc = reinterpret_cast<const float*>(c->scales.ptr);
  c->sc_stride = c->scales.stride[0];
  return true;
}

struct Requests {
  int32_t B;
  const int32_t *lens, *cu;
};

bool read_requests(PyObject* seq_lens, PyObject* cu, int64_t T, long dev, Requests* r) {
  Tensor t;
  if (T > INT32_MAX || !read(seq_lens, dev, 1, &t, g_i32) || t.size[0] > INT32_MAX) return false;
  r->B = static_cast<int32_t>(t.size[0]);
  r->lens = reinterpret_cast<const int32_t*>(t.ptr);
  r->cu = nullptr;
  if (cu == Py_None) return T == r->B;
  if (!read(cu, dev, 1, &t, g_i32) || t.size[0] != static_cast<int64_t>(r->B) + 1) return false;
  r->cu = reinterpret_cast<const int32_t*>(t.ptr);
  return true;
}

struct Table {
  const int32_t* ptr;
  int64_t stride, cols;
};

bool read_table(PyObject* table, int64_t rows, long dev, Table* o) {
  Tensor t;
  if (!read(table, dev, 2, &t, g_i32) || t.size[0] < rows) return false;
  o->ptr = reinterpret_cast<const int32_t*>(t.ptr);
  o->cols = t.size[1];
  o->stride = t.stride[0];
  return true;
}

template <class T>
T* as(const Tensor& t) {
  return reinterpret_cast<T*>(t.ptr);
}

// insert(q, k, weights, index_cache, index_scales, slot_mapping, fmt, weight_scale, positions, cos_sin_cache, q_out, w_out)
PyObject* py_insert(PyObject*, PyObject* const* a, Py_ssize_t n) {
  long dev;
  Ref device, q_out, w_out;
  Tensor q, k, w, slots, pos, cs, qo, wo;
  IndexCache c;
  int32_t fmt;
  float scale;
  if (n != 12 || !as_i32(a[6], &fmt) || !as_float(a[7], &scale) || !current(a[0], &dev, &device) ||
      !read(a[0], dev, 3, &q, g_bf16) || !read(a[1], dev, 2, &k, g_bf16) || !read(a[2], dev, 2, &w, g_f32) ||
      !read_index_cache(a[3], a[4], fmt, dev, &c) || !read(a[5], dev, 1, &slots, g_i64))
    return not_plain();
  const int64_t T = q.size[0], H = q.size[1];
  if (T > INT32_MAX || H > INT32_MAX || q.size[2] != 128 || k.size[0] != T || k.size[1] != 128 || w.size[0] != T || w.size[1] != H ||
      slots.size[0] != T)
    return not_plain();
  pos.ptr = cs.ptr = nullptr;
  cs.size[0] = 0;
  if (a[8] != Py_None && (!read(a[8], dev, 1, &pos, g_i64) || pos.size[0] != T)) return not_plain();
  if (a[9] != Py_None && (!read(a[9], dev, 2, &cs, g_f32) || cs.size[1] != 64 || cs.stride[0] != 64)) return not_plain();
  const int64_t qs[3] = {T, H, 128};
  const bool bf16 = fmt == MLA_CACHE_BF16;
  cudaStream_t stream;
  if (!output(a[10], dev, 3, qs, bf16 ? g_bf16 : g_u8, bf16 ? nullptr : g_i8, device.p, &qo, &q_out) || !packed(qo, 3) ||
      !output(a[11], dev, 2, qs, g_f32, nullptr, device.p, &wo, &w_out) || !packed(wo, 2) || !stream_of(dev, &stream))
    return not_plain();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = mla_index_q_cache_insert(q.ptr, q.stride[0], q.stride[1], k.ptr, k.stride[0], as<float>(w), w.stride[0], scale, qo.ptr,
                                as<float>(wo), c.keys.ptr, static_cast<mla_cache_format>(fmt), c.nb, c.block, c.entry,
                                const_cast<float*>(c.sc), c.sc_stride, c.bs, as<int64_t>(slots), as<int64_t>(pos), as<float>(cs),
                                cs.size[0], static_cast<int32_t>(T), static_cast<int32_t>(H), stream);
  Py_END_ALLOW_THREADS
  if (rc) return refused(rc);
  return PyTuple_Pack(2, q_out.p, w_out.p);
}

// gather(index_cache, index_scales, block_table, cu_seq_lens, seq_starts, fmt, num_tokens, dst)
PyObject* py_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  long dev;
  Ref device, dst;
  Tensor cu, starts, d;
  IndexCache c;
  Table tab;
  int32_t fmt;
  int64_t rows[2] = {0, 128};
  if (n != 8 || !as_i32(a[5], &fmt) || !as_i64(a[6], &rows[0]) || rows[0] < 0 || !current(a[0], &dev, &device) ||
      !read_index_cache(a[0], a[1], fmt, dev, &c) || !read(a[3], dev, 1, &cu, g_i32))
    return not_plain();
  const int64_t batch = cu.size[0] - 1;
  if (batch < 0 || batch > INT32_MAX || !read_table(a[2], batch, dev, &tab)) return not_plain();
  starts.ptr = nullptr;
  if (a[4] != Py_None && (!read(a[4], dev, 1, &starts, g_i32) || starts.size[0] < batch)) return not_plain();
  cudaStream_t stream;
  if (!output(a[7], dev, 2, rows, g_bf16, nullptr, device.p, &d, &dst) || !stream_of(dev, &stream)) return not_plain();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = mla_index_gather(c.keys.ptr, static_cast<mla_cache_format>(fmt), c.nb, c.block, c.entry, c.sc, c.sc_stride, c.bs, tab.ptr,
                        tab.stride, tab.cols, as<int32_t>(cu), as<int32_t>(starts), static_cast<int32_t>(batch), rows[0], d.ptr,
                        d.stride[0], stream);
  Py_END_ALLOW_THREADS
  if (rc) return refused(rc);
  return dst.release();
}

// scores(q, weights, index_cache, index_scales, block_table, seq_lens, cu_q_lens, fmt, block_tokens, max_context, scores)
PyObject* py_scores(PyObject*, PyObject* const* a, Py_ssize_t n) {
  long dev;
  Ref device, out;
  Tensor q, w, s;
  IndexCache c;
  Requests r;
  Table tab;
  int32_t fmt, bt;
  int64_t ctx;
  if (n != 11 || !as_i32(a[7], &fmt) || !as_i32(a[8], &bt) || bt < 1 || !as_i64(a[9], &ctx) || ctx < 0 ||
      !current(a[0], &dev, &device) ||
      !(fmt == MLA_CACHE_BF16 ? read(a[0], dev, 3, &q, g_bf16) : read(a[0], dev, 3, &q, g_u8, g_i8)) ||
      !read(a[1], dev, 2, &w, g_f32) || !read_index_cache(a[2], a[3], fmt, dev, &c))
    return not_plain();
  const int64_t T = q.size[0], H = q.size[1], cols = ctx / bt + (ctx % bt ? 1 : 0);
  if (H > INT32_MAX || q.size[2] != 128 || w.size[0] != T || w.size[1] != H || !read_requests(a[5], a[6], T, dev, &r) ||
      !read_table(a[4], r.B, dev, &tab))
    return not_plain();
  const int64_t size[2] = {T, cols};
  if (a[10] == Py_None) {
    if (!output(a[10], dev, 2, size, g_f32, nullptr, device.p, &s, &out)) return not_plain();
  } else {
    if (!read(a[10], dev, 2, &s, g_f32) || s.size[0] != T || s.size[1] < cols) return not_plain();
    Py_INCREF(a[10]);
    out.p = a[10];
  }
  cudaStream_t stream;
  if (!stream_of(dev, &stream)) return not_plain();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = mla_index_scores(q.ptr, q.stride[0], q.stride[1], as<float>(w), w.stride[0], c.keys.ptr, static_cast<mla_cache_format>(fmt),
                        c.nb, c.block, c.entry, c.sc, c.sc_stride, c.bs, tab.ptr, tab.stride, tab.cols, r.lens, r.cu, r.B,
                        static_cast<int32_t>(T), static_cast<int32_t>(H), bt, as<float>(s), s.stride[0], cols, stream);
  Py_END_ALLOW_THREADS
  if (rc) return refused(rc);
  return out.release();
}

// select(scores, seq_lens, topk, cu_q_lens, block_tokens, first, last, block_table, page_size, num_blocks, blocks, slots)
PyObject* py_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  long dev;
  Ref device, blocks, slots;
  Tensor x, b, s;
  Requests r;
  Table tab{nullptr, 0, 0};
  int32_t topk, bt, first, last, page;
  int64_t nb;
  if (n != 12 || !as_i32(a[2], &topk) || topk < 1 || !as_i32(a[4], &bt) || bt < 1 || !as_i32(a[5], &first) || !as_i32(a[6], &last) ||
      !as_i32(a[8], &page) || !as_i64(a[9], &nb) || !current(a[0], &dev, &device) || !read(a[0], dev, 2, &x, g_f32))
    return not_plain();
  const int64_t T = x.size[0], width = x.size[1], per_row = static_cast<int64_t>(topk) * bt;
  if (!read_requests(a[1], a[3], T, dev, &r)) return not_plain();
  const int64_t size[2] = {T, topk}, slot_size[2] = {T, per_row};
  if (!output(a[10], dev, 2, size, g_i32, nullptr, device.p, &b, &blocks)) return not_plain();
  s.ptr = nullptr;
  s.stride[0] = 0;
  if (a[7] != Py_None) {
    if (!read_table(a[7], r.B, dev, &tab) || !output(a[11], dev, 2, slot_size, g_i32, nullptr, device.p, &s, &slots))
      return not_plain();
  } else if (a[11] != Py_None) {
    return not_plain();
  }
  cudaStream_t stream;
  if (!stream_of(dev, &stream)) return not_plain();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = mla_index_select(as<float>(x), x.stride[0], width, r.lens, r.cu, r.B, static_cast<int32_t>(T), bt,
                        topk, first, last, as<int32_t>(b), b.stride[0], as<int32_t>(s), s.stride[0],
                        tab.ptr, tab.stride, tab.cols, page, nb, stream);
  Py_END_ALLOW_THREADS
  if (rc) return refused(rc);
  return PyTuple_Pack(2, blocks.p, slots.p ? slots.p : Py_None);
}

// selected(q, kv_cache, block_table, seq_lens, blocks, cu_q_lens, fmt, softmax_scale, q_scale, k_scale, out, return_lse,
//          workspace, lse)
PyObject* py_selected(PyObject*, PyObject* const* a, Py_ssize_t n) {
  long dev;
  Ref device, out, lse, work;
  Tensor q, kv, blk, o, l, ws;
  Requests r;
  Table tab;
  int32_t fmt;
  float sm, qsc, ksc;
  if (n != 14 || !as_i32(a[6], &fmt) || !as_float(a[7], &sm) || !as_float(a[8], &qsc) || !as_float(a[9], &ksc) ||
      !PyBool_Check(a[11]) || !current(a[0], &dev, &device) ||
      !(fmt == MLA_CACHE_FP8 ? read(a[0], dev, 3, &q, g_u8, g_i8) : read(a[0], dev, 3, &q, g_bf16)) ||
      !read(a[1], dev, 3, &kv, g_u8, g_i8, fmt == MLA_CACHE_BF16 ? g_bf16 : nullptr) || !read(a[4], dev, 2, &blk, g_i32))
    return not_plain();
  const int64_t T = q.size[0], H = q.size[1], topk = blk.size[1], es = kv.type == 2 ? 2 : 1;
  const int64_t entry = fmt == MLA_CACHE_BF16 ? 1152 : fmt == MLA_CACHE_FP8 ? 576 : 656;
  if (H > INT32_MAX || topk > INT32_MAX || kv.size[1] > INT32_MAX || kv.size[2] * es < entry || q.size[2] != 576 || blk.size[0] != T ||
      !read_requests(a[3], a[5], T, dev, &r) || r.B == 0 || !read_table(a[2], r.B, dev, &tab))
    return not_plain();
  const int64_t size[3] = {T, H, 512};
  if (a[10] == Py_None) {
    if (!output(a[10], dev, 3, size, g_bf16, nullptr, device.p, &o, &out)) return not_plain();
  } else {
    if (!read(a[10], dev, 3, &o, g_bf16) || o.size[0] != T || o.size[1] != H || o.size[2] < 512) return not_plain();
    Py_INCREF(a[10]);
    out.p = a[10];
  }
  l.ptr = nullptr;
  if (a[13] != Py_None || a[11] == Py_True) {
    if (!output(a[13], dev, 2, size, g_f32, nullptr, device.p, &l, &lse) || !packed(l, 2)) return not_plain();
  }
  const int32_t bs = static_cast<int32_t>(kv.size[1]);
  int64_t bytes = 0;
  if (a[12] == Py_None) {
    bytes = static_cast<int64_t>(mla_selected_decode_workspace_size(static_cast<mla_cache_format>(fmt), static_cast<int32_t>(T),
                                                                    static_cast<int32_t>(topk), bs, static_cast<int32_t>(H), 0));
    if (!output(a[12], dev, 1, &bytes, g_u8, nullptr, device.p, &ws, &work)) return not_plain();
  } else {
    if (!read(a[12], dev, 1, &ws, g_u8, g_i8)) return not_plain();
    bytes = ws.size[0];
  }
  cudaStream_t stream;
  if (!stream_of(dev, &stream)) return not_plain();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = mla_selected_decode(q.ptr, q.stride[0], q.stride[1], kv.ptr, static_cast<mla_cache_format>(fmt), kv.size[0], es * kv.stride[0],
                           es * kv.stride[1], bs, tab.ptr, tab.stride, tab.cols, r.lens, r.cu, as<int32_t>(blk),
                           blk.stride[0], static_cast<int32_t>(topk), r.B, static_cast<int32_t>(T),
                           static_cast<int32_t>(H), sm, qsc, ksc, o.ptr, o.stride[0], o.stride[1], as<float>(l), ws.ptr,
                           static_cast<size_t>(bytes), stream);
  Py_END_ALLOW_THREADS
  if (rc) return refused(rc);
  return PyTuple_Pack(2, out.p, lse.p ? lse.p : Py_None);
}

// init(Tensor, empty, current_device, current_raw_stream, check, bf16, uint8, int8, float32, int32, int64)
PyObject* py_init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  PyObject** kept[11] = {&g_tensor, &g_empty, &g_get_device, &g_stream, &g_check, &g_bf16, &g_u8, &g_i8, &g_f32, &g_i32, &g_i64};
  if (n != 11) {
    PyErr_SetString(PyExc_TypeError, "init takes 11 arguments");
    return nullptr;
  }
  for (int i = 0; i < 11; ++i) {
    Py_INCREF(a[i]);
    Py_XSETREF(*kept[i], a[i]);
  }
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {
    {"init", fast(py_init), METH_FASTCALL, nullptr},       {"insert", fast(py_insert), METH_FASTCALL, nullptr},
    {"gather", fast(py_gather), METH_FASTCALL, nullptr},   {"scores", fast(py_scores), METH_FASTCALL, nullptr},
    {"select", fast(py_select), METH_FASTCALL, nullptr},   {"selected", fast(py_selected), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "mla_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mla_marshal() {
  PyObject** names[6] = {&s_dtype, &s_shape, &s_stride, &s_ptr, &s_dev, &s_device};
  const char* text[6] = {"dtype", "shape", "stride", "data_ptr", "get_device", "device"};
  for (int i = 0; i < 6; ++i)
    if (!(*names[i] = PyUnicode_InternFromString(text[i]))) return nullptr;
  if (!(g_empty_kw = Py_BuildValue("(ss)", "dtype", "device"))) return nullptr;
  return PyModule_Create(&g_module);
}
