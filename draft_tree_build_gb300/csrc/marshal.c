/* The short way from Python to the paged cache's entry points.
 *
 * A call of a few microseconds on the GPU should not take ten on the host: this
 * module checks a call's tensors and calls the library without ctypes and with
 * no Python code in between (attention 10.2 -> 7.0 us, of which the launch is
 * 2.5).  It accepts what is plainly right and nothing else: every function
 * returns the library's return code, or None, with nothing called, where any
 * argument is not what the call takes; the binding then checks again, in
 * Python, and says what is wrong.
 *
 * A tensor is looked at through its Python attributes, so that nothing here
 * depends on how torch is built.
 *
 * The library runs without the interpreter's lock, as it does through ctypes: a
 * launch waits where the stream's queue is full, and other threads (a host
 * callback that the queue waits for among them) must get on meanwhile.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "bastion_cache.h"

typedef __typeof__(&bastion_paged_append) append_fn;
typedef __typeof__(&bastion_paged_append_held) append_held_fn;
typedef __typeof__(&bastion_paged_attention) attention_fn;
typedef __typeof__(&bastion_paged_evict) evict_fn;
typedef __typeof__(&bastion_paged_plan) plan_fn;
typedef __typeof__(&bastion_paged_plan_offset) plan_offset_fn;
typedef __typeof__(&bastion_qk_norm_rope) rope_fn;
typedef __typeof__(&bastion_paged_prefix_attention) prefix_fn;

static append_fn f_append;
static append_held_fn f_append_held;
static attention_fn f_attention;
static evict_fn f_evict;
static plan_fn f_plan;
static plan_offset_fn f_plan_offset;
static rope_fn f_rope;
static prefix_fn f_prefix;
static PyObject *dt_i64, *dt_f64;
static PyObject *dt_bf16, *dt_f16, *dt_f32, *dt_i32, *dt_u8, *fn_device, *fn_stream;
static PyObject *s_dtype, *s_shape, *s_stride, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_cuda_stream;

typedef struct {
  void *ptr;
  PyObject *dtype; /* borrowed: torch's dtypes live as long as torch */
  int dim;
  long dev;
  int64_t shape[4], stride[4];
} tensor;

/* Up to four integers of a tuple; -1: it is none, or longer. */
static int ints(PyObject *t, int64_t *to) {
  if (!t || !PyTuple_Check(t) || PyTuple_GET_SIZE(t) > 4) return -1;
  const int n = (int)PyTuple_GET_SIZE(t);
  for (int i = 0; i < n; ++i) {
    to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    if (to[i] == -1 && PyErr_Occurred()) return -1;
  }
  return n;
}

/* Type, shape, device and address of a tensor; 0: it is none. */
static int look(PyObject *o, tensor *t) {
  PyObject *x = PyObject_GetAttr(o, s_dtype);
  if (!x) return 0;
  t->dtype = x;
  Py_DECREF(x);
  x = PyObject_GetAttr(o, s_shape);
  t->dim = ints(x, t->shape);
  Py_XDECREF(x);
  if (t->dim < 0) return 0;
  x = PyObject_CallMethodNoArgs(o, s_get_device);
  if (!x) return 0;
  t->dev = PyLong_AsLong(x);
  Py_DECREF(x);
  x = PyObject_CallMethodNoArgs(o, s_data_ptr);
  if (!x) return 0;
  t->ptr = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return !PyErr_Occurred();
}

/* look, and the strides. */
static int look_strided(PyObject *o, tensor *t) {
  if (!look(o, t)) return 0;
  PyObject *x = PyObject_CallMethodNoArgs(o, s_stride);
  const int n = ints(x, t->stride);
  Py_XDECREF(x);
  return n == t->dim;
}

/* The address of a contiguous tensor of that device, type and shape. */
static int contiguous(PyObject *o, long dev, PyObject *dtype, int dim, const int64_t *shape, void **ptr) {
  tensor t;
  if (!look(o, &t) || t.dtype != dtype || t.dev != dev || t.dim != dim) return 0;
  for (int i = 0; i < dim; ++i)
    if (t.shape[i] != shape[i]) return 0;
  PyObject *x = PyObject_CallMethodNoArgs(o, s_is_contiguous);
  if (!x) return 0;
  const int ok = x == Py_True;
  Py_DECREF(x);
  *ptr = t.ptr;
  return ok;
}

/* The same, or None: a null address. */
static int contiguous_or_none(PyObject *o, long dev, PyObject *dtype, int dim, const int64_t *shape, void **ptr) {
  *ptr = NULL;
  return o == Py_None || contiguous(o, dev, dtype, dim, shape, ptr);
}

/* The cache of a call, and its device, which is the current one. */
static int cache_of(PyObject *k, PyObject *v, PyObject *table, bastion_paged_cache *c, long *dev, PyObject **dtype) {
  tensor tk, tv, tt;
  if (!look_strided(k, &tk) || !look_strided(v, &tv) || !look(table, &tt)) return 0;
  if (tk.dim != 4 || tv.dim != 4 || tt.dim != 2 || tk.dtype != tv.dtype || tk.dev != tt.dev || tv.dev != tt.dev || tt.dev < 0)
    return 0;
  for (int i = 0; i < 4; ++i)
    if (tk.shape[i] != tv.shape[i] || (tk.shape[i] != 1 && tk.stride[i] != tv.stride[i])) return 0;
  if (tk.stride[3] != 1 || (tk.dtype != dt_bf16 && tk.dtype != dt_f16)) return 0;
  void *at;
  if (!contiguous(table, tt.dev, dt_i32, 2, tt.shape, &at)) return 0;
  for (int i = 1; i < 4; ++i)
    if (tk.shape[i] > INT32_MAX) return 0;
  if (tt.shape[0] > INT32_MAX || tt.shape[1] > INT32_MAX) return 0;
  PyObject *x = PyObject_CallNoArgs(fn_device);
  if (!x) return 0;
  const long current = PyLong_AsLong(x);
  Py_DECREF(x);
  if (current != tt.dev) return 0;
  *dev = tt.dev;
  *dtype = tk.dtype;
  c->k_pool = tk.ptr;
  c->v_pool = tv.ptr;
  c->n_pages = tk.shape[0];
  c->stride_page = tk.stride[0];
  c->stride_slot = tk.stride[1];
  c->stride_head = tk.stride[2];
  c->page_table = at;
  c->dtype = tk.dtype == dt_bf16 ? BASTION_BF16 : BASTION_F16;
  c->B = (int32_t)tt.shape[0];
  c->Hkv = (int32_t)tk.shape[2];
  c->D = (int32_t)tk.shape[3];
  c->page_size = (int32_t)tk.shape[1];
  c->max_pages = (int32_t)tt.shape[1];
  return 1;
}

static int workspace_of(PyObject *o, long dev, void **ptr, size_t *bytes) {
  tensor t;
  if (!look(o, &t) || t.dim != 1) return 0;
  *bytes = (size_t)t.shape[0];
  return contiguous(o, dev, dt_u8, 1, t.shape, ptr);
}

static int stream_of(PyObject *o, PyObject *dev, bastion_stream_t *stream) {
  PyObject *x = o == Py_None ? PyObject_CallOneArg(fn_stream, dev) : PyObject_GetAttr(o, s_cuda_stream);
  if (!x) return 0;
  *stream = (bastion_stream_t)PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return !PyErr_Occurred();
}

static int stream_on(PyObject *o, long dev, bastion_stream_t *stream) {
  PyObject *d = PyLong_FromLong(dev);
  const int ok = d && stream_of(o, d, stream);
  Py_XDECREF(d);
  return ok;
}

static int int32_of(PyObject *o, int *to) {
  if (!PyLong_Check(o)) return 0;
  const long x = PyLong_AsLong(o);
  *to = (int)x;
  return x >= INT32_MIN && x <= INT32_MAX && !PyErr_Occurred();
}

static PyObject *declined(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

/* k_new, v_new, k_pool, v_pool, page_table, seq_len, seq_len_out, workspace, status, rows, n_new, acc, pos, n_seen,
 * n_seen_out, stream, and held or None, which may be left out */
static PyObject *append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  bastion_paged_cache c;
  tensor k, v, rows;
  PyObject *dtype;
  long dev;
  void *len, *len_out, *st, *n_new, *seen, *seen_out, *acc, *pos, *ws, *held = NULL;
  size_t bytes;
  bastion_stream_t stream;
  if ((n != 16 && n != 17) || !f_append || (n == 17 && !f_append_held) || !cache_of(a[2], a[3], a[4], &c, &dev, &dtype)) return declined();
  if (!look_strided(a[0], &k) || !look_strided(a[1], &v) || k.dim != 4 || v.dim != 4 || k.dtype != dtype ||
      v.dtype != dtype || k.dev != dev || v.dev != dev || k.stride[3] != 1)
    return declined();
  for (int i = 0; i < 4; ++i)
    if (k.shape[i] != v.shape[i] || (k.shape[i] != 1 && k.stride[i] != v.stride[i])) return declined();
  if (k.shape[0] != c.B || k.shape[2] != c.Hkv || k.shape[3] != c.D || k.shape[1] > INT32_MAX) return declined();
  int64_t m = k.shape[1];
  rows.ptr = NULL;
  if (a[9] != Py_None) {
    if (!look(a[9], &rows) || rows.dim != 2 || rows.shape[0] != c.B || rows.shape[1] > INT32_MAX ||
        !contiguous(a[9], dev, dt_i32, 2, rows.shape, &rows.ptr))
      return declined();
    m = rows.shape[1];
  }
  const int64_t B[1] = {c.B}, slots[3] = {c.B, c.Hkv, (int64_t)c.max_pages * c.page_size};
  if (!contiguous(a[5], dev, dt_i32, 1, B, &len) || !contiguous(a[6], dev, dt_i32, 1, B, &len_out) ||
      !workspace_of(a[7], dev, &ws, &bytes) || !contiguous(a[8], dev, dt_i32, 1, B, &st) ||
      !contiguous_or_none(a[10], dev, dt_i32, 1, B, &n_new) ||
      !contiguous_or_none(a[11], dev, dt_f32, 3, slots, &acc) || !contiguous_or_none(a[12], dev, dt_i32, 3, slots, &pos) ||
      !contiguous_or_none(a[13], dev, dt_i32, 1, B, &seen) || !contiguous_or_none(a[14], dev, dt_i32, 1, B, &seen_out) ||
      !stream_on(a[15], dev, &stream) || (n == 17 && !contiguous_or_none(a[16], dev, dt_i32, 1, B, &held)))
    return declined();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = held ? f_append_held(&c, held, k.ptr, v.ptr, (int)k.shape[1], k.stride[0], k.stride[1], k.stride[2], rows.ptr, (int)m,
                            n_new, len, len_out, seen, seen_out, acc, pos, ws, bytes, st, stream)
            : f_append(&c, k.ptr, v.ptr, (int)k.shape[1], k.stride[0], k.stride[1], k.stride[2], rows.ptr, (int)m, n_new, len,
                       len_out, seen, seen_out, acc, pos, ws, bytes, st, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* q, k_pool, v_pool, page_table, seq_len, scale, out, workspace, status, lse, acc, acc_out, stream */
static PyObject *attention(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  bastion_paged_cache c;
  tensor q;
  PyObject *dtype;
  long dev;
  void *len, *out, *ws, *st, *lse, *acc, *acc_out;
  size_t bytes;
  bastion_stream_t stream;
  if (n != 13 || !f_attention || !cache_of(a[1], a[2], a[3], &c, &dev, &dtype)) return declined();
  if (!look_strided(a[0], &q) || q.dim != 3 || q.dtype != dtype || q.dev != dev || q.shape[0] != c.B ||
      q.shape[2] != c.D || q.shape[1] > INT32_MAX || q.stride[2] != 1 || (q.shape[1] > 1 && q.stride[1] != c.D))
    return declined();
  const double scale = PyFloat_AsDouble(a[5]);
  if (scale == -1.0 && PyErr_Occurred()) return declined();
  const int64_t B[1] = {c.B}, heads[2] = {c.B, q.shape[1]},
                slots[3] = {c.B, c.Hkv, (int64_t)c.max_pages * c.page_size};
  if (!contiguous(a[4], dev, dt_i32, 1, B, &len) || !contiguous(a[6], dev, dtype, 3, q.shape, &out) ||
      !workspace_of(a[7], dev, &ws, &bytes) || !contiguous(a[8], dev, dt_i32, 1, B, &st) ||
      !contiguous_or_none(a[9], dev, dt_f32, 2, heads, &lse) ||
      !contiguous_or_none(a[10], dev, dt_f32, 3, slots, &acc) ||
      !contiguous_or_none(a[11], dev, dt_f32, 3, slots, &acc_out) || !stream_on(a[12], dev, &stream))
    return declined();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f_attention(&c, q.ptr, (int)q.shape[1], q.stride[0], len, (float)scale, out, lse, acc, acc_out, ws, bytes, st,
                   stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* k_pool, v_pool, page_table, seq_len, n_seen, acc, pos, budget, n_sink, n_recent, seq_len_out, acc_out, pos_out,
 * workspace, status, stream */
static PyObject *evict(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  bastion_paged_cache c;
  PyObject *dtype;
  long dev;
  void *len, *seen, *acc, *pos, *len_out, *acc_out, *pos_out, *ws, *st;
  int budget, sink, recent;
  size_t bytes;
  bastion_stream_t stream;
  if (n != 16 || !f_evict || !cache_of(a[0], a[1], a[2], &c, &dev, &dtype)) return declined();
  const int64_t B[1] = {c.B}, slots[3] = {c.B, c.Hkv, (int64_t)c.max_pages * c.page_size};
  if (!contiguous(a[3], dev, dt_i32, 1, B, &len) || !contiguous(a[4], dev, dt_i32, 1, B, &seen) ||
      !contiguous(a[5], dev, dt_f32, 3, slots, &acc) || !contiguous(a[6], dev, dt_i32, 3, slots, &pos) ||
      !int32_of(a[7], &budget) || !int32_of(a[8], &sink) || !int32_of(a[9], &recent) ||
      !contiguous(a[10], dev, dt_i32, 1, B, &len_out) || !contiguous(a[11], dev, dt_f32, 3, slots, &acc_out) ||
      !contiguous(a[12], dev, dt_i32, 3, slots, &pos_out) || !workspace_of(a[13], dev, &ws, &bytes) ||
      !contiguous(a[14], dev, dt_i32, 1, B, &st) || !stream_on(a[15], dev, &stream))
    return declined();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f_evict(&c, len, seen, acc, pos, budget, sink, recent, len_out, acc_out, pos_out, ws, bytes, st, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* Whether dev is a CUDA device, and the current one. */
static int is_current(long dev) {
  if (dev < 0) return 0;
  PyObject *x = PyObject_CallNoArgs(fn_device);
  if (!x) return 0;
  const long current = PyLong_AsLong(x);
  Py_DECREF(x);
  return current == dev;
}

/* page_table, page_size, seq_len, m, held, held_out, free_pages, n_free, n_free_out, slots, pos, workspace, status, n_new,
 * row_start, seq_len_out, trim, stream, and pos_offset or None, which may be left out */
static PyObject *plan(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  tensor table, stack, slots;
  void *at, *len, *held, *held_out, *pages, *left, *left_out, *slot, *pos, *ws, *st, *n_new, *start, *len_out, *offset = NULL;
  int page, m;
  size_t bytes;
  bastion_stream_t stream;
  if ((n != 18 && n != 19) || !f_plan || (n == 19 && !f_plan_offset) || !look(a[0], &table) || table.dim != 2 || !is_current(table.dev)) return declined();
  const long dev = table.dev;
  if (!contiguous(a[0], dev, dt_i32, 2, table.shape, &at) || table.shape[0] > INT32_MAX - 1 || table.shape[1] > INT32_MAX ||
      !int32_of(a[1], &page) || !int32_of(a[3], &m) || !look(a[6], &stack) || stack.dim != 1 || !look(a[9], &slots) ||
      slots.dim < 1)
    return declined();
  int64_t rows = 1;
  for (int i = 0; i < slots.dim; ++i) {
    if (slots.shape[i] > INT32_MAX || rows > INT32_MAX) return declined();
    rows *= slots.shape[i];
  }
  const int64_t B[1] = {table.shape[0]}, more[1] = {table.shape[0] + 1}, one[1] = {1};
  const int trim = PyObject_IsTrue(a[16]);
  if (trim < 0 || !contiguous(a[2], dev, dt_i32, 1, B, &len) || !contiguous(a[4], dev, dt_i32, 1, B, &held) ||
      !contiguous(a[5], dev, dt_i32, 1, B, &held_out) || !contiguous(a[6], dev, dt_i32, 1, stack.shape, &pages) ||
      !contiguous(a[7], dev, dt_i32, 1, one, &left) || !contiguous(a[8], dev, dt_i32, 1, one, &left_out) ||
      !contiguous(a[9], dev, dt_i64, slots.dim, slots.shape, &slot) ||
      !contiguous(a[10], dev, dt_i32, slots.dim, slots.shape, &pos) || !workspace_of(a[11], dev, &ws, &bytes) ||
      !contiguous(a[12], dev, dt_i32, 1, B, &st) || !contiguous_or_none(a[13], dev, dt_i32, 1, B, &n_new) ||
      !contiguous_or_none(a[14], dev, dt_i32, 1, more, &start) || !contiguous_or_none(a[15], dev, dt_i32, 1, B, &len_out) ||
      !stream_on(a[17], dev, &stream) || (n == 19 && !contiguous_or_none(a[18], dev, dt_i32, 1, B, &offset)))
    return declined();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = offset ? f_plan_offset(at, (int)table.shape[0], (int)table.shape[1], page, stack.shape[0], len, n_new, m, len_out, held,
                              held_out, pages, left, left_out, trim, slot, pos, rows, start, offset, ws, bytes, st, stream)
              : f_plan(at, (int)table.shape[0], (int)table.shape[1], page, stack.shape[0], len, n_new, m, len_out, held, held_out,
                       pages, left, left_out, trim, slot, pos, rows, start, ws, bytes, st, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* A token-by-token array [T, H, D] of the type on the device, or None: a null address. */
static int heads_of(PyObject *o, long dev, PyObject *dtype, int64_t T, int64_t H, int64_t D, tensor *t) {
  t->ptr = NULL;
  t->stride[0] = t->stride[1] = 0;
  if (o == Py_None) return 1;
  return look_strided(o, t) && t->dim == 3 && t->dtype == dtype && t->dev == dev && t->shape[0] == T && t->shape[1] == H &&
         t->shape[2] == D && t->stride[2] == 1;
}

/* q, k, pos, inv_freq, q_out, status, k_out, q_weight, k_weight, eps, interleaved, factor, v, k_pool, v_pool, slots,
 * stream */
static PyObject *rope(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  bastion_paged_cache c;
  tensor q, k, v, q_out, k_out, freq, tk, tv;
  void *pos, *at = NULL, *st, *qw, *kw, *slots;
  bastion_stream_t stream;
  if (n != 17 || !f_rope || !look_strided(a[0], &q) || !look(a[1], &k) || q.dim != 3 || k.dim != 3 || q.stride[2] != 1 ||
      !is_current(q.dev) || (q.dtype != dt_bf16 && q.dtype != dt_f16))
    return declined();
  const long dev = q.dev;
  const int64_t T = q.shape[0], Hq = q.shape[1], D = q.shape[2], Hkv = k.shape[1];
  if (T > INT32_MAX || Hq > INT32_MAX || D > INT32_MAX || Hkv > INT32_MAX || !heads_of(a[1], dev, q.dtype, T, Hkv, D, &k) ||
      !heads_of(a[12], dev, q.dtype, T, Hkv, D, &v) || !heads_of(a[4], dev, q.dtype, T, Hq, D, &q_out) ||
      !heads_of(a[6], dev, q.dtype, T, Hkv, D, &k_out))
    return declined();
  const double eps = PyFloat_AsDouble(a[9]), factor = PyFloat_AsDouble(a[11]);
  const int inter = PyObject_IsTrue(a[10]);
  if (PyErr_Occurred() || inter < 0) return declined();
  int rot = 0;
  if (a[3] != Py_None) {
    if (!look(a[3], &freq) || freq.dim != 1 || freq.shape[0] > 65536 || !contiguous(a[3], dev, dt_f64, 1, freq.shape, &at))
      return declined();
    rot = 2 * (int)freq.shape[0];
  }
  const int64_t tokens[1] = {T}, one[1] = {1}, width[1] = {D};
  if (!contiguous(a[2], dev, dt_i32, 1, tokens, &pos) || !contiguous(a[5], dev, dt_i32, 1, one, &st) ||
      !contiguous_or_none(a[7], dev, q.dtype, 1, width, &qw) || !contiguous_or_none(a[8], dev, q.dtype, 1, width, &kw) ||
      !contiguous_or_none(a[15], dev, dt_i64, 1, tokens, &slots))
    return declined();
  const int store = a[13] != Py_None;
  if (store != (a[14] != Py_None)) return declined();
  if (store) {
    if (!look_strided(a[13], &tk) || !look_strided(a[14], &tv) || tk.dim != 4 || tv.dim != 4 || tk.dtype != q.dtype ||
        tv.dtype != q.dtype || tk.dev != dev || tv.dev != dev || tk.stride[3] != 1)
      return declined();
    for (int i = 0; i < 4; ++i)
      if (tk.shape[i] != tv.shape[i] || (tk.shape[i] != 1 && tk.stride[i] != tv.stride[i]) || (i > 0 && tk.shape[i] > INT32_MAX))
        return declined();
    c.k_pool = tk.ptr;
    c.v_pool = tv.ptr;
    c.n_pages = tk.shape[0];
    c.stride_page = tk.stride[0];
    c.stride_slot = tk.stride[1];
    c.stride_head = tk.stride[2];
    c.page_table = st; /* not read: any address of the right alignment serves */
    c.dtype = tk.dtype == dt_bf16 ? BASTION_BF16 : BASTION_F16;
    c.B = 1;
    c.Hkv = (int32_t)tk.shape[2];
    c.D = (int32_t)tk.shape[3];
    c.page_size = (int32_t)tk.shape[1];
    c.max_pages = 1;
  }
  if (!stream_on(a[16], dev, &stream)) return declined();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f_rope(q.dtype == dt_bf16 ? BASTION_BF16 : BASTION_F16, (int)T, (int)Hq, (int)Hkv, (int)D, q.ptr, q.stride[0],
              q.stride[1], k.ptr, k.stride[0], k.stride[1], v.ptr, v.stride[0], v.stride[1], qw, kw, (float)eps, pos, at, rot,
              inter, (float)factor, q_out.ptr, q_out.stride[0], q_out.stride[1], k_out.ptr, k_out.stride[0], k_out.stride[1],
              store ? &c : NULL, slots, st, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* q, k_pool, v_pool, page_table, seq_len, prefix_table, prefix_len, group_start, scale, out, workspace, status, lse,
 * stream */
static PyObject *prefix(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  bastion_paged_cache c;
  tensor q, table;
  PyObject *dtype;
  long dev;
  void *len, *at, *pre_len, *start, *out, *ws, *st, *lse;
  size_t bytes;
  bastion_stream_t stream;
  if (n != 14 || !f_prefix || !cache_of(a[1], a[2], a[3], &c, &dev, &dtype)) return declined();
  if (!look_strided(a[0], &q) || q.dim != 3 || q.dtype != dtype || q.dev != dev || q.shape[0] != c.B ||
      q.shape[2] != c.D || q.shape[1] > INT32_MAX || q.stride[2] != 1 || (q.shape[1] > 1 && q.stride[1] != c.D))
    return declined();
  const double scale = PyFloat_AsDouble(a[8]);
  if (scale == -1.0 && PyErr_Occurred()) return declined();
  if (!look(a[5], &table) || table.dim != 2 || table.shape[0] > INT32_MAX - 1 || table.shape[1] > INT32_MAX) return declined();
  const int64_t B[1] = {c.B}, heads[2] = {c.B, q.shape[1]}, groups[1] = {table.shape[0]}, more[1] = {table.shape[0] + 1};
  if (!contiguous(a[4], dev, dt_i32, 1, B, &len) || !contiguous(a[5], dev, dt_i32, 2, table.shape, &at) ||
      !contiguous(a[6], dev, dt_i32, 1, groups, &pre_len) || !contiguous(a[7], dev, dt_i32, 1, more, &start) ||
      !contiguous(a[9], dev, dtype, 3, q.shape, &out) || !workspace_of(a[10], dev, &ws, &bytes) ||
      !contiguous(a[11], dev, dt_i32, 1, B, &st) || !contiguous_or_none(a[12], dev, dt_f32, 2, heads, &lse) ||
      !stream_on(a[13], dev, &stream))
    return declined();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f_prefix(&c, at, (int)table.shape[1], pre_len, start, (int)table.shape[0], q.ptr, (int)q.shape[1], q.stride[0], len,
                (float)scale, out, lse, ws, bytes, st, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* int64, float64, and the addresses of the page plan, the norm and rotation and the shared-prefix attention */
static PyObject *init_layer(PyObject *self, PyObject *args) {
  (void)self;
  PyObject *i64, *f64;
  unsigned long long f[3];
  if (!PyArg_ParseTuple(args, "OOKKK", &i64, &f64, &f[0], &f[1], &f[2])) return NULL;
  Py_INCREF(i64);
  Py_XSETREF(dt_i64, i64);
  Py_INCREF(f64);
  Py_XSETREF(dt_f64, f64);
  f_plan = (plan_fn)(uintptr_t)f[0];
  f_rope = (rope_fn)(uintptr_t)f[1];
  f_prefix = (prefix_fn)(uintptr_t)f[2];
  Py_RETURN_NONE;
}

/* The address of the append into held pages. */
static PyObject *init_held(PyObject *self, PyObject *args) {
  (void)self;
  unsigned long long f;
  if (!PyArg_ParseTuple(args, "K", &f)) return NULL;
  f_append_held = (append_held_fn)(uintptr_t)f;
  Py_RETURN_NONE;
}

/* The address of the page plan whose positions begin at offsets. */
static PyObject *init_offset(PyObject *self, PyObject *args) {
  (void)self;
  unsigned long long f;
  if (!PyArg_ParseTuple(args, "K", &f)) return NULL;
  f_plan_offset = (plan_offset_fn)(uintptr_t)f;
  Py_RETURN_NONE;
}

/* bfloat16, float16, float32, int32, uint8, current device, raw stream of a device, and the addresses of the
 * library's three functions */
static PyObject *init(PyObject *self, PyObject *args) {
  (void)self;
  PyObject *o[7];
  unsigned long long f[3];
  if (!PyArg_ParseTuple(args, "OOOOOOOKKK", &o[0], &o[1], &o[2], &o[3], &o[4], &o[5], &o[6], &f[0], &f[1], &f[2]))
    return NULL;
  PyObject **to[7] = {&dt_bf16, &dt_f16, &dt_f32, &dt_i32, &dt_u8, &fn_device, &fn_stream};
  for (int i = 0; i < 7; ++i) {
    Py_INCREF(o[i]);
    Py_XSETREF(*to[i], o[i]);
  }
  f_append = (append_fn)(uintptr_t)f[0];
  f_attention = (attention_fn)(uintptr_t)f[1];
  f_evict = (evict_fn)(uintptr_t)f[2];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"init", init, METH_VARARGS, NULL},
                                {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, NULL},
                                {"attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, NULL},
                                {"evict", (PyCFunction)(void (*)(void))evict, METH_FASTCALL, NULL},
                                {"init_layer", init_layer, METH_VARARGS, NULL},
                                {"init_held", init_held, METH_VARARGS, NULL},
                                {"init_offset", init_offset, METH_VARARGS, NULL},
                                {"plan", (PyCFunction)(void (*)(void))plan, METH_FASTCALL, NULL},
                                {"rope", (PyCFunction)(void (*)(void))rope, METH_FASTCALL, NULL},
                                {"prefix", (PyCFunction)(void (*)(void))prefix, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "bastion_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_bastion_marshal(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (!s_dtype || !s_shape || !s_stride || !s_get_device || !s_is_contiguous || !s_data_ptr || !s_cuda_stream)
    return NULL;
  return PyModule_Create(&module);
}
