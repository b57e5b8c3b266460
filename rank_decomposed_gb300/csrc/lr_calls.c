/* Argument marshalling of the calls over a context, as a CPython extension.
 *
 * These calls sit in a decode step whose kernels take a few microseconds, and
 * reading thirty properties of ten tensors from Python and converting them by
 * ctypes took most of a call (one token's rotation: 9.6 us, 3.4 of them the
 * library's launch; from here 5.1, the question where each tensor lies among
 * them, 50 ns each).  Each property is read once, checked, and
 * put into the structures of lr.h.  Tensors are read by their Python attributes
 * alone, so the extension knows no version of torch.  It holds no state but the
 * functions and types given to init().
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <math.h>
#include <stdint.h>
#include <string.h>

#include "lr.h"

typedef lr_status (*rope_fn)(const void*, int64_t, int32_t, const void*, int64_t, int32_t, lr_dtype, int64_t,
                             const int32_t*, const int32_t*, const lr_head_map*, void*, int64_t, void*, int64_t,
                             int32_t*, lr_stream);
typedef lr_status (*append_fn)(const void*, int64_t, const void*, int64_t, const void*, int64_t, int32_t, lr_dtype,
                               int64_t, const int32_t*, const int32_t*, const int32_t*, const lr_head_map*,
                               const lr_kv_cache*, void*, int64_t, int32_t*, lr_stream);
typedef lr_status (*attention_fn)(const void*, int64_t, void*, int64_t, lr_dtype, int64_t, const lr_attn_desc*, void*,
                                  size_t, int32_t*, lr_stream);

static rope_fn g_rope;
static append_fn g_append;
static attention_fn g_attention;
static PyObject *t_bf16, *t_f32, *t_i32; /* torch's dtypes */

/* Interned names. */
static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_is_contiguous, *s_nbytes, *s_head_dim, *s_norm, *s_eps,
    *s_q_gain, *s_k_gain, *s_rot_dim, *s_rot_style, *s_cos_sin, *s_k_pool, *s_v_pool, *s_n_kv_heads, *s_block_rows,
    *s_cache, *s_heads, *s_pos, *s_rows, *s_prefix_blocks, *s_prefix_len, *s_block_table, *s_lengths, *s_q_start,
    *s_max_q, *s_scale, *s_n_active, *s_is_cuda;

typedef struct {
  void* p;
  int64_t ld, rows, cols;
} Mat;

static int fail(PyObject* type, const char* fmt, const char* name) {
  PyErr_Format(type, fmt, name);
  return -1;
}

static int attr_i64(PyObject* o, PyObject* name, int64_t* out) {
  PyObject* v = PyObject_GetAttr(o, name);
  if (v == NULL) return -1;
  *out = PyLong_AsLongLong(v);
  Py_DECREF(v);
  return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int to_i32(int64_t v, const char* name, int32_t* out) {
  if (v < INT32_MIN || v > INT32_MAX) return fail(PyExc_OverflowError, "%s does not fit 32 bits", name);
  *out = (int32_t)v;
  return 0;
}

static int attr_i32(PyObject* o, PyObject* name, int32_t* out) {
  int64_t v;
  if (attr_i64(o, name, &v) < 0) return -1;
  return to_i32(v, PyUnicode_AsUTF8(name), out);
}

static int arg_i64(PyObject* v, int64_t* out) {
  *out = PyLong_AsLongLong(v);
  return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

/* The first tensor of the present call that is not on the GPU.  Calls without
 * rows touch no tensor, and the structures' sizes can be asked for without a
 * GPU; a launch refuses it, since the kernels would follow a host address. */
static _Thread_local const char* host_tensor;

static int on_gpu(int64_t rows) {
  if (rows <= 0 || host_tensor == NULL) return 0;
  return fail(PyExc_TypeError, "%s must be on the GPU", host_tensor);
}

/* Address of a tensor; None is NULL. */
static int address(PyObject* t, const char* name, void** out) {
  *out = NULL;
  if (t == Py_None) return 0;
  PyObject* dev = PyObject_GetAttr(t, s_is_cuda);
  if (dev == NULL) return -1;
  Py_DECREF(dev); /* a truth value */
  if (dev != Py_True && host_tensor == NULL) host_tensor = name;
  PyObject* v = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (v == NULL) return -1;
  const unsigned long long a = PyLong_AsUnsignedLongLong(v);
  Py_DECREF(v);
  if (a == (unsigned long long)-1 && PyErr_Occurred()) return -1;
  *out = (void*)(uintptr_t)a;
  return 0;
}

static PyObject* dtype_of(PyObject* t) { /* borrowed: torch keeps its dtypes */
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  Py_XDECREF(d);
  return d;
}

static int has_dtype(PyObject* t, const char* name, PyObject* want) {
  PyObject* d = dtype_of(t);
  if (d == NULL) return -1;
  if (d != want) {
    PyErr_Format(PyExc_TypeError, "%s must be %S", name, want);
    return -1;
  }
  return 0;
}

/* Code of a tensor of heads. */
static int code_of(PyObject* t, lr_dtype* code, PyObject** type) {
  PyObject* d = dtype_of(t);
  if (d == NULL) return -1;
  if (d != t_bf16 && d != t_f32) {
    PyErr_SetString(PyExc_TypeError, "a tensor of heads must be bfloat16 or float32");
    return -1;
  }
  *code = d == t_bf16 ? LR_BF16 : LR_F32;
  if (type != NULL) *type = d;
  return 0;
}

/* Items of a tuple of n integers; 1 if it is one, 0 if not, -1 on an error. */
static int ints(PyObject* tuple, Py_ssize_t n, int64_t* out) {
  if (tuple == NULL) return -1;
  int r = PyTuple_Check(tuple) && PyTuple_GET_SIZE(tuple) == n;
  for (Py_ssize_t i = 0; r == 1 && i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (out[i] == -1 && PyErr_Occurred()) r = -1;
  }
  Py_DECREF(tuple);
  return r;
}

/* A row-major matrix of a type; rows and cols < 0: any. */
static int matrix(PyObject* t, const char* name, PyObject* type, int64_t rows, int64_t cols, Mat* m) {
  int64_t shape[2], stride[2];
  if (has_dtype(t, name, type) < 0) return -1;
  int r = ints(PyObject_GetAttr(t, s_shape), 2, shape);
  if (r > 0) r = ints(PyObject_CallMethodNoArgs(t, s_stride), 2, stride);
  if (r < 0) return -1;
  if (r == 0 || (stride[1] != 1 && shape[1] > 1)) return fail(PyExc_ValueError, "%s must be a row-major 2-D tensor", name);
  if ((rows >= 0 && shape[0] != rows) || (cols >= 0 && shape[1] != cols))
    return fail(PyExc_ValueError, "%s has another number of rows or columns than the call needs", name);
  m->rows = shape[0];
  m->cols = shape[1];
  /* one row's stride says nothing: it counts as at least the row's width */
  m->ld = shape[0] > 1 || stride[0] >= shape[1] ? stride[0] : (shape[1] + 7) / 8 * 8;
  return address(t, name, &m->p);
}

/* A contiguous tensor of `dims` (1 or 2) dimensions; None is NULL with sizes 0.  n < 0: any first size. */
static int table(PyObject* t, const char* name, PyObject* type, int dims, int64_t n, void** p, int64_t* shape) {
  shape[0] = shape[dims - 1] = 0;
  *p = NULL;
  if (t == Py_None) return 0;
  if (has_dtype(t, name, type) < 0) return -1;
  int r = ints(PyObject_GetAttr(t, s_shape), dims, shape);
  if (r < 0) return -1;
  if (r > 0) {
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (c == NULL) return -1;
    r = PyObject_IsTrue(c);
    Py_DECREF(c);
    if (r < 0) return -1;
  }
  if (r == 0) {
    PyErr_Format(PyExc_TypeError, "%s must be a contiguous %d-D tensor", name, dims);
    return -1;
  }
  if (n >= 0 && shape[0] != n) return fail(PyExc_ValueError, "%s has another number of entries than the call needs", name);
  return address(t, name, p);
}

static int vector_i32(PyObject* t, const char* name, int64_t n, const int32_t** p) {
  int64_t shape[2];
  void* a;
  if (table(t, name, t_i32, 1, n, &a, shape) < 0) return -1;
  *p = (const int32_t*)a;
  return 0;
}

/* One int32 on the device, the first of a vector; None is NULL. */
static int word_i32(PyObject* t, const char* name, const int32_t** p) {
  int64_t shape[2];
  void* a;
  if (table(t, name, t_i32, 1, -1, &a, shape) < 0) return -1;
  if (t != Py_None && shape[0] < 1) return fail(PyExc_ValueError, "%s is empty", name);
  *p = (const int32_t*)a;
  return 0;
}

/* The status word: any int32 tensor with an element; None is NULL. */
static int status_word(PyObject* t, void** p) {
  *p = NULL;
  if (t == Py_None) return 0;
  if (has_dtype(t, "status", t_i32) < 0 || address(t, "status", p) < 0) return -1;
  return *p != NULL ? 0 : fail(PyExc_ValueError, "%s is empty", "status"); /* an empty tensor's address */
}

static int attr_table(PyObject* o, PyObject* attr, PyObject* type, int dims, int64_t n, void** p, int64_t* shape) {
  PyObject* t = PyObject_GetAttr(o, attr);
  if (t == NULL) return -1;
  const int r = table(t, PyUnicode_AsUTF8(attr), type, dims, n, p, shape);
  Py_DECREF(t); /* the object holds it */
  return r;
}

static int head_map(PyObject* o, lr_head_map* h) {
  int64_t shape[2];
  void* p;
  memset(h, 0, sizeof(*h));
  PyObject* v = PyObject_GetAttr(o, s_norm);
  if (v == NULL) return -1;
  const int norm = PyObject_IsTrue(v);
  Py_DECREF(v);
  if (norm < 0) return -1;
  h->norm = norm;
  if ((v = PyObject_GetAttr(o, s_eps)) == NULL) return -1;
  h->eps = (float)PyFloat_AsDouble(v);
  Py_DECREF(v);
  if (PyErr_Occurred()) return -1;
  if (attr_i32(o, s_head_dim, &h->head_dim) < 0 || attr_i32(o, s_rot_dim, &h->rot_dim) < 0 ||
      attr_i32(o, s_rot_style, &h->rot_style) < 0)
    return -1;
  if (attr_table(o, s_q_gain, t_bf16, 1, h->head_dim, &p, shape) < 0) return -1;
  h->q_gain = p;
  if (attr_table(o, s_k_gain, t_bf16, 1, h->head_dim, &p, shape) < 0) return -1;
  h->k_gain = p;
  if (h->rot_dim > 0) {
    if (attr_table(o, s_cos_sin, t_f32, 2, -1, &p, shape) < 0) return -1;
    if (p != NULL && shape[1] != h->rot_dim) return fail(PyExc_ValueError, "%s must be [max_pos][rot_dim]", "cos_sin");
    h->cos_sin = (const float*)p;
    h->max_pos = shape[0];
  }
  return 0;
}

static int kv_cache(PyObject* o, lr_kv_cache* c) {
  Mat k, v;
  int64_t heads, hd, br;
  memset(c, 0, sizeof(*c));
  PyObject* t = PyObject_GetAttr(o, s_k_pool);
  if (t == NULL) return -1;
  int r = matrix(t, "k_pool", t_bf16, -1, -1, &k);
  Py_DECREF(t);
  if (r < 0 || (t = PyObject_GetAttr(o, s_v_pool)) == NULL) return -1;
  r = matrix(t, "v_pool", t_bf16, k.rows, k.cols, &v);
  Py_DECREF(t);
  if (r < 0 || attr_i64(o, s_n_kv_heads, &heads) < 0 || attr_i64(o, s_head_dim, &hd) < 0 ||
      attr_i64(o, s_block_rows, &br) < 0)
    return -1;
  if (k.ld != v.ld) return fail(PyExc_ValueError, "%s must have one row stride", "k_pool and v_pool");
  if (to_i32(heads, "n_kv_heads", &c->n_kv_heads) < 0 || to_i32(hd, "head_dim", &c->head_dim) < 0 ||
      to_i32(br, "block_rows", &c->block_rows) < 0)
    return -1;
  if (k.cols < heads * hd) return fail(PyExc_ValueError, "%s are narrower than n_kv_heads * head_dim", "the pools' rows");
  if (br <= 0 || k.rows % br) return fail(PyExc_ValueError, "%s must be whole pages of block_rows", "the pools' rows");
  c->k = k.p;
  c->v = v.p;
  c->ld = k.ld;
  c->pool_blocks = k.rows / br;
  return 0;
}

static int attn_desc(int64_t n_heads, PyObject* cache, PyObject* prefix_blocks, PyObject* prefix_len,
                     PyObject* block_table, PyObject* lengths, PyObject* q_start, int64_t max_q, PyObject* scale,
                     lr_attn_desc* d) {
  int64_t shape[2], n;
  void* p;
  memset(d, 0, sizeof(*d));
  if (kv_cache(cache, &d->cache) < 0 || to_i32(n_heads, "n_heads", &d->n_heads) < 0 || to_i32(max_q, "max_q", &d->max_q) < 0)
    return -1;
  if (scale == Py_None) {
    d->scale = d->cache.head_dim > 0 ? (float)(1.0 / sqrt((double)d->cache.head_dim)) : 0.f;
  } else {
    d->scale = (float)PyFloat_AsDouble(scale);
    if (PyErr_Occurred()) return -1;
  }
  if (lengths == Py_None || block_table == Py_None) return fail(PyExc_TypeError, "%s are needed", "lengths and block_table");
  if (table(lengths, "lengths", t_i32, 1, -1, &p, shape) < 0) return -1;
  d->lengths = (const int32_t*)p;
  n = shape[0];
  if (to_i32(n, "the number of sequences", &d->n_seq) < 0) return -1;
  if (table(block_table, "block_table", t_i32, 2, n, &p, shape) < 0) return -1;
  d->block_table = (const int32_t*)p;
  if (to_i32(shape[1], "blocks_per_seq", &d->blocks_per_seq) < 0) return -1;
  if (table(prefix_blocks, "prefix_blocks", t_i32, 1, -1, &p, shape) < 0) return -1;
  d->prefix_blocks = (const int32_t*)p;
  if (to_i32(shape[0], "the number of prefix pages", &d->cap_prefix_blocks) < 0) return -1;
  if (word_i32(prefix_len, "prefix_len", &d->prefix_len) < 0) return -1;
  return vector_i32(q_start, "q_start", n + 1, &d->q_start);
}

static int stream_of(PyObject* v, lr_stream* s) {
  const unsigned long long a = PyLong_AsUnsignedLongLong(v);
  if (a == (unsigned long long)-1 && PyErr_Occurred()) return -1;
  *s = (lr_stream)(uintptr_t)a;
  return 0;
}

static int n_args(const char* name, Py_ssize_t got, Py_ssize_t want) {
  host_tensor = NULL;
  if (got == want && g_rope != NULL) return 0;
  PyErr_Format(PyExc_TypeError, "%s: %zd arguments after init(), not %zd", name, want, got);
  return -1;
}

/* (q, k, pos, heads, q_out, k_out, status, n_active, stream) -> status */
static PyObject* py_qk_norm_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n_args("qk_norm_rope", n, 9) < 0) return NULL;
  Mat q = {0}, k = {0}, qo = {0}, ko = {0};
  lr_head_map hm;
  const int32_t *pos, *active;
  void* status;
  lr_dtype code;
  lr_stream s;
  PyObject *first = a[0] != Py_None ? a[0] : a[1], *type;
  if (head_map(a[3], &hm) < 0) return NULL;
  if (first == Py_None || hm.head_dim <= 0) {
    PyErr_SetString(PyExc_ValueError, "qk_norm_rope: q or k and a positive head_dim are needed");
    return NULL;
  }
  if (code_of(first, &code, &type) < 0) return NULL;
  int64_t rows = -1;
  if (a[0] != Py_None) {
    if (matrix(a[0], "q", type, -1, -1, &q) < 0 || matrix(a[4], "q_out", t_bf16, q.rows, q.cols, &qo) < 0) return NULL;
    rows = q.rows;
  }
  if (a[1] != Py_None) {
    if (matrix(a[1], "k", type, rows, -1, &k) < 0 || matrix(a[5], "k_out", t_bf16, k.rows, k.cols, &ko) < 0) return NULL;
    rows = k.rows;
  }
  if (q.cols % hm.head_dim || k.cols % hm.head_dim) {
    PyErr_SetString(PyExc_ValueError, "qk_norm_rope: a width is not whole heads of head_dim");
    return NULL;
  }
  if (vector_i32(a[2], "pos", rows, &pos) < 0 || word_i32(a[7], "n_active", &active) < 0 ||
      status_word(a[6], &status) < 0 || stream_of(a[8], &s) < 0 || on_gpu(rows) < 0)
    return NULL;
  lr_status st;
  Py_BEGIN_ALLOW_THREADS
  st = g_rope(q.p, q.ld, (int32_t)(q.cols / hm.head_dim), k.p, k.ld, (int32_t)(k.cols / hm.head_dim), code, rows, pos,
              active, &hm, qo.p, qo.ld, ko.p, ko.ld, (int32_t*)status, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* (k, v, pos, rows, heads, cache, status, q, q_out, n_active, stream) -> status */
static PyObject* py_kv_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n_args("kv_append", n, 11) < 0) return NULL;
  Mat k, v, q = {0}, qo = {0};
  lr_head_map hm;
  lr_kv_cache c;
  const int32_t *pos, *rows, *active;
  void* status;
  lr_dtype code;
  lr_stream s;
  PyObject* type;
  if (head_map(a[4], &hm) < 0 || kv_cache(a[5], &c) < 0 || code_of(a[0], &code, &type) < 0) return NULL;
  if (matrix(a[0], "k", type, -1, (int64_t)c.n_kv_heads * c.head_dim, &k) < 0 ||
      matrix(a[1], "v", type, k.rows, k.cols, &v) < 0)
    return NULL;
  if (a[7] != Py_None) {
    if (matrix(a[7], "q", type, k.rows, -1, &q) < 0 || matrix(a[8], "q_out", t_bf16, k.rows, q.cols, &qo) < 0) return NULL;
    if (hm.head_dim <= 0 || q.cols % hm.head_dim) {
      PyErr_SetString(PyExc_ValueError, "kv_append: q's width is not whole heads of head_dim");
      return NULL;
    }
  }
  if (vector_i32(a[2], "pos", k.rows, &pos) < 0 || vector_i32(a[3], "rows", k.rows, &rows) < 0 ||
      word_i32(a[9], "n_active", &active) < 0 || status_word(a[6], &status) < 0 || stream_of(a[10], &s) < 0 ||
      on_gpu(k.rows) < 0)
    return NULL;
  lr_status st;
  Py_BEGIN_ALLOW_THREADS
  st = g_append(k.p, k.ld, v.p, v.ld, q.p, q.ld, a[7] == Py_None ? 0 : (int32_t)(q.cols / hm.head_dim), code, k.rows,
                pos, rows, active, &hm, &c, qo.p, qo.ld, (int32_t*)status, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* (q, n_heads, cache, prefix_blocks, prefix_len, block_table, lengths, out, workspace, status, q_start, max_q, scale,
 * stream) -> status */
static PyObject* py_prefix_attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n_args("prefix_attention", n, 14) < 0) return NULL;
  Mat q, out;
  lr_attn_desc d;
  lr_dtype code;
  lr_stream s;
  PyObject* type;
  void *ws, *status;
  int64_t heads, max_q, bytes = 0;
  if (arg_i64(a[1], &heads) < 0 || arg_i64(a[11], &max_q) < 0 ||
      attn_desc(heads, a[2], a[3], a[4], a[5], a[6], a[10], max_q, a[12], &d) < 0 || code_of(a[7], &code, &type) < 0)
    return NULL;
  if (matrix(a[0], "q", t_bf16, -1, (int64_t)d.n_heads * d.cache.head_dim, &q) < 0 ||
      matrix(a[7], "out", type, q.rows, q.cols, &out) < 0)
    return NULL;
  if (address(a[8], "workspace", &ws) < 0 || (a[8] != Py_None && attr_i64(a[8], s_nbytes, &bytes) < 0) ||
      status_word(a[9], &status) < 0 || stream_of(a[13], &s) < 0 || on_gpu(q.rows) < 0)
    return NULL;
  lr_status st;
  Py_BEGIN_ALLOW_THREADS
  st = g_attention(q.p, q.ld, out.p, out.ld, code, q.rows, &d, ws, (size_t)bytes, (int32_t*)status, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* The structures of lr.h as bytes, for the calls that take them from Python. */
static PyObject* py_head_map(PyObject* self, PyObject* o) {
  (void)self;
  lr_head_map h;
  return head_map(o, &h) < 0 ? NULL : PyBytes_FromStringAndSize((const char*)&h, sizeof(h));
}
static PyObject* py_kv_cache(PyObject* self, PyObject* o) {
  (void)self;
  lr_kv_cache c;
  return kv_cache(o, &c) < 0 ? NULL : PyBytes_FromStringAndSize((const char*)&c, sizeof(c));
}
/* (n_heads, cache, prefix_blocks, prefix_len, block_table, lengths, q_start, max_q, scale) */
static PyObject* py_attn_desc(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  lr_attn_desc d;
  int64_t heads, max_q;
  if (n_args("attn_desc", n, 9) < 0 || arg_i64(a[0], &heads) < 0 || arg_i64(a[7], &max_q) < 0 ||
      attn_desc(heads, a[1], a[2], a[3], a[4], a[5], a[6], max_q, a[8], &d) < 0)
    return NULL;
  return PyBytes_FromStringAndSize((const char*)&d, sizeof(d));
}
/* (context, M, n_heads, whether it is for a launch) */
static PyObject* py_context(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  PyObject* names[] = {s_cache, s_prefix_blocks, s_prefix_len, s_block_table, s_lengths, s_q_start, s_scale,
                       s_heads, s_pos, s_rows, s_n_active};
  PyObject* v[11] = {0};
  lr_context c;
  int64_t m, heads, max_q;
  int ok = n_args("context", n, 4) == 0 && arg_i64(a[1], &m) == 0 && arg_i64(a[2], &heads) == 0 &&
           attr_i64(a[0], s_max_q, &max_q) == 0;
  memset(&c, 0, sizeof(c));
  for (int i = 0; ok && i < 11; ++i) ok = (v[i] = PyObject_GetAttr(a[0], names[i])) != NULL;
  ok = ok && attn_desc(heads, v[0], v[1], v[2], v[3], v[4], v[5], max_q, v[6], &c.attn) == 0 &&
       head_map(v[7], &c.heads) == 0 && vector_i32(v[8], "pos", m, &c.pos) == 0 &&
       vector_i32(v[9], "rows", m, &c.rows) == 0 && word_i32(v[10], "n_active", &c.n_active) == 0 &&
       (a[3] != Py_True || on_gpu(m) == 0);
  for (int i = 0; i < 11; ++i) Py_XDECREF(v[i]);
  return ok ? PyBytes_FromStringAndSize((const char*)&c, sizeof(c)) : NULL;
}

/* (bfloat16, float32, int32, addresses of lr_qk_norm_rope, lr_kv_append, lr_prefix_attention) */
static PyObject* py_init(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 6) return PyErr_Format(PyExc_TypeError, "init: 6 arguments, not %zd", n);
  unsigned long long f[3];
  for (int i = 0; i < 3; ++i) {
    f[i] = PyLong_AsUnsignedLongLong(a[3 + i]);
    if (f[i] == (unsigned long long)-1 && PyErr_Occurred()) return NULL;
  }
  Py_XSETREF(t_bf16, Py_NewRef(a[0]));
  Py_XSETREF(t_f32, Py_NewRef(a[1]));
  Py_XSETREF(t_i32, Py_NewRef(a[2]));
  g_rope = (rope_fn)(uintptr_t)f[0];
  g_append = (append_fn)(uintptr_t)f[1];
  g_attention = (attention_fn)(uintptr_t)f[2];
  Py_RETURN_NONE;
}

#define FAST(f) ((PyCFunction)(void (*)(void))(f))
static PyMethodDef methods[] = {{"init", FAST(py_init), METH_FASTCALL, NULL},
                                {"qk_norm_rope", FAST(py_qk_norm_rope), METH_FASTCALL, NULL},
                                {"kv_append", FAST(py_kv_append), METH_FASTCALL, NULL},
                                {"prefix_attention", FAST(py_prefix_attention), METH_FASTCALL, NULL},
                                {"attn_desc", FAST(py_attn_desc), METH_FASTCALL, NULL},
                                {"context", FAST(py_context), METH_FASTCALL, NULL},
                                {"head_map", py_head_map, METH_O, NULL},
                                {"kv_cache", py_kv_cache, METH_O, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void) {
  struct {
    PyObject** at;
    const char* name;
  } names[] = {{&s_dtype, "dtype"}, {&s_shape, "shape"}, {&s_stride, "stride"}, {&s_data_ptr, "data_ptr"},
               {&s_is_contiguous, "is_contiguous"}, {&s_nbytes, "nbytes"}, {&s_head_dim, "head_dim"}, {&s_norm, "norm"},
               {&s_eps, "eps"}, {&s_q_gain, "q_gain"}, {&s_k_gain, "k_gain"}, {&s_rot_dim, "rot_dim"},
               {&s_rot_style, "rot_style"}, {&s_cos_sin, "cos_sin"}, {&s_k_pool, "k_pool"}, {&s_v_pool, "v_pool"},
               {&s_n_kv_heads, "n_kv_heads"}, {&s_block_rows, "block_rows"}, {&s_cache, "cache"}, {&s_heads, "heads"},
               {&s_pos, "pos"}, {&s_rows, "rows"}, {&s_prefix_blocks, "prefix_blocks"}, {&s_prefix_len, "prefix_len"},
               {&s_block_table, "block_table"}, {&s_lengths, "lengths"}, {&s_q_start, "q_start"}, {&s_max_q, "max_q"},
               {&s_scale, "scale"}, {&s_n_active, "n_active"}, {&s_is_cuda, "is_cuda"}};
  for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
    if ((*names[i].at = PyUnicode_InternFromString(names[i].name)) == NULL) return NULL;
  return PyModule_Create(&module);
}
