/* grouped_call.c -- the usual calls of the grouped operators, of the operators over rows of scores and of
 * linear layers, from torch tensors to the C ABI.
 *
 * The operators of a decode step take a few microseconds on the GPU; describing their tensors in
 * Python takes longer than that.  This CPython module does it for the usual case -- torch CUDA
 * tensors of the right types on the current device, outputs and workspace allocated here -- and
 * returns None for every other, which grouped.py then handles (and reports) in full.  It holds no
 * arithmetic and no torch headers: tensors are read through their Python attributes, and the
 * entry points' addresses are handed in (grouped.py, scores.py, linear.py).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "tmm_gemm.h"

static PyObject *s_dtype, *s_device, *s_is_cuda, *s_shape, *s_stride, *s_data_ptr, *s_get_device;
static PyObject *t_tensor, *t_empty, *t_raw_stream, *t_current_device, *t_row_groups, *t_uint8,
    *t_int32, *t_int64, *t_float32, *t_types[3], *t_kwnames;

static int (*f_group_rows)(int64_t, int64_t, int64_t, const void *, int, int32_t *, int32_t *,
                           int32_t *, int32_t *, void *, size_t, tmm_stream_t);
static size_t (*f_group_rows_size)(int64_t, int64_t, int64_t);
static int (*f_grouped)(int, int, int64_t, int64_t, int64_t, int64_t, const void *, int64_t,
                        int64_t, const int32_t *, const int32_t *, const void *, int64_t, int64_t,
                        void *, int64_t, void *, size_t, tmm_stream_t);
static size_t (*f_grouped_size)(int, int, int64_t, int64_t, int64_t, int64_t, const void *, int64_t,
                                int64_t, const int32_t *, const void *, int64_t, int64_t);
static int (*f_wgrad)(int, int64_t, int64_t, int64_t, int64_t, const void *, int64_t, int64_t,
                      const int32_t *, const int32_t *, const void *, int64_t, void *, int64_t,
                      int64_t, void *, size_t, tmm_stream_t);
static size_t (*f_wgrad_size)(int, int64_t, int64_t, int64_t, int64_t, const void *, int64_t,
                              int64_t, const int32_t *, const void *, int64_t);
static int (*f_lora)(int, int, int, int, int64_t, int64_t, int64_t, int64_t, int64_t, const void *,
                     int64_t, const int32_t *, const int32_t *, const void *, int64_t,
                     const void *, int64_t, int64_t, const void *, int64_t, int64_t, const float *,
                     void *, int64_t, void *, size_t, tmm_stream_t);
static size_t (*f_lora_size)(int, int, int, int, int64_t, int64_t, int64_t, int64_t, int64_t,
                             const void *, int64_t, const int32_t *, const void *, int64_t,
                             const void *, int64_t, int64_t, const void *, int64_t, int64_t);

/* A tensor as an operand: rows x cols matrices, `count` of them, or a vector (rows 1). */
typedef struct {
  int code;                 /* element type: TMM_*, or -1 for others */
  PyObject *type;           /* borrowed from torch: dtypes are never freed */
  long device;
  void *ptr;
  int64_t count, rows, cols, ld, stride;
  int trans;
} Operand;

static int as_ints(PyObject *t, int64_t *out, int want) {
  if (t == NULL || !PyTuple_Check(t) || PyTuple_GET_SIZE(t) != want) return 0;
  for (int i = 0; i < want; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
  return !PyErr_Occurred();
}

/* 1 when `x` is a CUDA tensor of `dims` dimensions in a layout that an operand may have. */
static int describe(PyObject *x, int dims, int transposable, Operand *o) {
  if (!PyObject_TypeCheck(x, (PyTypeObject *)t_tensor)) return 0;
  PyObject *v = PyObject_GetAttr(x, s_is_cuda);
  const int cuda = v == Py_True;
  Py_XDECREF(v);
  if (!cuda) return 0;
  int64_t n[3] = {1, 1, 1}, s[3] = {0, 0, 0};
  v = PyObject_GetAttr(x, s_shape);
  int ok = as_ints(v, n + 3 - dims, dims);
  Py_XDECREF(v);
  if (!ok) return 0;
  v = PyObject_CallMethodNoArgs(x, s_stride);
  ok = as_ints(v, s + 3 - dims, dims);
  Py_XDECREF(v);
  if (!ok) return 0;
  v = PyObject_GetAttr(x, s_dtype);
  if (v == NULL) return 0;
  o->type = v;
  o->code = v == t_types[0] ? TMM_F32 : v == t_types[1] ? TMM_BF16 : v == t_types[2] ? TMM_F16 : -1;
  Py_DECREF(v);
  v = PyObject_CallMethodNoArgs(x, s_get_device);
  o->device = v ? PyLong_AsLong(v) : -1;
  Py_XDECREF(v);
  v = PyObject_CallMethodNoArgs(x, s_data_ptr);
  o->ptr = v ? PyLong_AsVoidPtr(v) : NULL;
  Py_XDECREF(v);
  if (PyErr_Occurred()) return 0;
  o->count = n[0];
  o->rows = n[1];
  o->cols = n[2];
  o->stride = dims == 3 && n[0] > 1 ? s[0] : 0;
  if (n[0] < 1 || n[1] < 1 || n[2] < 1) return 0;
  if (s[2] == 1 && s[1] >= n[2]) {
    o->ld = s[1];
    o->trans = 0;
    return 1;
  }
  if (transposable && s[1] == 1 && s[2] >= n[1]) {
    o->ld = s[2];
    o->trans = 1;
    return 1;
  }
  return dims == 1 && s[2] == 1;
}

/* A contiguous int32 vector of `length` values (any with -1) on the operands' device. */
static int index_of(PyObject *x, const Operand *like, int64_t length, Operand *o) {
  return describe(x, 1, 0, o) && o->type == t_int32 && o->device == like->device &&
         (length < 0 || o->cols == length);
}

/* The current stream of the device, which has to be the current one. */
static int stream_of(long device, tmm_stream_t *out) {
  PyObject *v = PyObject_CallNoArgs(t_current_device);
  const long now = v ? PyLong_AsLong(v) : -1;
  Py_XDECREF(v);
  if (now != device) return 0;
  PyObject *d = PyLong_FromLong(device);
  v = d ? PyObject_CallOneArg(t_raw_stream, d) : NULL;
  Py_XDECREF(d);
  if (v == NULL) return 0;
  *out = (tmm_stream_t)PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return !PyErr_Occurred();
}

/* torch.empty(shape, dtype=type, device=device); steals shape. */
static PyObject *empty(PyObject *shape, PyObject *type, PyObject *device) {
  if (shape == NULL) return NULL;
  PyObject *args[3] = {shape, type, device};
  PyObject *r = PyObject_Vectorcall(t_empty, args, 1, t_kwnames);
  Py_DECREF(shape);
  return r;
}

static void *pointer(PyObject *x) {
  PyObject *v = PyObject_CallMethodNoArgs(x, s_data_ptr);
  void *p = v ? PyLong_AsVoidPtr(v) : NULL;
  Py_XDECREF(v);
  return p;
}

/* A workspace of `need` bytes in *ws (NULL for none); 0 on failure. */
static int scratch(size_t need, PyObject *device, PyObject **ws, void **p) {
  *ws = NULL;
  *p = NULL;
  if (need == 0) return 1;
  if (need > (size_t)PY_SSIZE_T_MAX) return 0;
  *ws = empty(Py_BuildValue("(n)", (Py_ssize_t)need), t_uint8, device);
  if (*ws == NULL) return 0;
  *p = pointer(*ws);
  return *p != NULL;
}

/* rc = call, with the interpreter's lock released: a launch may block, on a full queue or while its
 * kernel is loaded, and holds only this call's own values. */
#define WITHOUT_LOCK(call)                  \
  int rc;                                   \
  Py_BEGIN_ALLOW_THREADS rc = (call);       \
  Py_END_ALLOW_THREADS

/* None, with no error set: the caller's Python path takes over (and meets the error itself). */
static PyObject *other(PyObject *a, PyObject *b, PyObject *c) {
  Py_XDECREF(a);
  Py_XDECREF(b);
  Py_XDECREF(c);
  PyErr_Clear();
  Py_RETURN_NONE;
}

static PyObject *grouped(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  Operand x, w, off, rows;
  if (n != 4 || !describe(a[0], 2, 0, &x) || x.code < 0 || !describe(a[1], 3, 1, &w) ||
      w.type != x.type || w.device != x.device || w.rows != x.cols ||
      !index_of(a[2], &x, w.count + 1, &off))
    return other(NULL, NULL, NULL);
  int64_t R = x.rows;
  const int32_t *index = NULL;
  if (a[3] != Py_None) {
    if (!index_of(a[3], &x, -1, &rows)) return other(NULL, NULL, NULL);
    R = rows.cols;
    index = rows.ptr;
  }
  tmm_stream_t s;
  if (!stream_of(x.device, &s)) return other(NULL, NULL, NULL);
  PyObject *device = PyObject_GetAttr(a[0], s_device), *ws = NULL, *y = NULL;
  void *wp, *yp;
  const size_t need = f_grouped_size(x.code, w.trans, w.count, R, w.cols, x.cols, x.ptr, x.rows,
                                     x.ld, index, w.ptr, w.ld, w.stride);
  if (device == NULL || !scratch(need, device, &ws, &wp)) return other(device, ws, NULL);
  y = empty(Py_BuildValue("(LL)", (long long)R, (long long)w.cols), x.type, device);
  if (y == NULL || (yp = pointer(y)) == NULL) return other(device, ws, y);
  WITHOUT_LOCK(f_grouped(x.code, w.trans, w.count, R, w.cols, x.cols, x.ptr, x.rows, x.ld, off.ptr,
                         index, w.ptr, w.ld, w.stride, yp, w.cols, wp, need, s))
  if (rc != TMM_OK) return other(device, ws, y);
  Py_DECREF(device);
  Py_XDECREF(ws);
  return y;
}

static PyObject *wgrad(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  Operand x, dy, off, rows;
  if (n != 4 || !describe(a[0], 2, 0, &x) || x.code < 0 || !describe(a[1], 2, 0, &dy) ||
      dy.type != x.type || dy.device != x.device || !index_of(a[2], &x, -1, &off) || off.cols < 2)
    return other(NULL, NULL, NULL);
  const int32_t *index = NULL;
  if (a[3] != Py_None) {
    if (!index_of(a[3], &x, dy.rows, &rows)) return other(NULL, NULL, NULL);
    index = rows.ptr;
  } else if (x.rows != dy.rows) {
    return other(NULL, NULL, NULL);
  }
  const int64_t groups = off.cols - 1, K = x.cols, N = dy.cols;
  tmm_stream_t s;
  if (!stream_of(x.device, &s)) return other(NULL, NULL, NULL);
  PyObject *device = PyObject_GetAttr(a[0], s_device), *ws = NULL, *dw = NULL;
  void *wp, *dwp;
  const size_t need =
      f_wgrad_size(x.code, groups, dy.rows, N, K, x.ptr, x.rows, x.ld, index, dy.ptr, dy.ld);
  if (device == NULL || !scratch(need, device, &ws, &wp)) return other(device, ws, NULL);
  dw = empty(Py_BuildValue("(LLL)", (long long)groups, (long long)K, (long long)N), x.type, device);
  if (dw == NULL || (dwp = pointer(dw)) == NULL) return other(device, ws, dw);
  WITHOUT_LOCK(f_wgrad(x.code, groups, dy.rows, N, K, x.ptr, x.rows, x.ld, off.ptr, index, dy.ptr,
                       dy.ld, dwp, N, K * N, wp, need, s))
  if (rc != TMM_OK) return other(device, ws, dw);
  Py_DECREF(device);
  Py_XDECREF(ws);
  return dw;
}

static PyObject *lora(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  Operand x, w, la, lb, scale, off, rows;
  if (n != 7 || !describe(a[0], 2, 0, &x) || x.code < 0 || !describe(a[1], 2, 1, &w) ||
      !describe(a[2], 3, 1, &la) || !describe(a[3], 3, 1, &lb) || w.type != x.type ||
      la.type != x.type || lb.type != x.type || w.device != x.device || la.device != x.device ||
      lb.device != x.device || w.rows != x.cols || la.rows != x.cols || lb.cols != w.cols ||
      lb.rows != la.cols || lb.count != la.count || !describe(a[4], 1, 0, &scale) ||
      scale.type != t_float32 || scale.device != x.device || scale.cols != la.count ||
      !index_of(a[5], &x, la.count + 1, &off))
    return other(NULL, NULL, NULL);
  const int32_t *index = NULL;
  if (a[6] != Py_None) {
    if (!index_of(a[6], &x, x.rows, &rows)) return other(NULL, NULL, NULL);
    index = rows.ptr;
  }
  const int64_t T = x.rows, K = x.cols, N = w.cols, r = la.cols;
  tmm_stream_t s;
  if (!stream_of(x.device, &s)) return other(NULL, NULL, NULL);
  PyObject *device = PyObject_GetAttr(a[0], s_device), *ws = NULL, *y = NULL;
  void *wp, *yp;
  const size_t need =
      f_lora_size(x.code, w.trans, la.trans, lb.trans, la.count, T, N, K, r, x.ptr, x.ld, index,
                  w.ptr, w.ld, la.ptr, la.ld, la.stride, lb.ptr, lb.ld, lb.stride);
  if (device == NULL || !scratch(need, device, &ws, &wp)) return other(device, ws, NULL);
  y = empty(Py_BuildValue("(LL)", (long long)T, (long long)N), x.type, device);
  if (y == NULL || (yp = pointer(y)) == NULL) return other(device, ws, y);
  WITHOUT_LOCK(f_lora(x.code, w.trans, la.trans, lb.trans, la.count, T, N, K, r, x.ptr, x.ld, off.ptr,
                      index, w.ptr, w.ld, la.ptr, la.ld, la.stride, lb.ptr, lb.ld, lb.stride,
                      scale.ptr, yp, N, wp, need, s))
  if (rc != TMM_OK) return other(device, ws, y);
  Py_DECREF(device);
  Py_XDECREF(ws);
  return y;
}

static PyObject *group_rows_(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  Operand x;
  if (n != 2 || !PyLong_Check(a[1])) return other(NULL, NULL, NULL);
  const long groups = PyLong_AsLong(a[1]);
  int two = describe(a[0], 2, 0, &x);
  if (!two) {
    PyErr_Clear();
    if (!describe(a[0], 1, 0, &x)) return other(NULL, NULL, NULL);
  }
  if ((x.type != t_int32 && x.type != t_int64) || groups < 1 || groups > TMM_MAX_GROUPS ||
      (two && x.ld != x.cols))
    return other(NULL, NULL, NULL);
  const int64_t tokens = two ? x.rows : x.cols, fan = two ? x.cols : 1, slots = tokens * fan;
  tmm_stream_t s;
  if (!stream_of(x.device, &s)) return other(NULL, NULL, NULL);
  PyObject *device = PyObject_GetAttr(a[0], s_device), *ws = NULL, *r = NULL;
  if (device == NULL) return other(NULL, NULL, NULL);
  PyObject *out[4] = {NULL, NULL, NULL, NULL};
  void *p[4] = {NULL, NULL, NULL, NULL}, *wp;
  const size_t need = f_group_rows_size(tokens, fan, groups);
  int ok = scratch(need, device, &ws, &wp);
  for (int i = 0; i < 4 && ok; ++i) {
    out[i] = empty(Py_BuildValue("(L)", (long long)(i == 0 ? groups + 1 : slots)), t_int32, device);
    ok = out[i] != NULL && (p[i] = pointer(out[i])) != NULL;
  }
  if (ok) {
    WITHOUT_LOCK(f_group_rows(tokens, fan, groups, x.ptr, x.type == t_int64 ? 64 : 32, p[0], p[1],
                              p[2], p[3], wp, need, s))
    if (rc == TMM_OK) r = PyObject_Vectorcall(t_row_groups, out, 4, NULL);
  }
  for (int i = 0; i < 4; ++i) Py_XDECREF(out[i]);
  if (r == NULL) return other(device, ws, NULL);
  Py_DECREF(device);
  Py_XDECREF(ws);
  return r;
}

/* start(objects, addresses): what grouped.py hands in, once. */
static PyObject *start(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (n != 2 || !PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 12 || !PyTuple_Check(a[1]) ||
      PyTuple_GET_SIZE(a[1]) != 8) {
    PyErr_SetString(PyExc_TypeError, "start(objects, addresses)");
    return NULL;
  }
  PyObject **const to[12] = {&t_tensor,     &t_empty,    &t_raw_stream, &t_current_device,
                             &t_row_groups, &t_uint8,    &t_int32,      &t_int64,
                             &t_float32,    &t_types[0], &t_types[1],   &t_types[2]};
  void **const fn[8] = {(void **)&f_group_rows, (void **)&f_group_rows_size, (void **)&f_grouped,
                        (void **)&f_grouped_size, (void **)&f_wgrad, (void **)&f_wgrad_size,
                        (void **)&f_lora, (void **)&f_lora_size};
  for (int i = 0; i < 12; ++i) {
    *to[i] = PyTuple_GET_ITEM(a[0], i);
    Py_INCREF(*to[i]);
  }
  for (int i = 0; i < 8; ++i) *fn[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[1], i));
  if (PyErr_Occurred()) return NULL;
  Py_RETURN_NONE;
}

/* ---- rows of scores ---------------------------------------------------------------------- */

static PyObject *t_row_routes, *t_row_logprobs;
static int (*f_route)(int, int64_t, int64_t, const void *, int64_t, const float *, int, int64_t,
                      int64_t, int, int64_t, int, float, int32_t *, float *, tmm_stream_t);
static int (*f_route_grad)(int, int64_t, int64_t, int64_t, const float *, const void *, int64_t,
                           const int32_t *, int, int, float, void *, int64_t, tmm_stream_t);
static int (*f_logprob)(int, int64_t, int64_t, const void *, int64_t, float, const void *, int, int,
                        float *, float *, float *, int32_t *, float *, tmm_stream_t);
static int (*f_logprob_grad)(int, int64_t, int64_t, const void *, int64_t, float, const float *,
                             const void *, int, const float *, const float *, const float *, int,
                             const int32_t *, const float *, void *, int64_t, tmm_stream_t);

/* A whole number that fits an int, a truth value, a float: 0 for anything else. */
static int int_of(PyObject *x, int *out) {
  if (!PyLong_CheckExact(x)) return 0;
  int over = 0;
  const long v = PyLong_AsLongAndOverflow(x, &over);
  *out = (int)v;
  return !over && v == (long)*out;
}
static int truth_of(PyObject *x, int *out) {
  *out = x == Py_True;
  return x == Py_True || x == Py_False;
}
static int float_of(PyObject *x, float *out) {
  if (!PyFloat_CheckExact(x)) return 0;
  *out = (float)PyFloat_AS_DOUBLE(x);
  return 1;
}

/* The address of a contiguous tensor of `rows` x `cols` (rows 0: `cols` values) of a type, on the
 * operands' device; NULL for None where that is allowed. */
static int array_of(PyObject *x, const Operand *like, PyObject *type, int64_t rows, int64_t cols,
                    int none, void **out) {
  Operand o;
  *out = NULL;
  if (x == Py_None) return none;
  if (!describe(x, rows ? 2 : 1, 0, &o) || o.type != type || o.device != like->device ||
      o.cols != cols || (rows && (o.rows != rows || o.ld != cols)))
    return 0;
  *out = o.ptr;
  return 1;
}

/* New outputs: r[i] of shape (a) or, with b[i] >= 0, (a, b[i]). */
static int new_outputs(int n, PyObject **r, void **p, int64_t a, const int64_t *b,
                       PyObject *const *types, PyObject *device) {
  for (int i = 0; i < n; ++i) {
    r[i] = empty(b[i] < 0 ? Py_BuildValue("(L)", (long long)a)
                          : Py_BuildValue("(LL)", (long long)a, (long long)b[i]),
                 types[i], device);
    if (r[i] == NULL || (p[i] = pointer(r[i])) == NULL) return 0;
  }
  return 1;
}
static PyObject *drop_all(int n, PyObject **r, PyObject *device) {
  for (int i = 0; i < n; ++i) Py_XDECREF(r[i]);
  return other(device, NULL, NULL);
}

static PyObject *route(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  Operand x;
  int k, score, groups, top, best, renormalise;
  float scale;
  void *bias, *p[2];
  tmm_stream_t s;
  if (n != 9 || !describe(a[0], 2, 0, &x) || x.code < 0 || !int_of(a[1], &k) ||
      !array_of(a[2], &x, t_float32, 0, x.cols, 1, &bias) || !int_of(a[3], &score) ||
      !int_of(a[4], &groups) || !int_of(a[5], &top) || !int_of(a[6], &best) ||
      !truth_of(a[7], &renormalise) || !float_of(a[8], &scale) || k < 1 || k > TMM_MAX_FAN ||
      !stream_of(x.device, &s))
    return other(NULL, NULL, NULL);
  PyObject *device = PyObject_GetAttr(a[0], s_device), *r[2] = {NULL, NULL};
  PyObject *const types[2] = {t_int32, t_float32};
  const int64_t cols[2] = {k, k};
  if (device == NULL || !new_outputs(2, r, p, x.rows, cols, types, device))
    return drop_all(2, r, device);
  WITHOUT_LOCK(f_route(x.code, x.rows, x.cols, x.ptr, x.ld, bias, score, groups, top, best, k,
                       renormalise, scale, p[0], p[1], s))
  if (rc != TMM_OK) return drop_all(2, r, device);
  PyObject *out = PyObject_Vectorcall(t_row_routes, r, 2, NULL);
  for (int i = 0; i < 2; ++i) Py_DECREF(r[i]);
  Py_DECREF(device);
  return out;
}

static PyObject *route_grad(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  Operand dw, x;
  int score, renormalise;
  float scale;
  void *chosen, *p;
  tmm_stream_t s;
  if (n != 6 || !describe(a[0], 2, 0, &dw) || !describe(a[1], 2, 0, &x) || x.code < 0 ||
      dw.type != t_float32 || dw.device != x.device || dw.rows != x.rows || dw.ld != dw.cols ||
      !array_of(a[2], &x, t_int32, x.rows, dw.cols, 0, &chosen) || !int_of(a[3], &score) ||
      !truth_of(a[4], &renormalise) || !float_of(a[5], &scale) || !stream_of(x.device, &s))
    return other(NULL, NULL, NULL);
  PyObject *device = PyObject_GetAttr(a[1], s_device), *r = NULL;
  if (device == NULL || !new_outputs(1, &r, &p, x.rows, &x.cols, &x.type, device))
    return drop_all(1, &r, device);
  WITHOUT_LOCK(f_route_grad(x.code, x.rows, x.cols, dw.cols, dw.ptr, x.ptr, x.ld, chosen, score,
                            renormalise, scale, p, x.cols, s))
  if (rc != TMM_OK) return drop_all(1, &r, device);
  Py_DECREF(device);
  return r;
}

/* Tokens of int32 or int64, or None. */
static int tokens_of(PyObject *x, const Operand *like, void **p, int *bits) {
  *bits = 32;
  if (array_of(x, like, t_int32, 0, like->rows, 1, p)) return 1;
  *bits = 64;
  return !PyErr_Occurred() && array_of(x, like, t_int64, 0, like->rows, 0, p);
}

static PyObject *logprob(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  Operand x;
  int top, bits;
  float scale;
  void *tokens, *p[5] = {NULL, NULL, NULL, NULL, NULL};
  tmm_stream_t s;
  if (n != 4 || !describe(a[0], 2, 0, &x) || x.code < 0 || !tokens_of(a[1], &x, &tokens, &bits) ||
      !int_of(a[2], &top) || top < 0 || top > TMM_MAX_TOP || !float_of(a[3], &scale) ||
      !stream_of(x.device, &s))
    return other(NULL, NULL, NULL);
  PyObject *device = PyObject_GetAttr(a[0], s_device), *r[5] = {NULL, NULL, NULL, NULL, NULL};
  PyObject *const types[5] = {t_float32, t_float32, t_float32, t_int32, t_float32};
  const int64_t cols[5] = {-1, -1, -1, top, top};
  const int skip = tokens == NULL;
  if (device == NULL ||
      !new_outputs((top ? 5 : 3) - skip, r + skip, p + skip, x.rows, cols + skip, types + skip,
                   device))
    return drop_all(5, r, device);
  WITHOUT_LOCK(f_logprob(x.code, x.rows, x.cols, x.ptr, x.ld, scale, tokens, bits, top, p[0], p[1],
                         p[2], p[3], p[4], s))
  if (rc != TMM_OK) return drop_all(5, r, device);
  for (int i = 0; i < 5; ++i)
    if (r[i] == NULL) {
      r[i] = Py_None;
      Py_INCREF(Py_None);
    }
  PyObject *out = PyObject_Vectorcall(t_row_logprobs, r, 5, NULL);
  for (int i = 0; i < 5; ++i) Py_DECREF(r[i]);
  Py_DECREF(device);
  return out;
}

static PyObject *logprob_grad(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  Operand x, e;
  int bits, top = 0;
  float scale;
  void *tokens, *lse, *g, *entropy, *h, *ids = NULL, *dtop = NULL, *p;
  tmm_stream_t s;
  if (n != 9 || !describe(a[0], 2, 0, &x) || x.code < 0 || !tokens_of(a[1], &x, &tokens, &bits) ||
      !array_of(a[2], &x, t_float32, 0, x.rows, 0, &lse) ||
      !array_of(a[3], &x, t_float32, 0, x.rows, 1, &g) ||
      !array_of(a[4], &x, t_float32, 0, x.rows, 1, &entropy) ||
      !array_of(a[5], &x, t_float32, 0, x.rows, 1, &h) || (g && !tokens) || (h && !entropy) ||
      !float_of(a[8], &scale) || !stream_of(x.device, &s))
    return other(NULL, NULL, NULL);
  if (a[7] != Py_None) {
    if (!describe(a[7], 2, 0, &e) || e.cols > TMM_MAX_TOP ||
        !array_of(a[7], &x, t_float32, x.rows, e.cols, 0, &dtop) ||
        !array_of(a[6], &x, t_int32, x.rows, e.cols, 0, &ids))
      return other(NULL, NULL, NULL);
    top = (int)e.cols;
  }
  PyObject *device = PyObject_GetAttr(a[0], s_device), *r = NULL;
  if (device == NULL || !new_outputs(1, &r, &p, x.rows, &x.cols, &x.type, device))
    return drop_all(1, &r, device);
  WITHOUT_LOCK(f_logprob_grad(x.code, x.rows, x.cols, x.ptr, x.ld, scale, lse, tokens, bits, g,
                              entropy, h, top, ids, dtop, p, x.cols, s))
  if (rc != TMM_OK) return drop_all(1, &r, device);
  Py_DECREF(device);
  return r;
}

/* ---- linear layers ------------------------------------------------------------------------ */

static PyObject *t_linear_grads, *s_t;
static int (*f_linear)(int, int, int, int64_t, int64_t, int64_t, const void *, int64_t, const void *,
                       int64_t, const void *, int, const void *, int64_t, void *, int64_t, void *,
                       int64_t, void *, size_t, tmm_stream_t);
static size_t (*f_linear_size)(int, int, int64_t, int64_t, int64_t, const void *, int64_t,
                               const void *, int64_t);
static int (*f_linear_grad)(int, int, int, int64_t, int64_t, int64_t, const void *, int64_t,
                            const void *, int64_t, const void *, int64_t, const void *, int64_t,
                            void *, int64_t, void *, int64_t, int, float *, void *, size_t,
                            tmm_stream_t);
static size_t (*f_linear_grad_size)(int, int, int, int64_t, int64_t, int64_t, const void *, int64_t,
                                    const void *, int64_t, const void *, int64_t, const void *,
                                    const void *, int, const void *);

static PyObject *linear(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  Operand x, w, res;
  int act, pre, bias_f32 = 0;
  void *bias = NULL, *p[2] = {NULL, NULL}, *wp;
  tmm_stream_t s;
  if (n != 6 || !describe(a[0], 2, 0, &x) || x.code < 0 || !describe(a[1], 2, 1, &w) ||
      w.type != x.type || w.device != x.device || w.rows != x.cols || !int_of(a[3], &act))
    return other(NULL, NULL, NULL);
  if (a[2] != Py_None && !array_of(a[2], &x, x.type, 0, w.cols, 0, &bias)) {
    bias_f32 = 1;
    if (PyErr_Occurred() || !array_of(a[2], &x, t_float32, 0, w.cols, 0, &bias))
      return other(NULL, NULL, NULL);
  }
  res.ptr = NULL;
  res.ld = 1;
  if (a[4] != Py_None && (!describe(a[4], 2, 0, &res) || res.type != x.type ||
                          res.device != x.device || res.rows != x.rows || res.cols != w.cols))
    return other(NULL, NULL, NULL);
  pre = a[5] == Py_True;
  if ((!pre && a[5] != Py_False && a[5] != Py_None) || !stream_of(x.device, &s))
    return other(NULL, NULL, NULL);
  const int64_t M = x.rows, N = w.cols, K = x.cols, cols[2] = {N, N};
  PyObject *device = PyObject_GetAttr(a[0], s_device), *ws = NULL, *r[2] = {NULL, NULL};
  PyObject *const types[2] = {x.type, x.type};
  const size_t need = f_linear_size(x.code, w.trans, M, N, K, x.ptr, x.ld, w.ptr, w.ld);
  if (device == NULL || !scratch(need, device, &ws, &wp) ||
      !new_outputs(1 + pre, r, p, M, cols, types, device)) {
    Py_XDECREF(ws);
    return drop_all(2, r, device);
  }
  WITHOUT_LOCK(f_linear(x.code, w.trans, act, M, N, K, x.ptr, x.ld, w.ptr, w.ld, bias, bias_f32,
                        res.ptr, res.ld, p[0], N, p[1], N, wp, need, s))
  Py_XDECREF(ws);
  if (rc != TMM_OK) return drop_all(2, r, device);
  Py_DECREF(device);
  if (!pre) return r[0];
  PyObject *out = PyTuple_Pack(2, r[0], r[1]);
  for (int i = 0; i < 2; ++i) Py_DECREF(r[i]);
  return out;
}

static PyObject *linear_grad(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  Operand dy, x, w, z;
  int act, want_bias;
  void *p[3] = {NULL, NULL, NULL}, *wp;
  tmm_stream_t s;
  if (n != 6 || !describe(a[0], 2, 0, &dy) || dy.code < 0 || !describe(a[1], 2, 0, &x) ||
      !describe(a[2], 2, 1, &w) || x.type != dy.type || w.type != dy.type ||
      x.device != dy.device || w.device != dy.device || x.rows != dy.rows || w.rows != x.cols ||
      w.cols != dy.cols || !int_of(a[4], &act) || act < 0 || !truth_of(a[5], &want_bias))
    return other(NULL, NULL, NULL);
  z.ptr = NULL;
  z.ld = 1;
  if (act != TMM_ACT_NONE &&
      (!describe(a[3], 2, 0, &z) || z.type != dy.type || z.device != dy.device ||
       z.rows != dy.rows || z.cols != dy.cols))
    return other(NULL, NULL, NULL);
  if (!stream_of(dy.device, &s)) return other(NULL, NULL, NULL);
  const int64_t M = dy.rows, N = dy.cols, K = x.cols;
  const int64_t lddw = w.trans ? K : N;
  PyObject *device = PyObject_GetAttr(a[0], s_device), *ws = NULL, *r[3] = {NULL, NULL, NULL};
  const int64_t none = -1;
  int ok = device != NULL && new_outputs(1, r, p, M, &K, &dy.type, device) &&
           new_outputs(1, r + 1, p + 1, w.trans ? N : K, &lddw, &dy.type, device) &&
           (!want_bias || new_outputs(1, r + 2, p + 2, N, &none, &t_float32, device));
  size_t need = 0;
  if (ok) {
    need = f_linear_grad_size(dy.code, w.trans, act, M, N, K, dy.ptr, dy.ld, x.ptr, x.ld, w.ptr,
                              w.ld, p[0], p[1], w.trans, p[2]);
    ok = scratch(need, device, &ws, &wp);
  }
  if (ok && w.trans) {      // laid out as w is
    PyObject *v = PyObject_CallMethodNoArgs(r[1], s_t);
    ok = v != NULL;
    if (ok) {
      Py_DECREF(r[1]);
      r[1] = v;
    }
  }
  if (!ok) {
    Py_XDECREF(ws);
    return drop_all(3, r, device);
  }
  WITHOUT_LOCK(f_linear_grad(dy.code, w.trans, act, M, N, K, dy.ptr, dy.ld, x.ptr, x.ld, w.ptr, w.ld,
                             z.ptr, z.ld, p[0], K, p[1], lddw, w.trans, p[2], wp, need, s))
  Py_XDECREF(ws);
  if (rc != TMM_OK) return drop_all(3, r, device);
  if (!want_bias) {
    r[2] = Py_None;
    Py_INCREF(Py_None);
  }
  PyObject *out = PyObject_Vectorcall(t_linear_grads, r, 3, NULL);
  for (int i = 0; i < 3; ++i) Py_DECREF(r[i]);
  Py_DECREF(device);
  return out;
}

/* What the modules hand in, once each: result types, and entry points. */
static PyObject *take(PyObject *const *a, Py_ssize_t n, int objects, PyObject **const *to,
                      int functions, void **const *fn) {
  if (n != 2 || !PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != objects || !PyTuple_Check(a[1]) ||
      PyTuple_GET_SIZE(a[1]) != functions) {
    PyErr_SetString(PyExc_TypeError, "two tuples: objects, addresses");
    return NULL;
  }
  for (int i = 0; i < objects; ++i) {
    *to[i] = PyTuple_GET_ITEM(a[0], i);
    Py_INCREF(*to[i]);
  }
  for (int i = 0; i < functions; ++i) *fn[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[1], i));
  if (PyErr_Occurred()) return NULL;
  Py_RETURN_NONE;
}
static PyObject *start_scores(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  PyObject **const to[2] = {&t_row_routes, &t_row_logprobs};
  void **const fn[4] = {(void **)&f_route, (void **)&f_route_grad, (void **)&f_logprob,
                        (void **)&f_logprob_grad};
  return take(a, n, 2, to, 4, fn);
}
static PyObject *start_linear(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  PyObject **const to[1] = {&t_linear_grads};
  void **const fn[4] = {(void **)&f_linear, (void **)&f_linear_size, (void **)&f_linear_grad,
                        (void **)&f_linear_grad_size};
  return take(a, n, 1, to, 4, fn);
}

static PyMethodDef methods[] = {
    {"start_scores", (PyCFunction)(void (*)(void))start_scores, METH_FASTCALL, NULL},
    {"start_linear", (PyCFunction)(void (*)(void))start_linear, METH_FASTCALL, NULL},
    {"route", (PyCFunction)(void (*)(void))route, METH_FASTCALL, NULL},
    {"route_grad", (PyCFunction)(void (*)(void))route_grad, METH_FASTCALL, NULL},
    {"logprob", (PyCFunction)(void (*)(void))logprob, METH_FASTCALL, NULL},
    {"logprob_grad", (PyCFunction)(void (*)(void))logprob_grad, METH_FASTCALL, NULL},
    {"linear", (PyCFunction)(void (*)(void))linear, METH_FASTCALL, NULL},
    {"linear_grad", (PyCFunction)(void (*)(void))linear_grad, METH_FASTCALL, NULL},
    {"start", (PyCFunction)(void (*)(void))start, METH_FASTCALL, NULL},
    {"grouped", (PyCFunction)(void (*)(void))grouped, METH_FASTCALL, NULL},
    {"wgrad", (PyCFunction)(void (*)(void))wgrad, METH_FASTCALL, NULL},
    {"lora", (PyCFunction)(void (*)(void))lora, METH_FASTCALL, NULL},
    {"group_rows", (PyCFunction)(void (*)(void))group_rows_, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "grouped_call", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_grouped_call(void) {
  PyObject **const names[7] = {&s_dtype, &s_device,   &s_is_cuda,   &s_shape,
                               &s_stride, &s_data_ptr, &s_get_device};
  static const char *const text[7] = {"dtype",  "device",   "is_cuda",   "shape",
                                      "stride", "data_ptr", "get_device"};
  for (int i = 0; i < 7; ++i)
    if ((*names[i] = PyUnicode_InternFromString(text[i])) == NULL) return NULL;
  if ((s_t = PyUnicode_InternFromString("t")) == NULL) return NULL;
  t_kwnames = Py_BuildValue("(OO)", s_dtype, s_device);
  if (t_kwnames == NULL) return NULL;
  return PyModule_Create(&module);
}
