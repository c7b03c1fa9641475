/* grouped_call.c -- the usual calls of the grouped operators, from torch tensors to the C ABI.
 *
 * The operators of a decode step take a few microseconds on the GPU; describing their tensors in
 * Python takes longer than that.  This CPython module does it for the usual case -- torch CUDA
 * tensors of the right types on the current device, outputs and workspace allocated here -- and
 * returns None for every other, which grouped.py then handles (and reports) in full.  It holds no
 * arithmetic and no torch headers: tensors are read through their Python attributes, and the
 * entry points' addresses are handed in.
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

static PyMethodDef methods[] = {
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
  t_kwnames = Py_BuildValue("(OO)", s_dtype, s_device);
  if (t_kwnames == NULL) return NULL;
  return PyModule_Create(&module);
}
