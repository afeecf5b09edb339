/*
 * tq_call.c -- argument marshalling of the norm/rotation, append, attention,
 * adapter and sampling calls for Python, in C: for a few tokens these calls run
 * for 2 to 8 us on the GPU, and the same look at the tensors written in Python
 * took 9.
 *
 * Each function takes the objects of the Python call, checks shapes, types and
 * placement, and calls the C ABI through the address setup() was given. It
 * returns the status code (0, a negative TQ_ERR_*), or kOtherDevice when the
 * tensors are not on the current device; nothing is enqueued in that case.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/tq.h"

enum { kOtherDevice = 1 };

static PyObject *n_shape, *n_stride, *n_dtype, *n_data_ptr, *n_get_device, *n_numel,
    *n_is_contiguous, *n_cuda_stream, *n_element_size;
static PyObject *dtypes[3], *dtype_i32;          /* torch.float32, float16, bfloat16; int32 */
static PyObject *get_device, *current_stream;    /* of the current device; of a device */

typedef int (*qk_fn)(const void *, int64_t, const void *, int64_t, int, void *, int64_t, void *,
                     int64_t, int, int64_t, int64_t, int64_t, int64_t, const float *, const float *,
                     float, const tq_rope *, const int32_t *, void *);
typedef int (*append_fn)(const void *, int64_t, const void *, int64_t, const void *, int64_t, int,
                         void *, int64_t, const tq_paged_kv *, const int32_t *, const int32_t *,
                         int64_t, int64_t, const float *, const float *, float, const tq_rope *,
                         void *);
typedef int (*attend_fn)(const void *, int64_t, const tq_paged_kv *, const int32_t *,
                         const int32_t *, void *, int64_t, int, float *, int64_t, int64_t, int64_t,
                         int64_t, float, int64_t, void *, int64_t, void *);
typedef int (*lora_fn)(const void *, int64_t, int, const tq_lora *, const int32_t *, const void *,
                       int64_t, void *, int64_t, int, int64_t, void *, int64_t, void *);
typedef int (*sample_fn)(const void *, int64_t, int, int64_t, int64_t, const float *, const float *,
                         const int32_t *, const float *, const float *, int32_t *, float *, void *);
static qk_fn call_qk;
static append_fn call_append;
static attend_fn call_attend;
static lora_fn call_lora;
static sample_fn call_sample;

/* A [tokens][heads][head_dim] tensor. */
typedef struct {
  int64_t n, h, d, stride;
  int type;
  void *p;
} rows_t;

/* Results of the helpers: 0, a status code, or kRaised with an exception set. */
enum { kRaised = -1000 };

static int raise_value(const char *what) {
  PyErr_SetString(PyExc_ValueError, what);
  return kRaised;
}

static int read_dims_of(PyObject *size, int64_t *out, int n) {
  if (!size) return kRaised;
  if (!PyTuple_Check(size) || PyTuple_GET_SIZE(size) != n) {
    Py_DECREF(size);
    return TQ_ERR_SHAPE;
  }
  for (int i = 0; i < n; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(size, i));
  Py_DECREF(size);
  return PyErr_Occurred() ? kRaised : 0;
}

static int read_dims(PyObject *size, int64_t out[3]) { return read_dims_of(size, out, 3); }

static int read_shape(PyObject *t, rows_t *r) {
  int64_t d[3] = {0, 0, 0};
  const int rc = read_dims(PyObject_GetAttr(t, n_shape), d);
  r->n = d[0];
  r->h = d[1];
  r->d = d[2];
  return rc;
}

static int type_of(PyObject *t, int *type) {
  PyObject *d = PyObject_GetAttr(t, n_dtype);
  if (!d) return kRaised;
  Py_DECREF(d);   /* torch keeps its dtypes */
  for (int i = 0; i < 3; ++i)
    if (d == dtypes[i]) {
      *type = i;
      return 0;
    }
  return TQ_ERR_TYPE;
}

/* The device of a call's tensors so far, -1 before the first: one more of them. */
static int same_device(int64_t d, int64_t *dev) {
  if (d < 0) return raise_value("tensor must live on a CUDA device");
  if (*dev >= 0 && d != *dev) return raise_value("the tensors must be on one device");
  *dev = d;
  return 0;
}

static int on_device(PyObject *t, int64_t *dev) {
  PyObject *i = PyObject_CallMethodNoArgs(t, n_get_device);
  if (!i) return kRaised;
  const int64_t d = PyLong_AsLongLong(i);
  Py_DECREF(i);
  return PyErr_Occurred() ? kRaised : same_device(d, dev);
}

static int address(PyObject *t, void **p) {
  PyObject *a = PyObject_CallMethodNoArgs(t, n_data_ptr);
  if (!a) return kRaised;
  *p = PyLong_AsVoidPtr(a);
  Py_DECREF(a);
  return PyErr_Occurred() ? kRaised : 0;
}

/* Type, placement, strides and address of a tensor whose shape was read. */
static int read_rows(PyObject *t, rows_t *r, int64_t *dev) {
  int rc = type_of(t, &r->type);
  if (rc) return rc;
  if ((rc = on_device(t, dev))) return rc;
  int64_t s[3];
  if ((rc = read_dims(PyObject_CallMethodNoArgs(t, n_stride), s))) return rc;
  if ((r->d > 1 && s[2] != 1) || (r->h > 1 && s[1] != r->d))
    return raise_value("the heads of a token must be contiguous");
  r->stride = r->n > 1 ? s[0] : r->h * r->d;
  return address(t, &r->p);
}

/* A [rows][values] tensor whose rows are contiguous: h is 1. */
static int read_matrix(PyObject *t, rows_t *r, int64_t *dev) {
  int64_t d[2], s[2];
  int rc = read_dims_of(PyObject_GetAttr(t, n_shape), d, 2);
  if (rc) return rc;
  r->n = d[0];
  r->h = 1;
  r->d = d[1];
  if ((rc = type_of(t, &r->type))) return rc;
  if ((rc = on_device(t, dev))) return rc;
  if ((rc = read_dims_of(PyObject_CallMethodNoArgs(t, n_stride), s, 2))) return rc;
  if (r->d > 1 && s[1] != 1) return raise_value("the values of a row must be contiguous");
  r->stride = r->n > 1 ? s[0] : r->d;
  return address(t, &r->p);
}

/* A contiguous vector of n values of a type, or None. */
static int read_vector(PyObject *t, PyObject *dtype, int64_t n, void **p, int64_t *dev) {
  *p = NULL;
  if (t == Py_None) return 0;
  PyObject *d = PyObject_GetAttr(t, n_dtype);
  if (!d) return kRaised;
  Py_DECREF(d);
  if (d != dtype) return TQ_ERR_TYPE;
  PyObject *c = PyObject_CallMethodNoArgs(t, n_numel);
  if (!c) return kRaised;
  const int64_t count = PyLong_AsLongLong(c);
  Py_DECREF(c);
  if (count != n) return TQ_ERR_SHAPE;
  const int rc = on_device(t, dev);
  if (rc) return rc;
  PyObject *b = PyObject_CallMethodNoArgs(t, n_is_contiguous);
  if (!b) return kRaised;
  Py_DECREF(b);
  if (b != Py_True) return raise_value("tensor must be contiguous");
  return address(t, p);
}

/* The stream's handle: the given one's, or the current one's of the tensors'
 * device, which has to be the current device. */
static int read_stream(int64_t dev, PyObject *stream, void **s) {
  PyObject *cur = PyObject_CallNoArgs(get_device);
  if (!cur) return kRaised;
  const int64_t here = PyLong_AsLongLong(cur);
  PyObject *h = NULL;
  if (here == dev)
    h = stream == Py_None ? PyObject_CallOneArg(current_stream, cur) : PyObject_GetAttr(stream, n_cuda_stream);
  Py_DECREF(cur);
  if (here != dev) return PyErr_Occurred() ? kRaised : kOtherDevice;
  if (!h) return kRaised;
  *s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  return PyErr_Occurred() ? kRaised : 0;
}

/* A contiguous buffer of any type, or None, and its bytes. */
static int read_workspace(PyObject *t, void **p, int64_t *bytes, int64_t *dev) {
  *p = NULL;
  *bytes = 0;
  if (t == Py_None) return 0;
  int rc = on_device(t, dev);
  if (rc) return rc;
  PyObject *b = PyObject_CallMethodNoArgs(t, n_is_contiguous);
  if (!b) return kRaised;
  Py_DECREF(b);
  if (b != Py_True) return raise_value("tensor must be contiguous");
  if ((rc = address(t, p))) return rc;
  PyObject *n = PyObject_CallMethodNoArgs(t, n_numel);
  PyObject *e = n ? PyObject_CallMethodNoArgs(t, n_element_size) : NULL;
  if (e) *bytes = PyLong_AsLongLong(n) * PyLong_AsLongLong(e);
  Py_XDECREF(n);
  Py_XDECREF(e);
  return PyErr_Occurred() ? kRaised : 0;
}

static int same_shape(const rows_t *a, const rows_t *b) {
  return a->n == b->n && a->h == b->h && a->d == b->d;
}

static int read_address(PyObject *o, void **p) {
  *p = o == Py_None ? NULL : PyLong_AsVoidPtr(o);
  return PyErr_Occurred() ? kRaised : 0;
}

/* What the binding's objects point to: the C struct and the device of its tensors. */
typedef struct {
  tq_rope c;
  int64_t device;
} placed_rope;
typedef struct {
  tq_paged_kv c;
  int64_t device;
} placed_kv;
typedef struct {
  tq_lora c;
  int64_t device;
} placed_lora;

static PyObject *result(int rc) { return rc == kRaised ? NULL : PyLong_FromLong(rc); }

#define TRY(x)                        \
  do {                                \
    const int rc_ = (x);              \
    if (rc_) return result(rc_);      \
  } while (0)
#define CHECK(cond, code) \
  do {                    \
    if (!(cond)) return result(code); \
  } while (0)

/* (Xq, Xk, Yq, Yk, positions, rope, q_weight, k_weight, eps, stream) */
static PyObject *qk_norm_rope(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
  (void)self;
  if (nargs != 10) return PyErr_Format(PyExc_TypeError, "10 arguments expected");
  rows_t xq = {0}, xk = {0}, yq = {0}, yk = {0};
  int64_t dev = -1;
  const int keys = a[1] != Py_None;
  TRY(read_shape(a[0], &xq));
  TRY(read_shape(a[2], &yq));
  CHECK(same_shape(&xq, &yq), TQ_ERR_SHAPE);
  if (keys) {
    TRY(read_shape(a[1], &xk));
    TRY(read_shape(a[3], &yk));
    CHECK(same_shape(&xk, &yk) && xk.n == xq.n && xk.d == xq.d, TQ_ERR_SHAPE);
  }
  TRY(read_rows(a[0], &xq, &dev));
  TRY(read_rows(a[2], &yq, &dev));
  if (keys) {
    TRY(read_rows(a[1], &xk, &dev));
    TRY(read_rows(a[3], &yk, &dev));
    CHECK(xk.type == xq.type && yk.type == yq.type, TQ_ERR_TYPE);
  }
  void *pos, *rope, *qw, *kw, *stream;
  TRY(read_vector(a[4], dtype_i32, xq.n, &pos, &dev));
  TRY(read_address(a[5], &rope));
  if (rope) TRY(same_device(((const placed_rope *)rope)->device, &dev));
  TRY(read_vector(a[6], dtypes[0], xq.d, &qw, &dev));
  TRY(read_vector(a[7], dtypes[0], xq.d, &kw, &dev));
  const double eps = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred()) return NULL;
  TRY(read_stream(dev, a[9], &stream));
  return result(call_qk(xq.p, xq.stride, xk.p, xk.stride, xq.type, yq.p, yq.stride, yk.p, yk.stride,
                        yq.type, xq.n, xq.h, xk.h, xq.d, qw, kw, (float)eps, rope, pos, stream));
}

/* (Xq, Xk, Xv, Yq, kv, seq_ids, positions, rope, q_weight, k_weight, eps, stream) */
static PyObject *kv_append(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
  (void)self;
  if (nargs != 12) return PyErr_Format(PyExc_TypeError, "12 arguments expected");
  rows_t xq = {0}, xk = {0}, xv = {0}, yq = {0};
  int64_t dev = -1;
  const int queries = a[0] != Py_None;
  void *kvp;
  TRY(read_address(a[4], &kvp));
  const tq_paged_kv *kv = kvp;
  TRY(read_shape(a[1], &xk));
  TRY(read_shape(a[2], &xv));
  CHECK(same_shape(&xk, &xv) && xk.h == kv->heads && xk.d == kv->head_dim, TQ_ERR_SHAPE);
  if (queries) {
    TRY(read_shape(a[0], &xq));
    TRY(read_shape(a[3], &yq));
    CHECK(same_shape(&xq, &yq) && xq.n == xk.n && xq.d == xk.d, TQ_ERR_SHAPE);
  }
  TRY(read_rows(a[1], &xk, &dev));
  TRY(read_rows(a[2], &xv, &dev));
  CHECK(xv.type == xk.type, TQ_ERR_TYPE);
  if (queries) {
    TRY(read_rows(a[0], &xq, &dev));
    TRY(read_rows(a[3], &yq, &dev));
    CHECK(xq.type == xk.type && yq.type == kv->type, TQ_ERR_TYPE);
  }
  TRY(same_device(((const placed_kv *)kvp)->device, &dev));
  void *seq, *pos, *rope, *qw, *kw, *stream;
  TRY(read_vector(a[5], dtype_i32, xk.n, &seq, &dev));
  TRY(read_vector(a[6], dtype_i32, xk.n, &pos, &dev));
  TRY(read_address(a[7], &rope));
  if (rope) TRY(same_device(((const placed_rope *)rope)->device, &dev));
  TRY(read_vector(a[8], dtypes[0], xk.d, &qw, &dev));
  TRY(read_vector(a[9], dtypes[0], xk.d, &kw, &dev));
  const double eps = PyFloat_AsDouble(a[10]);
  if (PyErr_Occurred()) return NULL;
  TRY(read_stream(dev, a[11], &stream));
  return result(call_append(xq.p, xq.stride, xk.p, xk.stride, xv.p, xv.stride, xk.type, yq.p, yq.stride,
                            kv, seq, pos, xk.n, xq.h, qw, kw, (float)eps, rope, stream));
}

/* (Q, kv, q_start, kv_len, O, max_q, max_kv, scale, workspace, window, lse, stream) */
static PyObject *paged_attention(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
  (void)self;
  if (nargs != 12) return PyErr_Format(PyExc_TypeError, "12 arguments expected");
  rows_t q = {0}, o = {0};
  int64_t dev = -1;
  void *kvp;
  TRY(read_address(a[1], &kvp));
  const tq_paged_kv *kv = kvp;
  TRY(read_shape(a[0], &q));
  TRY(read_shape(a[4], &o));
  CHECK(same_shape(&q, &o) && q.d == kv->head_dim, TQ_ERR_SHAPE);
  TRY(read_rows(a[0], &q, &dev));
  TRY(read_rows(a[4], &o, &dev));
  CHECK(q.type == kv->type, TQ_ERR_TYPE);
  TRY(same_device(((const placed_kv *)kvp)->device, &dev));
  void *start, *len, *ws, *lse, *stream;
  TRY(read_vector(a[2], dtype_i32, kv->nseq + 1, &start, &dev));
  TRY(read_vector(a[3], dtype_i32, kv->nseq, &len, &dev));
  TRY(read_vector(a[10], dtypes[0], q.n * q.h, &lse, &dev));
  const int64_t max_q = PyLong_AsLongLong(a[5]), max_kv = PyLong_AsLongLong(a[6]);
  const double scale = PyFloat_AsDouble(a[7]);
  const int64_t window = PyLong_AsLongLong(a[9]);
  if (PyErr_Occurred()) return NULL;
  int64_t ws_bytes;
  TRY(read_workspace(a[8], &ws, &ws_bytes, &dev));
  TRY(read_stream(dev, a[11], &stream));
  return result(call_attend(q.p, q.stride, kv, start, len, o.p, o.stride, o.type, lse, q.n, q.h, max_q,
                            max_kv, (float)scale, window, ws, ws_bytes, stream));
}

/* (X, lora, ids, Y, Z, workspace, stream) */
static PyObject *lora_add(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
  (void)self;
  if (nargs != 7) return PyErr_Format(PyExc_TypeError, "7 arguments expected");
  rows_t x = {0}, y = {0}, z = {0};
  int64_t dev = -1;
  void *lp;
  TRY(read_address(a[1], &lp));
  const tq_lora *l = lp;
  const int base = a[4] != Py_None;
  TRY(read_matrix(a[0], &x, &dev));
  TRY(read_matrix(a[3], &y, &dev));
  CHECK(x.n == y.n && x.d == l->cols && y.d == l->rows, TQ_ERR_SHAPE);
  if (base) {
    TRY(read_matrix(a[4], &z, &dev));
    CHECK(same_shape(&z, &y), TQ_ERR_SHAPE);
    CHECK(z.type == y.type, TQ_ERR_TYPE);
  }
  TRY(same_device(((const placed_lora *)lp)->device, &dev));
  void *ids, *ws, *stream;
  int64_t ws_bytes;
  TRY(read_vector(a[2], dtype_i32, x.n, &ids, &dev));
  TRY(read_workspace(a[5], &ws, &ws_bytes, &dev));
  TRY(read_stream(dev, a[6], &stream));
  return result(call_lora(x.p, x.stride, x.type, l, ids, z.p, z.stride, y.p, y.stride, y.type, x.n, ws,
                          ws_bytes, stream));
}

/* (logits, u, tokens, temperature, top_k, top_p, min_p, logp, stream) */
static PyObject *sample(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
  (void)self;
  if (nargs != 9) return PyErr_Format(PyExc_TypeError, "9 arguments expected");
  rows_t x = {0};
  int64_t dev = -1;
  TRY(read_matrix(a[0], &x, &dev));
  void *u, *tokens, *temperature, *top_k, *top_p, *min_p, *logp, *stream;
  TRY(read_vector(a[1], dtypes[0], x.n, &u, &dev));
  TRY(read_vector(a[2], dtype_i32, x.n, &tokens, &dev));
  TRY(read_vector(a[3], dtypes[0], x.n, &temperature, &dev));
  TRY(read_vector(a[4], dtype_i32, x.n, &top_k, &dev));
  TRY(read_vector(a[5], dtypes[0], x.n, &top_p, &dev));
  TRY(read_vector(a[6], dtypes[0], x.n, &min_p, &dev));
  TRY(read_vector(a[7], dtypes[0], x.n, &logp, &dev));
  TRY(read_stream(dev, a[8], &stream));
  return result(call_sample(x.p, x.stride, x.type, x.n, x.d, u, temperature, top_k, top_p, min_p, tokens,
                            logp, stream));
}

/* ((float32, float16, bfloat16, int32), get_device, current_stream, (five addresses)) */
static PyObject *setup(PyObject *self, PyObject *args) {
  (void)self;
  PyObject *types[4], *dev, *str;
  unsigned long long fn[5];
  if (!PyArg_ParseTuple(args, "(OOOO)OO(KKKKK)", &types[0], &types[1], &types[2], &types[3], &dev, &str,
                        &fn[0], &fn[1], &fn[2], &fn[3], &fn[4]))
    return NULL;
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(types[i]);
    dtypes[i] = types[i];
  }
  Py_INCREF(types[3]);
  dtype_i32 = types[3];
  Py_INCREF(dev);
  get_device = dev;
  Py_INCREF(str);
  current_stream = str;
  call_qk = (qk_fn)(uintptr_t)fn[0];
  call_append = (append_fn)(uintptr_t)fn[1];
  call_attend = (attend_fn)(uintptr_t)fn[2];
  call_lora = (lora_fn)(uintptr_t)fn[3];
  call_sample = (sample_fn)(uintptr_t)fn[4];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, NULL},
    {"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, NULL},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, NULL},
    {"paged_attention", (PyCFunction)(void (*)(void))paged_attention, METH_FASTCALL, NULL},
    {"lora_add", (PyCFunction)(void (*)(void))lora_add, METH_FASTCALL, NULL},
    {"sample", (PyCFunction)(void (*)(void))sample, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tq_call", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__tq_call(void) {
  const struct {
    PyObject **at;
    const char *name;
  } names[] = {{&n_shape, "shape"}, {&n_stride, "stride"}, {&n_dtype, "dtype"},
               {&n_data_ptr, "data_ptr"}, {&n_get_device, "get_device"},
               {&n_numel, "numel"}, {&n_is_contiguous, "is_contiguous"},
               {&n_cuda_stream, "cuda_stream"}, {&n_element_size, "element_size"}};
  for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
    if (!(*names[i].at = PyUnicode_InternFromString(names[i].name))) return NULL;
  return PyModule_Create(&module);
}
