/* Python binding of the residual block's norms and of gradient clipping, by
 * the CPython C API.
 *
 * These calls are small: with the tensors described in Python, their
 * arguments took longer than the kernels of a decode step (6 us for two
 * tensors and a launch, 15 us for the post norm's backward).  The module does
 * what the ctypes functions beside it do -- check each tensor's type, device,
 * shape and strides, take its address, call the library with the current
 * stream -- on the same library: _lib.py hands it the loaded functions'
 * addresses.  It knows of torch what Python knows: attributes and methods.
 *
 * Every function returns the library's status, or raises ValueError for a
 * tensor that it cannot describe. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>
#include <stdio.h>
#include <string.h>

#include "moe.h"

static struct {
  __typeof__(&moe_block_pre_norm_fwd) pre_fwd;
  __typeof__(&moe_block_pre_norm_bwd) pre_bwd;
  __typeof__(&moe_block_post_norm_fwd) post_fwd;
  __typeof__(&moe_block_post_norm_bwd) post_bwd;
  __typeof__(&moe_grad_norm) grad_norm;
  __typeof__(&moe_clip_grads) clip;
} lib;

static struct {
  PyObject *bf16, *f32, *i32;                 /* torch dtypes */
  PyObject *data_ptr, *stride, *numel, *element_size, *is_contiguous; /* torch.Tensor's methods */
  PyObject *raw_stream, *device;              /* torch._C functions */
  PyObject *s_dtype, *s_is_cuda, *s_shape, *s_cuda_stream;
  PyObject *k_pre_w, *k_pre_b, *k_post_w, *k_post_b, *k_gate, *k_row_of, *k_topk_w, *k_y_out;
} py;

/* ---------------------------------------------------------- one tensor */
static int call_long(PyObject* method, PyObject* t, long long* out) {
  PyObject* r = PyObject_Vectorcall(method, &t, 1, NULL);
  if (!r) return -1;
  *out = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int address(PyObject* t, void** out) {
  PyObject* r = PyObject_Vectorcall(py.data_ptr, &t, 1, NULL);
  if (!r) return -1;
  *out = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return !*out && PyErr_Occurred() ? -1 : 0;
}

static PyObject* dtype_of(int t) { return t == MOE_DTYPE_FP32 ? py.f32 : py.bf16; }

/* Fails unless t is a CUDA tensor of the type. */
static int check_type(PyObject* t, PyObject* dtype) {
  PyObject* have = PyObject_GetAttr(t, py.s_dtype);
  if (!have) return -1;
  PyObject* cuda = PyObject_GetAttr(t, py.s_is_cuda);
  if (!cuda) {
    Py_DECREF(have);
    return -1;
  }
  const int ok = have == dtype && cuda == Py_True;
  if (!ok)
    PyErr_Format(PyExc_ValueError, "expected a %S CUDA tensor, got %S%s", dtype, have,
                 cuda == Py_True ? "" : " on another device");
  Py_DECREF(have);
  Py_DECREF(cuda);
  return ok ? 0 : -1;
}

/* Sizes (or strides) of a tuple of two, or -1. */
static int two(PyObject* tuple, long long* a, long long* b) {
  if (!PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) != 2) return -1;
  *a = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, 0));
  *b = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, 1));
  return PyErr_Occurred() ? -1 : 0;
}

/* An [n, d] tensor (n < 0: any number of rows, given back in *rows) with unit
 * stride along the channels; None gives no rows. */
static int get_rows(PyObject* t, long long n, long long d, PyObject* dtype, moe_rows_t* out,
                    long long* rows) {
  out->p = NULL;
  out->ld = 0;
  if (!t || t == Py_None) return 0;
  if (check_type(t, dtype) < 0) return -1;
  PyObject* shape = PyObject_GetAttr(t, py.s_shape);
  if (!shape) return -1;
  long long a = -1, b = -1;
  const int ok = two(shape, &a, &b) == 0 && (n < 0 || a == n) && b == d;
  if (!ok && !PyErr_Occurred())
    PyErr_Format(PyExc_ValueError, "expected a tensor of shape (%lld, %lld), got %S", n, d, shape);
  Py_DECREF(shape);
  if (!ok) return -1;
  PyObject* strides = PyObject_Vectorcall(py.stride, &t, 1, NULL);
  if (!strides) return -1;
  long long ld = 0, step = 0;
  const int fine = two(strides, &ld, &step) == 0 && (step == 1 || d <= 1) && (ld >= d || a <= 1);
  if (!fine && !PyErr_Occurred())
    PyErr_Format(PyExc_ValueError, "rows must be contiguous and apart, got strides %S", strides);
  Py_DECREF(strides);
  if (!fine) return -1;
  out->ld = a > 1 || ld > d ? ld : d;
  if (rows) *rows = a;
  return address(t, &out->p);
}

/* A contiguous tensor of n values of the type (n < 0: any number). */
static int get_vector(PyObject* t, long long n, PyObject* dtype, void** out) {
  *out = NULL;
  if (!t || t == Py_None) return 0;
  long long have;
  if (check_type(t, dtype) < 0 || call_long(py.numel, t, &have) < 0) return -1;
  PyObject* c = PyObject_Vectorcall(py.is_contiguous, &t, 1, NULL);
  if (!c) return -1;
  const int ok = c == Py_True && (n < 0 || have == n);
  Py_DECREF(c);
  if (!ok) {
    PyErr_Format(PyExc_ValueError, "expected a contiguous tensor of %lld values, got %lld", n, have);
    return -1;
  }
  return address(t, out);
}

/* A contiguous CUDA buffer of any type. */
static int get_buffer(PyObject* t, void** out, size_t* bytes) {
  long long n, size;
  PyObject* cuda = PyObject_GetAttr(t, py.s_is_cuda);
  if (!cuda) return -1;
  PyObject* c = PyObject_Vectorcall(py.is_contiguous, &t, 1, NULL);
  const int ok = cuda == Py_True && c == Py_True;
  Py_DECREF(cuda);
  Py_XDECREF(c);
  if (!c) return -1;
  if (!ok) {
    PyErr_SetString(PyExc_ValueError, "tensors passed to libmoe must be contiguous CUDA tensors");
    return -1;
  }
  if (call_long(py.numel, t, &n) < 0 || call_long(py.element_size, t, &size) < 0) return -1;
  *bytes = (size_t)(n * size);
  return address(t, out);
}

/* ------------------------------------------------------------ the call */
static int get_stream(PyObject* stream, cudaStream_t* out) {
  PyObject* r;
  if (stream == Py_None) {
    PyObject* dev = PyObject_Vectorcall(py.device, NULL, 0, NULL);
    if (!dev) return -1;
    r = PyObject_Vectorcall(py.raw_stream, &dev, 1, NULL);
    Py_DECREF(dev);
  } else {
    r = PyObject_GetAttr(stream, py.s_cuda_stream);
  }
  if (!r) return -1;
  *out = (cudaStream_t)PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return PyErr_Occurred() ? -1 : 0;
}

/* The descriptor's bytes (a ctypes structure), copied. */
static int get_desc(PyObject* o, moe_block_norm_desc_t* d) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) < 0) return -1;
  const int ok = b.len == (Py_ssize_t)sizeof(*d);
  if (ok) memcpy(d, b.buf, sizeof(*d));
  PyBuffer_Release(&b);
  if (!ok) PyErr_SetString(PyExc_ValueError, "expected a moe_block_norm_desc_t");
  return ok ? 0 : -1;
}

/* dict of optional tensors {pre_w, pre_b, post_w, post_b, gate}. */
static int get_params(PyObject* p, const moe_block_norm_desc_t* d, moe_block_params_t* out) {
  PyObject* dt = dtype_of(d->param_dtype);
  memset(out, 0, sizeof(*out));
  if (!PyDict_Check(p)) {
    PyErr_SetString(PyExc_TypeError, "expected a dict of parameters");
    return -1;
  }
  if (get_vector(PyDict_GetItem(p, py.k_pre_w), d->d, dt, &out->pre_w) < 0 ||
      get_vector(PyDict_GetItem(p, py.k_pre_b), d->d, dt, &out->pre_b) < 0 ||
      get_vector(PyDict_GetItem(p, py.k_post_w), d->d, dt, &out->post_w) < 0 ||
      get_vector(PyDict_GetItem(p, py.k_post_b), d->d, dt, &out->post_b) < 0)
    return -1;
  PyObject* g = PyDict_GetItem(p, py.k_gate);
  if (!g || g == Py_None || d->gate == MOE_GATE_NONE) return 0;
  if (d->gate == MOE_GATE_CHANNEL) return get_vector(g, d->d, dt, &out->gate.p);
  if (d->gate == MOE_GATE_FULL)
    return get_rows(g, d->T, d->d, dtype_of(d->dtype), &out->gate, NULL);
  if (check_type(g, py.f32) < 0) return -1;
  PyObject* strides = PyObject_Vectorcall(py.stride, &g, 1, NULL);
  if (!strides) return -1;
  long long n = 0, step = -1;
  if (PyTuple_GET_SIZE(strides) == 1) step = PyLong_AsLongLong(PyTuple_GET_ITEM(strides, 0));
  Py_DECREF(strides);
  if (call_long(py.numel, g, &n) < 0) return -1;
  if (step < 0 || n != d->T || (step < 1 && d->T > 1)) {
    PyErr_Format(PyExc_ValueError, "expected an fp32 gate of %d tokens, apart from each other",
                 (int)d->T);
    return -1;
  }
  out->gate.ld = step < 1 ? 1 : step;
  return address(g, &out->gate.p);
}

static int want(Py_ssize_t have, Py_ssize_t n) {
  if (have == n) return 0;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", n, have);
  return -1;
}

#define CALL(status, expression) \
  do {                           \
    Py_BEGIN_ALLOW_THREADS       \
    status = (expression);       \
    Py_END_ALLOW_THREADS         \
  } while (0)

/* desc, res, w, b, x, stream */
static PyObject* pre_norm_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  moe_block_norm_desc_t d;
  moe_rows_t res, x;
  void *w, *b;
  cudaStream_t s;
  int st;
  (void)self;
  if (want(n, 6) < 0 || get_desc(a[0], &d) < 0) return NULL;
  PyObject* dt = dtype_of(d.param_dtype);
  if (get_rows(a[1], d.T, d.d, dtype_of(d.res_dtype), &res, NULL) < 0 ||
      get_vector(a[2], d.d, dt, &w) < 0 || get_vector(a[3], d.d, dt, &b) < 0 ||
      get_rows(a[4], d.T, d.d, dtype_of(d.dtype), &x, NULL) < 0 || get_stream(a[5], &s) < 0)
    return NULL;
  CALL(st, lib.pre_fwd(&d, res, w, b, x, s));
  return PyLong_FromLong(st);
}

/* desc, dx, res, w, dres_in, dres, dw, db, ws, dres_scale, stream */
static PyObject* pre_norm_bwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  moe_block_norm_desc_t d;
  moe_rows_t dx, res, dres_in, dres;
  void *w, *dw, *db, *ws;
  size_t bytes;
  cudaStream_t s;
  int st;
  (void)self;
  if (want(n, 11) < 0 || get_desc(a[0], &d) < 0) return NULL;
  PyObject *dt = dtype_of(d.param_dtype), *rt = dtype_of(d.res_dtype);
  const double scale = PyFloat_AsDouble(a[9]);
  if (PyErr_Occurred()) return NULL;
  if (get_rows(a[1], d.T, d.d, dtype_of(d.dtype), &dx, NULL) < 0 ||
      get_rows(a[2], d.T, d.d, rt, &res, NULL) < 0 || get_vector(a[3], d.d, dt, &w) < 0 ||
      get_rows(a[4], d.T, d.d, rt, &dres_in, NULL) < 0 ||
      get_rows(a[5], d.T, d.d, rt, &dres, NULL) < 0 || get_vector(a[6], d.d, dt, &dw) < 0 ||
      get_vector(a[7], d.d, dt, &db) < 0 || get_buffer(a[8], &ws, &bytes) < 0 ||
      get_stream(a[10], &s) < 0)
    return NULL;
  CALL(st, lib.pre_bwd(&d, dx, res, w, dres_in, (float)scale, dres, dw, db, ws, bytes, s));
  return PyLong_FromLong(st);
}

/* desc, res, y, params, res_out, x, routed, stream */
static PyObject* post_norm_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  moe_block_norm_desc_t d;
  moe_rows_t res, y, res_out, x;
  moe_block_params_t p;
  moe_routed_rows_t r;
  cudaStream_t s;
  int st;
  const int routed = n > 6 && a[6] != Py_None;
  (void)self;
  if (want(n, 8) < 0 || get_desc(a[0], &d) < 0) return NULL;
  PyObject *at = dtype_of(d.dtype), *rt = dtype_of(d.res_dtype);
  long long capacity = d.T;
  if (get_rows(a[1], d.T, d.d, rt, &res, NULL) < 0 ||
      get_rows(a[2], routed ? -1 : d.T, d.d, at, &y, &capacity) < 0 ||
      get_params(a[3], &d, &p) < 0 || get_rows(a[4], d.T, d.d, rt, &res_out, NULL) < 0 ||
      get_rows(a[5], d.T, d.d, at, &x, NULL) < 0 || get_stream(a[7], &s) < 0)
    return NULL;
  if (routed) {
    if (!PyDict_Check(a[6])) {
      PyErr_SetString(PyExc_TypeError, "expected a dict of routed rows");
      return NULL;
    }
    PyObject *row_of = PyDict_GetItem(a[6], py.k_row_of), *w = PyDict_GetItem(a[6], py.k_topk_w);
    if (!row_of || !w) {
      PyErr_SetString(PyExc_ValueError, "routed rows need row_of and topk_w");
      return NULL;
    }
    PyObject* shape = PyObject_GetAttr(row_of, py.s_shape);
    if (!shape) return NULL;
    long long rows = -1, k = -1;
    const int ok = two(shape, &rows, &k) == 0 && rows == d.T && k <= INT_MAX && capacity <= INT_MAX;
    Py_DECREF(shape);
    if (!ok) {
      if (!PyErr_Occurred())
        PyErr_SetString(PyExc_ValueError, "row_of must be int32 [T,k] and topk_w fp32 [T,k]");
      return NULL;
    }
    void *rp, *wp;
    if (get_vector(row_of, rows * k, py.i32, &rp) < 0 || get_vector(w, rows * k, py.f32, &wp) < 0 ||
        get_rows(PyDict_GetItem(a[6], py.k_y_out), d.T, d.d, at, &r.y_out, NULL) < 0)
      return NULL;
    r.row_of = rp;
    r.topk_w = wp;
    r.k = (int32_t)k;
    r.capacity = (int32_t)capacity;
  }
  CALL(st, lib.post_fwd(&d, res, y, &p, res_out, x, routed ? &r : NULL, s));
  return PyLong_FromLong(st);
}

/* desc, dres_in, dx, res_out, y, params, dres, dy, grads, ws, dres_scale, stream */
static PyObject* post_norm_bwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  moe_block_norm_desc_t d;
  moe_rows_t dres_in, dx, res_out, y, dres, dy;
  moe_block_params_t p, g;
  void* ws;
  size_t bytes;
  cudaStream_t s;
  int st;
  (void)self;
  if (want(n, 12) < 0 || get_desc(a[0], &d) < 0) return NULL;
  PyObject *at = dtype_of(d.dtype), *rt = dtype_of(d.res_dtype);
  const double scale = PyFloat_AsDouble(a[10]);
  if (PyErr_Occurred()) return NULL;
  if (get_rows(a[1], d.T, d.d, rt, &dres_in, NULL) < 0 ||
      get_rows(a[2], d.T, d.d, at, &dx, NULL) < 0 ||
      get_rows(a[3], d.T, d.d, rt, &res_out, NULL) < 0 ||
      get_rows(a[4], d.T, d.d, at, &y, NULL) < 0 || get_params(a[5], &d, &p) < 0 ||
      get_rows(a[6], d.T, d.d, rt, &dres, NULL) < 0 ||
      get_rows(a[7], d.T, d.d, at, &dy, NULL) < 0 || get_params(a[8], &d, &g) < 0 ||
      get_buffer(a[9], &ws, &bytes) < 0 || get_stream(a[11], &s) < 0)
    return NULL;
  CALL(st, lib.post_bwd(&d, dres_in, (float)scale, dx, res_out, y, &p, dres, dy, &g, ws, bytes, s));
  return PyLong_FromLong(st);
}

/* -------------------------------------------------------- gradient lists */
/* The list's descriptions (a ctypes array of moe_grad_t). */
static int get_grads(PyObject* o, Py_buffer* b, Py_ssize_t n) {
  if (PyObject_GetBuffer(o, b, PyBUF_SIMPLE) < 0) return -1;
  if (b->len >= n * (Py_ssize_t)sizeof(moe_grad_t)) return 0;
  PyBuffer_Release(b);
  PyErr_SetString(PyExc_ValueError, "expected an array of moe_grad_t");
  return -1;
}

/* Whether t is n contiguous elements (layout None), or has the shape and strides
 * of the layout (a tuple of both); -1 on failure. */
static int has_layout(PyObject* t, PyObject* layout, long long n) {
  if (layout == Py_None) {
    long long have;
    if (call_long(py.numel, t, &have) < 0) return -1;
    if (have != n) return 0;
    PyObject* c = PyObject_Vectorcall(py.is_contiguous, &t, 1, NULL);
    if (!c) return -1;
    Py_DECREF(c);
    return c == Py_True;
  }
  PyObject* shape = PyObject_GetAttr(t, py.s_shape);
  if (!shape) return -1;
  int same = PyObject_RichCompareBool(shape, PyTuple_GET_ITEM(layout, 0), Py_EQ);
  Py_DECREF(shape);
  if (same <= 0) return same;
  PyObject* strides = PyObject_Vectorcall(py.stride, &t, 1, NULL);
  if (!strides) return -1;
  same = PyObject_RichCompareBool(strides, PyTuple_GET_ITEM(layout, 1), Py_EQ);
  Py_DECREF(strides);
  return same;
}

/* Whether t is still the tensor at p of the type and layout; -1 on failure. */
static int is_still(PyObject* t, const void* p, int type, PyObject* layout, long long n) {
  void* at;
  if (address(t, &at) < 0) return -1;
  if (at != p) return 0;
  PyObject* dtype = PyObject_GetAttr(t, py.s_dtype);
  if (!dtype) return -1;
  const int same = dtype == dtype_of(type);
  Py_DECREF(dtype);
  return same ? has_layout(t, layout, n) : 0;
}

/* array, tensors, outs or None, layouts (pairs of None or (shape, strides), of
 * the tensor and its out): whether every tensor is what the array says. */
static PyObject* in_place(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Py_buffer b;
  (void)self;
  if (want(n, 4) < 0) return NULL;
  if (!PyList_Check(a[1]) || (a[2] != Py_None && !PyList_Check(a[2])) || !PyList_Check(a[3])) {
    PyErr_SetString(PyExc_TypeError, "expected lists of tensors and layouts");
    return NULL;
  }
  const Py_ssize_t count = PyList_GET_SIZE(a[1]);
  const int outs = a[2] != Py_None;
  if ((outs && PyList_GET_SIZE(a[2]) != count) || PyList_GET_SIZE(a[3]) != count) Py_RETURN_FALSE;
  if (get_grads(a[0], &b, count) < 0) return NULL;
  const moe_grad_t* g = b.buf;
  int same = 1;
  for (Py_ssize_t i = 0; i < count && same > 0; ++i) {
    PyObject* pair = PyList_GET_ITEM(a[3], i);
    const long long elements = (long long)(g[i].rows * g[i].cols);
    same = is_still(PyList_GET_ITEM(a[1], i), g[i].grad, g[i].dtype, PyTuple_GET_ITEM(pair, 0),
                    elements);
    if (outs && same > 0)
      same = is_still(PyList_GET_ITEM(a[2], i), g[i].out, g[i].out_dtype, PyTuple_GET_ITEM(pair, 1),
                      elements);
  }
  PyBuffer_Release(&b);
  if (same < 0) return NULL;
  return PyBool_FromLong(same);
}

/* array, n, norm_type, norm, norms, ws, stream */
static PyObject* grad_norm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Py_buffer b;
  void *norm, *norms, *ws;
  size_t bytes;
  cudaStream_t s;
  int st;
  (void)self;
  if (want(n, 7) < 0) return NULL;
  const long count = PyLong_AsLong(a[1]), type = PyLong_AsLong(a[2]);
  if (PyErr_Occurred()) return NULL;
  if (a[3] == Py_None) {
    PyErr_SetString(PyExc_ValueError, "norm must be one fp32 value");
    return NULL;
  }
  if (get_vector(a[3], 1, py.f32, &norm) < 0 || get_vector(a[4], count, py.f32, &norms) < 0 ||
      get_buffer(a[5], &ws, &bytes) < 0 || get_stream(a[6], &s) < 0 ||
      get_grads(a[0], &b, count) < 0)
    return NULL;
  CALL(st, lib.grad_norm(b.buf, (int32_t)count, (int32_t)type, norm, norms, ws, bytes, s));
  PyBuffer_Release(&b);
  return PyLong_FromLong(st);
}

/* array, n, norm, max_norm, eps, stream */
static PyObject* clip_grads(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Py_buffer b;
  void* norm;
  cudaStream_t s;
  int st;
  (void)self;
  if (want(n, 6) < 0) return NULL;
  const long count = PyLong_AsLong(a[1]);
  const double most = PyFloat_AsDouble(a[3]), eps = PyFloat_AsDouble(a[4]);
  if (PyErr_Occurred()) return NULL;
  if (a[2] == Py_None) {
    PyErr_SetString(PyExc_ValueError, "norm must be one fp32 value");
    return NULL;
  }
  if (get_vector(a[2], 1, py.f32, &norm) < 0 || get_stream(a[5], &s) < 0 ||
      get_grads(a[0], &b, count) < 0)
    return NULL;
  CALL(st, lib.clip(b.buf, (int32_t)count, norm, (float)most, (float)eps, s));
  PyBuffer_Release(&b);
  return PyLong_FromLong(st);
}

/* ------------------------------------------------------------- the module */
/* The object at `path` (names between dots) from `from`. */
static PyObject* attr(PyObject* from, const char* path) {
  char name[64];
  PyObject* o = from;
  Py_INCREF(o);
  while (o && *path) {
    const size_t n = strcspn(path, ".");
    snprintf(name, sizeof(name), "%.*s", (int)n, path);
    PyObject* next = PyObject_GetAttrString(o, name);
    Py_DECREF(o);
    o = next;
    path += n + (path[n] == '.');
  }
  return o;
}

/* torch, the six functions' addresses in the order of `lib` */
static PyObject* setup(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (want(n, 7) < 0) return NULL;
  struct {
    PyObject** to;
    const char* path;
  } found[] = {{&py.bf16, "bfloat16"},
               {&py.f32, "float32"},
               {&py.i32, "int32"},
               {&py.data_ptr, "Tensor.data_ptr"},
               {&py.stride, "Tensor.stride"},
               {&py.numel, "Tensor.numel"},
               {&py.element_size, "Tensor.element_size"},
               {&py.is_contiguous, "Tensor.is_contiguous"},
               {&py.raw_stream, "_C._cuda_getCurrentRawStream"},
               {&py.device, "cuda.current_device"}};
  for (size_t i = 0; i < sizeof(found) / sizeof(found[0]); ++i) {
    PyObject* o = attr(a[0], found[i].path);
    if (!o) return NULL;
    Py_XSETREF(*found[i].to, o);
  }
  void* f[6];
  for (int i = 0; i < 6; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function's address is missing");
      return NULL;
    }
  }
  memcpy(&lib, f, sizeof(lib));
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, NULL},
    {"pre_norm_fwd", (PyCFunction)(void (*)(void))pre_norm_fwd, METH_FASTCALL, NULL},
    {"pre_norm_bwd", (PyCFunction)(void (*)(void))pre_norm_bwd, METH_FASTCALL, NULL},
    {"post_norm_fwd", (PyCFunction)(void (*)(void))post_norm_fwd, METH_FASTCALL, NULL},
    {"post_norm_bwd", (PyCFunction)(void (*)(void))post_norm_bwd, METH_FASTCALL, NULL},
    {"in_place", (PyCFunction)(void (*)(void))in_place, METH_FASTCALL, NULL},
    {"grad_norm", (PyCFunction)(void (*)(void))grad_norm, METH_FASTCALL, NULL},
    {"clip_grads", (PyCFunction)(void (*)(void))clip_grads, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  struct {
    PyObject** to;
    const char* text;
  } names[] = {{&py.s_dtype, "dtype"},     {&py.s_is_cuda, "is_cuda"},
               {&py.s_shape, "shape"},     {&py.s_cuda_stream, "cuda_stream"},
               {&py.k_pre_w, "pre_w"},     {&py.k_pre_b, "pre_b"},
               {&py.k_post_w, "post_w"},   {&py.k_post_b, "post_b"},
               {&py.k_gate, "gate"},       {&py.k_row_of, "row_of"},
               {&py.k_topk_w, "topk_w"},   {&py.k_y_out, "y_out"}};
  for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i) {
    *names[i].to = PyUnicode_InternFromString(names[i].text);
    if (!*names[i].to) return NULL;
  }
  return PyModule_Create(&module);
}
