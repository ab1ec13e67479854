/* pycall.c -- the Python binding's checks and calls, for operators whose work on the GPU
 * is shorter than the same checks take in Python (a decode step's plan, its rotation).
 *
 * Each function takes the tensors of one call, checks them (dtype, device, contiguous,
 * shape) and calls the library.  It returns the library's status, or -1 when a tensor
 * is not what it has to be: the caller then finds out in Python what to say about it.
 * Nothing but the CPython C API: a tensor is an object with the attributes that it has
 * in Python.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "pkv.h"

static pkv_status (*plan_step_fn)(const int32_t *, const int32_t *, const int32_t *, int32_t *,
                                  int32_t *, const int32_t *, int32_t *, int32_t *, int32_t *,
                                  int32_t *, int32_t *, int32_t *, int, int64_t, int, int, int64_t,
                                  int64_t, int32_t *, void *);
static pkv_status (*norm_rope_fn)(uint16_t *, uint16_t *, const uint16_t *, const uint16_t *,
                                  const uint16_t *, uint16_t *, uint16_t *, const int32_t *,
                                  const int32_t *, const uint64_t *, const uint16_t *,
                                  const uint16_t *, int64_t, int, int, int, int64_t, int64_t,
                                  int64_t, int, int, float, float, int64_t, int, int32_t *,
                                  void *);
static pkv_status (*shared_attn_fn)(uint16_t *, const uint16_t *, const uint16_t *,
                                    const uint16_t *, const int32_t *, const int32_t *,
                                    const int32_t *, const int32_t *, int, int, int, int, int, int,
                                    int, int64_t, float, void *, size_t, int32_t *, void *);

static PyObject *bf16, *i32, *i64, *u8; /* torch's dtypes */
static PyObject *s_dtype, *s_get_device, *s_is_contiguous, *s_shape, *s_data_ptr, *s_stride, *s_dim,
    *s_numel;

/* Whether t's attribute `name` is, or its method `name` returns, a whole number; there. */
static int method_long(PyObject *t, PyObject *name, long long *x) {
  PyObject *r = PyObject_CallMethodNoArgs(t, name);
  if (r == NULL) return 0;
  *x = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return !(*x == -1 && PyErr_Occurred());
}

static int dims_of(PyObject *t, int ndim, long long *dims) {
  PyObject *shape = PyObject_GetAttr(t, s_shape);
  int ok = shape != NULL && PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == ndim;
  for (int i = 0; ok && i < ndim; ++i) {
    dims[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
    ok = dims[i] >= 0;
  }
  Py_XDECREF(shape);
  return ok;
}

/* A tensor of a dtype, on device dev; its dims and address.  strides: NULL for one that
 * has to be contiguous.  0 (without an exception) when it is anything else. */
static int tensor(PyObject *t, PyObject *dtype, long long dev, int ndim, long long *dims,
                  long long *strides, void **ptr) {
  int ok;
  long long x;
  PyObject *r = PyObject_GetAttr(t, s_dtype);
  ok = r == dtype;
  Py_XDECREF(r);
  if (ok) ok = method_long(t, s_get_device, &x) && x == dev;
  if (ok) ok = dims_of(t, ndim, dims);
  if (ok && strides == NULL) {
    r = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    ok = r == Py_True;
    Py_XDECREF(r);
  } else if (ok) {
    r = PyObject_CallMethodNoArgs(t, s_stride);
    ok = r != NULL && PyTuple_Check(r) && PyTuple_GET_SIZE(r) == ndim;
    for (int i = 0; ok && i < ndim; ++i) strides[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(r, i));
    Py_XDECREF(r);
  }
  if (ok) {
    r = PyObject_CallMethodNoArgs(t, s_data_ptr);
    ok = r != NULL;
    if (ok) *ptr = PyLong_AsVoidPtr(r);
    Py_XDECREF(r);
  }
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return 0;
  }
  return ok;
}

/* The same with its dims given, or none at all (a NULL pointer) for None. */
static int of_shape(PyObject *t, PyObject *dtype, long long dev, int ndim, long long d0,
                    long long d1, long long d2, long long d3, void **ptr) {
  const long long want[4] = {d0, d1, d2, d3};
  long long dims[4];
  if (!tensor(t, dtype, dev, ndim, dims, NULL, ptr)) return 0;
  for (int i = 0; i < ndim; ++i)
    if (dims[i] != want[i]) return 0;
  return 1;
}

/* dev_status: None, or of any shape with something in it. */
static int status_of(PyObject *t, long long dev, void **ptr) {
  long long x[8], numel, ndim;
  *ptr = NULL;
  if (t == Py_None) return 1;
  if (!method_long(t, s_dim, &ndim) || !method_long(t, s_numel, &numel)) {
    PyErr_Clear();
    return 0;
  }
  return ndim <= 8 && numel > 0 && tensor(t, i32, dev, (int)ndim, x, NULL, ptr);
}

/* A whole number as an argument of the library: what does not fit stays too large or
 * becomes -1 (refused there), instead of wrapping around.  0 with an exception set when
 * it is none. */
static int number(PyObject *o, long long most, long long *x) {
  int over;
  PyObject *r = PyNumber_Index(o);
  if (r == NULL) return 0;
  *x = PyLong_AsLongLongAndOverflow(r, &over);
  Py_DECREF(r);
  if (over > 0 || *x > most) *x = most;
  if (over < 0 || *x < -1) *x = -1;
  return !PyErr_Occurred();
}

#define NOT_PLAIN return PyLong_FromLong(-1)

static int have(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 1;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return 0;
}

/* plan_step(dev, stream, new_lens, context_lens, block_tables, free_blocks, num_free,
 * new_context_lens, new_num_free, slot_mapping, positions, cu_seqlens_q, cu_seqlens_k,
 * num_blocks, block_size, borrowed_blocks, dev_status) */
static PyObject *plan_step(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  void *p[13];
  long long dev, table[2], rows[1], free_blocks[1], num_blocks, block_size;
  (void)self;
  if (!have(n, 17)) return NULL;
  dev = PyLong_AsLongLong(a[0]);
  void *stream = PyLong_AsVoidPtr(a[1]);
  if (PyErr_Occurred()) return NULL;
  if (!tensor(a[4], i32, dev, 2, table, NULL, &p[2]) ||
      !tensor(a[5], i32, dev, 1, free_blocks, NULL, &p[3]) ||
      !tensor(a[9], i32, dev, 1, rows, NULL, &p[7]))
    NOT_PLAIN;
  const long long S = table[0];
  p[11] = NULL;
  if (!of_shape(a[2], i32, dev, 1, S, 0, 0, 0, &p[0]) ||
      !of_shape(a[3], i32, dev, 1, S, 0, 0, 0, &p[1]) ||
      !of_shape(a[6], i32, dev, 1, 1, 0, 0, 0, &p[4]) ||
      !of_shape(a[7], i32, dev, 1, S, 0, 0, 0, &p[5]) ||
      !of_shape(a[8], i32, dev, 1, 1, 0, 0, 0, &p[6]) ||
      !of_shape(a[10], i32, dev, 1, rows[0], 0, 0, 0, &p[8]) ||
      !of_shape(a[11], i32, dev, 1, S + 1, 0, 0, 0, &p[9]) ||
      !of_shape(a[12], i32, dev, 1, S + 1, 0, 0, 0, &p[10]) ||
      (a[15] != Py_None && !of_shape(a[15], i32, dev, 1, S, 0, 0, 0, &p[11])) ||
      !status_of(a[16], dev, &p[12]) || S > INT32_MAX || table[1] > INT32_MAX)
    NOT_PLAIN;
  if (!number(a[13], INT64_MAX, &num_blocks) || !number(a[14], INT32_MAX, &block_size)) return NULL;
  pkv_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = plan_step_fn(p[0], p[1], p[11], p[2], p[3], p[4], p[5], p[6], p[7], p[8],
                                      p[9], p[10], (int)S, rows[0], (int)table[1], (int)block_size,
                                      num_blocks, free_blocks[0], p[12], stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* Rows of q, k or v [T, heads, D]: contiguous, at any distance.  (Strides of dims of size
 * one, and of tokens of which there is one, say nothing.) */
static int rows_of(PyObject *t, long long dev, long long *dims, long long *step, void **ptr) {
  long long st[3];
  if (!tensor(t, bf16, dev, 3, dims, st, ptr)) return 0;
  *step = dims[0] > 1 ? st[0] : 0;  /* (0, to the library: contiguous) */
  return (st[2] == 1 || dims[2] <= 1) && (st[1] == dims[2] || dims[1] <= 1) &&
         (dims[0] <= 1 || *step > 0);
}

/* norm_rope_store(dev, stream, q_out, q, k, v, positions, turns, k_cache, v_cache,
 * slot_mapping, k_out, q_weight, k_weight, eps, interleaved, amplitude, dev_status) */
static PyObject *norm_rope_store(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  void *q_out, *q, *k, *v = NULL, *positions, *turns, *k_cache = NULL, *v_cache = NULL,
                           *slots = NULL, *k_out = NULL, *q_weight = NULL, *k_weight = NULL, *status;
  long long dev, qd[3], kd[3], vd[3], cd[4] = {0, 0, 0, 0}, pairs[1], q_step, k_step, v_step = 0;
  (void)self;
  if (!have(n, 18)) return NULL;
  dev = PyLong_AsLongLong(a[0]);
  void *stream = PyLong_AsVoidPtr(a[1]);
  if (PyErr_Occurred()) return NULL;
  const int store = a[8] != Py_None, norm = a[12] != Py_None;
  if (store != (a[9] != Py_None) || store != (a[10] != Py_None) || norm != (a[13] != Py_None))
    NOT_PLAIN;
  if (!rows_of(a[3], dev, qd, &q_step, &q) || !rows_of(a[4], dev, kd, &k_step, &k) ||
      kd[0] != qd[0] || kd[2] != qd[2])
    NOT_PLAIN;
  const long long T = qd[0], Hq = qd[1], Hkv = kd[1], D = qd[2];
  if (!of_shape(a[2], bf16, dev, 3, T, Hq, D, 0, &q_out) ||
      !of_shape(a[6], i32, dev, 1, T, 0, 0, 0, &positions) ||
      !tensor(a[7], i64, dev, 1, pairs, NULL, &turns))
    NOT_PLAIN;
  if (store && (!rows_of(a[5], dev, vd, &v_step, &v) || vd[0] != T || vd[1] != Hkv || vd[2] != D ||
                !tensor(a[8], bf16, dev, 4, cd, NULL, &k_cache) || cd[2] != Hkv || cd[3] != D ||
                !of_shape(a[9], bf16, dev, 4, cd[0], cd[1], cd[2], cd[3], &v_cache) ||
                !of_shape(a[10], i32, dev, 1, T, 0, 0, 0, &slots)))
    NOT_PLAIN;
  if ((a[11] != Py_None && !of_shape(a[11], bf16, dev, 3, T, Hkv, D, 0, &k_out)) ||
      (norm && (!of_shape(a[12], bf16, dev, 1, D, 0, 0, 0, &q_weight) ||
                !of_shape(a[13], bf16, dev, 1, D, 0, 0, 0, &k_weight))) ||
      !status_of(a[17], dev, &status) || Hq > INT32_MAX || Hkv > INT32_MAX || D > INT32_MAX ||
      pairs[0] > INT32_MAX / 2 || cd[1] > INT32_MAX)
    NOT_PLAIN;
  const double eps = PyFloat_AsDouble(a[14]), amplitude = PyFloat_AsDouble(a[16]);
  const int interleaved = PyObject_IsTrue(a[15]);
  if (PyErr_Occurred()) return NULL;
  pkv_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = norm_rope_fn(q_out, k_out, q, k, v, k_cache, v_cache, slots, positions,
                                      turns, q_weight, k_weight, T, (int)Hq, (int)Hkv, (int)D,
                                      q_step, k_step, v_step, (int)(2 * pairs[0]), interleaved,
                                      (float)eps, (float)amplitude, cd[0], (int)cd[1], status,
                                      stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* paged_decode_shared_attn(dev, stream, out, q, k_cache, v_cache, block_tables,
 * context_lens, group_starts, shared_blocks, scale, workspace, dev_status) */
static PyObject *paged_decode_shared_attn(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  void *out, *q, *k_cache, *v_cache, *tables, *lens, *starts, *shared, *workspace, *status;
  long long dev, qd[3], cd[4], td[2], groups[1], bytes[1];
  (void)self;
  if (!have(n, 13)) return NULL;
  dev = PyLong_AsLongLong(a[0]);
  void *stream = PyLong_AsVoidPtr(a[1]);
  if (PyErr_Occurred()) return NULL;
  if (!tensor(a[3], bf16, dev, 3, qd, NULL, &q) || !tensor(a[4], bf16, dev, 4, cd, NULL, &k_cache) ||
      !tensor(a[6], i32, dev, 2, td, NULL, &tables) ||
      !tensor(a[9], i32, dev, 1, groups, NULL, &shared) ||
      !tensor(a[11], u8, dev, 1, bytes, NULL, &workspace) || cd[3] != qd[2] || td[0] != qd[0])
    NOT_PLAIN;
  const long long S = qd[0], Hq = qd[1], D = qd[2];
  if (!of_shape(a[2], bf16, dev, 3, S, Hq, D, 0, &out) ||
      !of_shape(a[5], bf16, dev, 4, cd[0], cd[1], cd[2], cd[3], &v_cache) ||
      !of_shape(a[7], i32, dev, 1, S, 0, 0, 0, &lens) ||
      !of_shape(a[8], i32, dev, 1, groups[0] + 1, 0, 0, 0, &starts) ||
      !status_of(a[12], dev, &status) || S > INT32_MAX || groups[0] > INT32_MAX || Hq > INT32_MAX ||
      D > INT32_MAX || cd[1] > INT32_MAX || cd[2] > INT32_MAX || td[1] > INT32_MAX)
    NOT_PLAIN;
  const double scale = PyFloat_AsDouble(a[10]);
  if (PyErr_Occurred()) return NULL;
  pkv_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = shared_attn_fn(out, q, k_cache, v_cache, tables, lens, starts, shared,
                                        (int)S, (int)groups[0], (int)Hq, (int)cd[2], (int)D,
                                        (int)cd[1], (int)td[1], cd[0], (float)scale, workspace,
                                        (size_t)bytes[0], status, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

/* bind(torch.bfloat16, torch.int32, torch.int64, torch.uint8, address of pkv_plan_step,
 * of pkv_norm_rope_store, of pkv_paged_decode_shared_attn) */
static PyObject *bind(PyObject *self, PyObject *args) {
  PyObject *t[4];
  unsigned long long f[3];
  (void)self;
  if (!PyArg_ParseTuple(args, "OOOOKKK", &t[0], &t[1], &t[2], &t[3], &f[0], &f[1], &f[2]))
    return NULL;
  for (int i = 0; i < 4; ++i) Py_INCREF(t[i]); /* (kept for good, as the module is) */
  bf16 = t[0];
  i32 = t[1];
  i64 = t[2];
  u8 = t[3];
  *(void **)&plan_step_fn = (void *)(uintptr_t)f[0];
  *(void **)&norm_rope_fn = (void *)(uintptr_t)f[1];
  *(void **)&shared_attn_fn = (void *)(uintptr_t)f[2];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, NULL},
    {"plan_step", (PyCFunction)(void (*)(void))plan_step, METH_FASTCALL, NULL},
    {"norm_rope_store", (PyCFunction)(void (*)(void))norm_rope_store, METH_FASTCALL, NULL},
    {"paged_decode_shared_attn", (PyCFunction)(void (*)(void))paged_decode_shared_attn,
     METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkv_call", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pkv_call(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_shape = PyUnicode_InternFromString("shape");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_stride = PyUnicode_InternFromString("stride");
  s_dim = PyUnicode_InternFromString("dim");
  s_numel = PyUnicode_InternFromString("numel");
  if (!s_dtype || !s_get_device || !s_is_contiguous || !s_shape || !s_data_ptr || !s_stride ||
      !s_dim || !s_numel)
    return NULL;
  return PyModule_Create(&module);
}
