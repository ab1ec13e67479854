// pycall.cc -- the Python binding's checks and calls, for operators whose work on the GPU
// is shorter than the same checks take in Python (a decode step's plan, its rotation).
//
// Each function takes the tensors of one call, checks them (dtype, device, contiguous,
// shape) and calls the library.  It returns the library's status, or -1 when a tensor
// is not what it has to be: the caller then finds out in Python what to say about it.
// A tensor's fields are read through torch's own C++ class (asked for as attributes in
// Python, through the C API, those of plan_step's 13 tensors took 3.0 us of a call's 6.0),
// so the module is for the torch that it was built with, which bind() checks.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "pkv.h"

namespace {

decltype(&pkv_plan_step) plan_step_fn;
decltype(&pkv_norm_rope_store) norm_rope_fn;
decltype(&pkv_paged_decode_shared_attn) shared_attn_fn;

// A tensor of a dtype, on device dev; its dims and address.  strides: NULL for one that
// has to be contiguous.  False when it is anything else (one without storage, too).
bool tensor(PyObject *o, at::ScalarType dtype, int64_t dev, int ndim, int64_t *dims, int64_t *strides,
            void **ptr) noexcept {
  try {
    if (!THPVariable_Check(o)) return false;
    const at::TensorBase &t = THPVariable_Unpack(o);
    if (!t.defined() || t.scalar_type() != dtype || t.layout() != at::kStrided || !t.is_cuda() ||
        t.get_device() != dev || t.dim() != ndim)
      return false;
    if (strides == nullptr ? !t.is_contiguous() : false) return false;
    for (int i = 0; i < ndim; ++i) {
      dims[i] = t.size(i);
      if (strides != nullptr) strides[i] = t.stride(i);
    }
    *ptr = t.data_ptr();
    return true;
  } catch (...) {
    return false;
  }
}

// The device of a call on this tensor, if it is the current one (the library launches
// there), and the stream: the one given, a number, or for None torch's current one there.
bool place(PyObject *o, PyObject *given, int64_t *dev, void **stream) noexcept {
  try {
    if (!THPVariable_Check(o)) return false;
    const at::TensorBase &t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda()) return false;
    *dev = t.get_device();
    if (c10::cuda::current_device() != *dev) return false;
    if (given == Py_None)
      *stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)*dev).stream();
    else
      *stream = PyLong_AsVoidPtr(given);
    return true;
  } catch (...) {
    return false;
  }
}

constexpr at::ScalarType bf16 = at::kBFloat16, i32 = at::kInt, i64 = at::kLong, u8 = at::kByte;

// The same with its dims given.
bool of_shape(PyObject *t, at::ScalarType dtype, int64_t dev, int ndim, int64_t d0, int64_t d1,
              int64_t d2, int64_t d3, void **ptr) noexcept {
  const int64_t want[4] = {d0, d1, d2, d3};
  int64_t dims[4];
  if (!tensor(t, dtype, dev, ndim, dims, nullptr, ptr)) return false;
  for (int i = 0; i < ndim; ++i)
    if (dims[i] != want[i]) return false;
  return true;
}

// dev_status: None, or of any shape with something in it.
bool status_of(PyObject *o, int64_t dev, void **ptr) noexcept {
  int64_t x[8];
  *ptr = nullptr;
  if (o == Py_None) return true;
  if (!THPVariable_Check(o)) return false;
  int64_t ndim = 9, numel = 0;
  try {
    const at::TensorBase &t = THPVariable_Unpack(o);
    ndim = t.dim();
    numel = t.numel();
  } catch (...) {
    return false;
  }
  return ndim <= 8 && numel > 0 && tensor(o, i32, dev, (int)ndim, x, nullptr, ptr);
}

// A whole number as an argument of the library: what does not fit stays too large or
// becomes -1 (refused there), instead of wrapping around.  0 with an exception set when
// it is none.
int number(PyObject *o, long long most, long long *x) {
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

int have(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 1;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return 0;
}

// plan_step(stream, new_lens, context_lens, block_tables, free_blocks, num_free,
// new_context_lens, new_num_free, slot_mapping, positions, cu_seqlens_q, cu_seqlens_k,
// num_blocks, block_size, borrowed_blocks, dev_status)
PyObject *plan_step(PyObject *, PyObject *const *given, Py_ssize_t n) {
  void *p[13], *stream;
  int64_t dev, table[2], rows[1], free_blocks[1];
  long long num_blocks, block_size;
  if (!have(n, 16)) return NULL;
  PyObject *const *a = given - 1;  // (numbered from the stream on)
  if (!place(a[4], a[1], &dev, &stream)) NOT_PLAIN;
  if (PyErr_Occurred()) return NULL;
  if (!tensor(a[4], i32, dev, 2, table, NULL, &p[2]) ||
      !tensor(a[5], i32, dev, 1, free_blocks, NULL, &p[3]) ||
      !tensor(a[9], i32, dev, 1, rows, NULL, &p[7]))
    NOT_PLAIN;
  const int64_t S = table[0];
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
  int32_t *x[13];
  for (int i = 0; i < 13; ++i) x[i] = static_cast<int32_t *>(p[i]);
  pkv_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = plan_step_fn(x[0], x[1], x[11], x[2], x[3], x[4], x[5], x[6], x[7], x[8], x[9], x[10],
                    (int)S, rows[0], (int)table[1], (int)block_size, num_blocks, free_blocks[0],
                    x[12], stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

// Rows of q, k or v [T, heads, D]: contiguous, at any distance.  (Strides of dims of size
// one, and of tokens of which there is one, say nothing.)
bool rows_of(PyObject *t, int64_t dev, int64_t *dims, int64_t *step, void **ptr) noexcept {
  int64_t st[3];
  if (!tensor(t, bf16, dev, 3, dims, st, ptr)) return false;
  *step = dims[0] > 1 ? st[0] : 0;  // (0, to the library: contiguous)
  return (st[2] == 1 || dims[2] <= 1) && (st[1] == dims[2] || dims[1] <= 1) &&
         (dims[0] <= 1 || *step > 0);
}

uint16_t *b16(void *p) { return static_cast<uint16_t *>(p); }
int32_t *n32(void *p) { return static_cast<int32_t *>(p); }

// norm_rope_store(stream, q_out, q, k, v, positions, turns, k_cache, v_cache, slot_mapping,
// k_out, q_weight, k_weight, eps, interleaved, amplitude, dev_status)
PyObject *norm_rope_store(PyObject *, PyObject *const *given, Py_ssize_t n) {
  void *q_out, *q, *k, *v = NULL, *positions, *turns, *k_cache = NULL, *v_cache = NULL,
                           *slots = NULL, *k_out = NULL, *q_weight = NULL, *k_weight = NULL, *status,
                           *stream;
  int64_t dev, qd[3], kd[3], vd[3], cd[4] = {0, 0, 0, 0}, pairs[1], q_step, k_step, v_step = 0;
  if (!have(n, 17)) return NULL;
  PyObject *const *a = given - 1;
  if (!place(a[3], a[1], &dev, &stream)) NOT_PLAIN;
  if (PyErr_Occurred()) return NULL;
  const bool store = a[8] != Py_None, norm = a[12] != Py_None;
  if (store != (a[9] != Py_None) || store != (a[10] != Py_None) || norm != (a[13] != Py_None))
    NOT_PLAIN;
  if (!rows_of(a[3], dev, qd, &q_step, &q) || !rows_of(a[4], dev, kd, &k_step, &k) ||
      kd[0] != qd[0] || kd[2] != qd[2])
    NOT_PLAIN;
  const int64_t T = qd[0], Hq = qd[1], Hkv = kd[1], D = qd[2];
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
  st = norm_rope_fn(b16(q_out), b16(k_out), b16(q), b16(k), b16(v), b16(k_cache), b16(v_cache),
                    n32(slots), n32(positions), static_cast<uint64_t *>(turns), b16(q_weight),
                    b16(k_weight), T, (int)Hq, (int)Hkv, (int)D, q_step, k_step, v_step,
                    (int)(2 * pairs[0]), interleaved, (float)eps, (float)amplitude, cd[0],
                    (int)cd[1], n32(status), stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

// paged_decode_shared_attn(stream, out, q, k_cache, v_cache, block_tables, context_lens,
// group_starts, shared_blocks, scale, workspace, dev_status)
PyObject *paged_decode_shared_attn(PyObject *, PyObject *const *given, Py_ssize_t n) {
  void *out, *q, *k_cache, *v_cache, *tables, *lens, *starts, *shared, *workspace, *status, *stream;
  int64_t dev, qd[3], cd[4], td[2], groups[1], bytes[1];
  if (!have(n, 12)) return NULL;
  PyObject *const *a = given - 1;
  if (!place(a[3], a[1], &dev, &stream)) NOT_PLAIN;
  if (PyErr_Occurred()) return NULL;
  if (!tensor(a[3], bf16, dev, 3, qd, NULL, &q) || !tensor(a[4], bf16, dev, 4, cd, NULL, &k_cache) ||
      !tensor(a[6], i32, dev, 2, td, NULL, &tables) ||
      !tensor(a[9], i32, dev, 1, groups, NULL, &shared) ||
      !tensor(a[11], u8, dev, 1, bytes, NULL, &workspace) || cd[3] != qd[2] || td[0] != qd[0])
    NOT_PLAIN;
  const int64_t S = qd[0], Hq = qd[1], D = qd[2];
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
  st = shared_attn_fn(b16(out), b16(q), b16(k_cache), b16(v_cache), n32(tables), n32(lens),
                      n32(starts), n32(shared), (int)S, (int)groups[0], (int)Hq, (int)cd[2], (int)D,
                      (int)cd[1], (int)td[1], cd[0], (float)scale, workspace, (size_t)bytes[0],
                      n32(status), stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

// bind(torch's version, address of pkv_plan_step, of pkv_norm_rope_store, of
// pkv_paged_decode_shared_attn)
PyObject *bind(PyObject *, PyObject *args) {
  const char *version;
  unsigned long long f[3];
  if (!PyArg_ParseTuple(args, "sKKK", &version, &f[0], &f[1], &f[2])) return NULL;
  if (strcmp(version, PKV_TORCH_VERSION) != 0)  // (of the build)
    return PyErr_Format(PyExc_ImportError, "built for torch %s, this is %s", PKV_TORCH_VERSION, version);
  plan_step_fn = reinterpret_cast<decltype(plan_step_fn)>((uintptr_t)f[0]);
  norm_rope_fn = reinterpret_cast<decltype(norm_rope_fn)>((uintptr_t)f[1]);
  shared_attn_fn = reinterpret_cast<decltype(shared_attn_fn)>((uintptr_t)f[2]);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, NULL},
    {"plan_step", fast(plan_step), METH_FASTCALL, NULL},
    {"norm_rope_store", fast(norm_rope_store), METH_FASTCALL, NULL},
    {"paged_decode_shared_attn", fast(paged_decode_shared_attn), METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkv_call", NULL, -1, methods, NULL, NULL, NULL, NULL};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_call(void) { return PyModule_Create(&module); }
