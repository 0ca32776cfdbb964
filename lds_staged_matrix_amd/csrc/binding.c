/*
 * binding.c -- the Python side of the enqueueing entry points (CPython C API).
 *
 * A small product takes a few microseconds on the GPU and hipLaunchKernel 2.4 us
 * on the host; the same call through ctypes added 1.6 us of marshalling, this
 * adds 0.4.  Arguments are taken by position, as the package's functions of the
 * same names pass them:
 *   handle   what a ctypes.c_void_p parameter takes (a c_void_p, an integer, None);
 *            anything else raises ctypes.ArgumentError
 *   pointers integers, None, or objects with a data_ptr() method
 *   integers anything int() takes; one that its C parameter cannot hold raises
 *            OverflowError
 *   stream   an integer, None, or an object with a cuda_stream attribute
 * and the gemm_status comes back.  bind() takes the addresses of the entry
 * points in the loaded library.
 */
/* The stable ABI from Python 3.10 on, the oldest that torch's ROCm builds serve:
 * one build loads in every later Python. */
#define Py_LIMITED_API 0x030A0000
#include <Python.h>

#include <stdint.h>

#include "lds_gemm.h"

static __typeof__(gemm_run) *p_run;
static __typeof__(gemm_scaled_run) *p_scaled;
static __typeof__(gemm_w4_run) *p_w4;
static __typeof__(gemm_rmsnorm_run) *p_rmsnorm;
static PyObject *s_data_ptr, *s_cuda_stream, *s_value;
static PyObject *c_void_p, *c_cast;                 /* of ctypes */

/* int(x) as an address; the low 64 bits count. */
static int int_address(PyObject *x, void **out) {
  PyObject *i = PyNumber_Long(x);
  if (!i) return -1;
  *out = (void *)(uintptr_t)PyLong_AsUnsignedLongLongMask(i);
  Py_DECREF(i);
  return PyErr_Occurred() ? -1 : 0;
}

/* x, or x.name (called if `call`) where x has it, as an address. */
static int address(PyObject *x, PyObject *name, int call, void **out) {
  *out = NULL;
  if (x == Py_None) return 0;
  if (PyLong_Check(x)) return int_address(x, out);
  PyObject *v = PyObject_GetAttr(x, name);
  if (!v) {
    if (!PyErr_ExceptionMatches(PyExc_AttributeError)) return -1;
    PyErr_Clear();
    return int_address(x, out);
  }
  if (call) {
    PyObject *r = PyObject_CallNoArgs(v);
    Py_DECREF(v);
    if (!r) return -1;
    v = r;
  }
  const int e = v == Py_None ? 0 : int_address(v, out);
  Py_DECREF(v);
  return e;
}

/* A handle's address.  The library reads what it points to, so nothing is taken
 * for one that ctypes would not convert to a pointer: no float, no number of
 * another library, no object that merely has a value. */
static int handle(PyObject *x, void **out) {
  *out = NULL;
  if (x == Py_None) return 0;
  if (PyLong_Check(x)) return int_address(x, out);
  const int is = PyObject_IsInstance(x, c_void_p);
  if (is < 0) return -1;
  PyObject *p = is ? Py_NewRef(x) : PyObject_CallFunctionObjArgs(c_cast, x, c_void_p, NULL);
  if (!p) return -1;
  PyObject *v = PyObject_GetAttr(p, s_value);
  Py_DECREF(p);
  if (!v) return -1;
  const int e = v == Py_None ? 0 : int_address(v, out);
  Py_DECREF(v);
  return e;
}

static int integer(PyObject *x, const char *name, int bits, int64_t *out) {
  PyObject *i = PyNumber_Long(x);
  if (!i) return -1;
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(i, &over);
  int e = 0;
  if (over || (bits == 32 && (v < INT32_MIN || v > INT32_MAX))) {
    PyErr_Format(PyExc_OverflowError, "%s=%S does not fit the C ABI's int%d_t parameter", name, i, bits);
    e = -1;
  }
  Py_DECREF(i);
  if (e || PyErr_Occurred()) return -1;
  *out = v;
  return 0;
}

/* An entry point's arguments: the handle, `np` pointers, `nw` 64-bit integers,
 * `nf` floats, `nn` 32-bit integers, the stream. */
struct shape {
  const char *name;
  int np, nw, nf, nn;
  const char *ints[16];
};
struct values {
  gemm_handle_t h;
  void *p[8];
  int64_t w[12];
  float f[1];
  int n[8];
  hipStream_t s;
};

static int take(const struct shape *t, PyObject *const *a, Py_ssize_t n, struct values *v) {
  const Py_ssize_t want = 2 + t->np + t->nw + t->nf + t->nn;
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", t->name, want, n);
    return -1;
  }
  void *x;
  if (handle(*a++, &x)) return -1;
  v->h = (gemm_handle_t)x;
  for (int i = 0; i < t->np; i++)
    if (address(*a++, s_data_ptr, 1, &v->p[i])) return -1;
  const char *const *name = t->ints;
  for (int i = 0; i < t->nw; i++)
    if (integer(*a++, *name++, 64, &v->w[i])) return -1;
  for (int i = 0; i < t->nf; i++) {
    const double d = PyFloat_AsDouble(*a++);
    if (d == -1.0 && PyErr_Occurred()) return -1;
    v->f[i] = (float)d;
  }
  for (int i = 0; i < t->nn; i++) {
    int64_t k;
    if (integer(*a++, *name++, 32, &k)) return -1;
    v->n[i] = (int)k;
  }
  if (address(*a++, s_cuda_stream, 0, &x)) return -1;
  v->s = (hipStream_t)x;
  return 0;
}

#define CALL(p, ...)                                                        \
  do {                                                                      \
    int st;                                                                 \
    if (!(p)) {                                                             \
      PyErr_SetString(PyExc_RuntimeError, "the library is not bound");      \
      return NULL;                                                          \
    }                                                                       \
    Py_BEGIN_ALLOW_THREADS st = (p)(__VA_ARGS__);                           \
    Py_END_ALLOW_THREADS return PyLong_FromLong(st);                        \
  } while (0)

static PyObject *py_run(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  static const struct shape t = {"gemm_run", 3, 6, 0, 3,
                                 {"M", "N", "K", "lda", "ldb", "ldc", "layoutA", "layoutB", "dtype"}};
  struct values v;
  (void)self;
  if (take(&t, a, n, &v)) return NULL;
  CALL(p_run, v.h, v.p[0], v.p[1], v.p[2], v.w[0], v.w[1], v.w[2], v.w[3], v.w[4], v.w[5], v.n[0], v.n[1], v.n[2],
       v.s);
}

static PyObject *py_scaled(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  static const struct shape t = {
      "gemm_scaled_run", 5, 6, 0, 5,
      {"M", "N", "K", "lda", "ldb", "ldc", "incA", "incB", "layoutA", "layoutB", "dtype"}};
  struct values v;
  (void)self;
  if (take(&t, a, n, &v)) return NULL;
  CALL(p_scaled, v.h, v.p[0], v.p[1], v.p[2], (const float *)v.p[3], (const float *)v.p[4], v.w[0], v.w[1], v.w[2],
       v.w[3], v.w[4], v.w[5], v.n[0], v.n[1], v.n[2], v.n[3], v.n[4], v.s);
}

static PyObject *py_w4(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  static const struct shape t = {"gemm_w4_run", 5, 9, 0, 1,
                                 {"M", "N", "K", "group", "lda", "ldb", "lds", "ldz", "ldc", "dtype"}};
  struct values v;
  (void)self;
  if (take(&t, a, n, &v)) return NULL;
  CALL(p_w4, v.h, v.p[0], v.p[1], v.p[2], v.p[3], v.p[4], v.w[0], v.w[1], v.w[2], v.w[3], v.w[4], v.w[5], v.w[6],
       v.w[7], v.w[8], v.n[0], v.s);
}

static PyObject *py_rmsnorm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  static const struct shape t = {"gemm_rmsnorm_run", 6, 6, 1, 1, {"M", "N", "ldx", "ldr", "ldh", "ldy", "dtype"}};
  struct values v;
  (void)self;
  if (take(&t, a, n, &v)) return NULL;
  CALL(p_rmsnorm, v.h, v.p[0], v.p[1], v.p[2], v.p[3], v.p[4], (float *)v.p[5], v.w[0], v.w[1], v.w[2], v.w[3],
       v.w[4], v.w[5], v.f[0], v.n[0], v.s);
}

static PyObject *py_bind(PyObject *self, PyObject *args) {
  unsigned long long run, scaled, w4, rmsnorm;
  (void)self;
  if (!PyArg_ParseTuple(args, "KKKK", &run, &scaled, &w4, &rmsnorm)) return NULL;
  p_run = (__typeof__(p_run))(uintptr_t)run;
  p_scaled = (__typeof__(p_scaled))(uintptr_t)scaled;
  p_w4 = (__typeof__(p_w4))(uintptr_t)w4;
  p_rmsnorm = (__typeof__(p_rmsnorm))(uintptr_t)rmsnorm;
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", py_bind, METH_VARARGS, "Addresses of gemm_run, gemm_scaled_run, gemm_w4_run, gemm_rmsnorm_run."},
    {"run", (PyCFunction)(void (*)(void))py_run, METH_FASTCALL, "gemm_run"},
    {"scaled", (PyCFunction)(void (*)(void))py_scaled, METH_FASTCALL, "gemm_scaled_run"},
    {"w4", (PyCFunction)(void (*)(void))py_w4, METH_FASTCALL, "gemm_w4_run"},
    {"rmsnorm", (PyCFunction)(void (*)(void))py_rmsnorm, METH_FASTCALL, "gemm_rmsnorm_run"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  s_value = PyUnicode_InternFromString("value");
  if (!s_data_ptr || !s_cuda_stream || !s_value) return NULL;
  PyObject *ctypes = PyImport_ImportModule("ctypes");
  if (!ctypes) return NULL;
  c_void_p = PyObject_GetAttrString(ctypes, "c_void_p");
  c_cast = PyObject_GetAttrString(ctypes, "cast");
  Py_DECREF(ctypes);
  if (!c_void_p || !c_cast) return NULL;
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddIntConstant(m, "limited_api", Py_LIMITED_API) < 0) {
    Py_DECREF(m);
    return NULL;
  }
  return m;
}
