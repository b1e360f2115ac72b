/* qmm_call.c -- CPython calls of the C entry points that a decode step makes
 * once per layer.  They only turn Python integers and floats into C arguments,
 * as ctypes does, at a fraction of its time: a call of 23 arguments takes
 * about 0.5 us here and 3 us there, beside 2 us for the kernel's launch.
 * bind(name, address) sets the library function that the wrapper of that name
 * calls.  The interpreter lock is released during the call. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <string.h>

#include "../../../include/qmm.h"

typedef union {
  long long i;
  double f;
} Arg;

/* One argument per letter of spec: i an integer (or address), f a float. */
static int parse(PyObject *const *a, Py_ssize_t n, const char *spec, Arg *v) {
  if (n != (Py_ssize_t)strlen(spec)) {
    PyErr_Format(PyExc_TypeError, "%zu arguments are needed, got %zd", strlen(spec), n);
    return 0;
  }
  for (Py_ssize_t k = 0; k < n; ++k) {
    if (spec[k] == 'f') v[k].f = PyFloat_AsDouble(a[k]);
    else v[k].i = PyLong_AsLongLong(a[k]);
  }
  return !PyErr_Occurred();
}

#define I(k) v[k].i
#define N(k) (int)v[k].i
#define P(k) (void *)(uintptr_t)v[k].i
#define F(k) (float)v[k].f

#define CALL(fn, spec, ...)                                                   \
  static __typeof__(&fn) p_##fn;                                              \
  static PyObject *w_##fn(PyObject *self, PyObject *const *a, Py_ssize_t n) { \
    Arg v[sizeof(spec)];                                                      \
    int status;                                                               \
    if (!parse(a, n, spec, v)) return NULL;                                   \
    if (!p_##fn) {                                                            \
      PyErr_SetString(PyExc_RuntimeError, #fn " is not bound");               \
      return NULL;                                                            \
    }                                                                         \
    Py_BEGIN_ALLOW_THREADS                                                    \
    status = p_##fn(__VA_ARGS__);                                             \
    Py_END_ALLOW_THREADS                                                      \
    return PyLong_FromLong(status);                                           \
  }

CALL(qmm_rope, "iiifiiiiiiiiiii", P(0), I(1), N(2), F(3), P(4), P(5), N(6), I(7), P(8), N(9), I(10), I(11), I(12), I(13),
     P(14))
CALL(qmm_kv_write, "iiiiiiiiiiiiiiii", N(0), N(1), P(2), P(3), I(4), I(5), I(6), I(7), P(8), I(9), P(10), I(11), N(12),
     P(13), I(14), P(15))
CALL(qmm_kv_append, "iiifiiiiiiiiiiiiiiiiiiiiiii", P(0), I(1), N(2), F(3), P(4), P(5), I(6), I(7), P(8), N(9), I(10),
     N(11), N(12), P(13), P(14), I(15), I(16), I(17), I(18), P(19), I(20), P(21), I(22), N(23), P(24), I(25), P(26))
CALL(qmm_kv_read, "iiiiiiiiiiiiii", N(0), N(1), P(2), P(3), I(4), I(5), I(6), I(7), P(8), I(9), P(10), P(11), N(12),
     P(13))
CALL(qmm_attn_decode, "iiiiiiiiiiiiiiiifiiiiii", N(0), N(1), P(2), P(3), I(4), I(5), I(6), I(7), P(8), N(9), I(10), I(11),
     P(12), I(13), P(14), I(15), F(16), I(17), P(18), P(19), P(20), (size_t)I(21), P(22))

static PyObject *bind(PyObject *self, PyObject *args) {
  const char *name;
  unsigned long long address;
  if (!PyArg_ParseTuple(args, "sK", &name, &address)) return NULL;
#define SET(fn) \
  if (!strcmp(name, #fn)) { p_##fn = (__typeof__(&fn))(uintptr_t)address; Py_RETURN_NONE; }
  SET(qmm_rope) SET(qmm_kv_write) SET(qmm_kv_append) SET(qmm_kv_read) SET(qmm_attn_decode)
#undef SET
  PyErr_Format(PyExc_ValueError, "no wrapper named %s", name);
  return NULL;
}

#define METHOD(fn) {#fn, (PyCFunction)(void (*)(void))w_##fn, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    METHOD(qmm_rope), METHOD(qmm_kv_write), METHOD(qmm_kv_append), METHOD(qmm_kv_read), METHOD(qmm_attn_decode),
    {"bind", bind, METH_VARARGS, NULL}, {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmm_call", NULL, -1, methods, NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__qmm_call(void) { return PyModule_Create(&module); }
