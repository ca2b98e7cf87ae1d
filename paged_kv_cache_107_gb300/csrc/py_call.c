/* py_call.c — the 8-bit cache's and the rotary calls of pa.h for Python, without ctypes.
 *
 * ctypes takes 1.9 us to convert the 23 arguments of a rotary store, about as long as the launch
 * itself; here it is 0.2 us. Arguments are the C function's in order: integers (an address for a
 * pointer, None for NULL), a float for the scale; the result is the status. The functions are
 * those of the library that the binding has loaded (bind), called without the interpreter's lock.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

#include "../../include/pa.h"

static struct {
  __typeof__(&pa_store_kvcache_q8) store_q8;
  __typeof__(&pa_load_kvcache_q8) load_q8;
  __typeof__(&pa_decode_q8) decode_q8;
  __typeof__(&pa_rotary_store) rotary;
  __typeof__(&pa_rotary_store_q8) rotary_q8;
} lib;

/* Arguments by their C types, one character each: p a pointer (an address, or None for NULL), i an
 * int, l an int64_t, z a size_t, f a float. What does not fit its type is an exception. */
#define MAX_ARGS 24
typedef struct {
  uint64_t v[MAX_ARGS];
  float f;
} call_args;

static int take(PyObject* const* args, Py_ssize_t given, const char* types, call_args* out) {
  const Py_ssize_t n = (Py_ssize_t)strlen(types);
  if (given != n) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd needed", given, n);
    return -1;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* x = args[i];
    out->v[i] = 0;
    if (types[i] == 'f') {
      const double f = PyFloat_AsDouble(x);
      if (f == -1.0 && PyErr_Occurred()) return -1;
      out->f = (float)f;
    } else if (types[i] == 'p' && x == Py_None) {
      continue;
    } else if (!PyLong_Check(x)) {
      PyErr_Format(PyExc_TypeError, "argument %zd must be an integer, not %s", i,
                   Py_TYPE(x)->tp_name);
      return -1;
    } else if (types[i] == 'p' || types[i] == 'z') {
      out->v[i] = PyLong_AsUnsignedLongLong(x);
      if (out->v[i] == UINT64_MAX && PyErr_Occurred()) return -1;
    } else {
      const long long w = PyLong_AsLongLong(x);
      if (w == -1 && PyErr_Occurred()) return -1;
      if (types[i] == 'i' && (w < INT32_MIN || w > INT32_MAX)) {
        PyErr_Format(PyExc_OverflowError, "argument %zd does not fit 32 bits", i);
        return -1;
      }
      out->v[i] = (uint64_t)w;
    }
  }
  return 0;
}

#define P(i) ((void*)(uintptr_t)a.v[i])
#define I64(i) ((int64_t)a.v[i])
#define I32(i) ((int)(int64_t)a.v[i])

static PyObject* status(int rc) { return PyLong_FromLong(rc); }

static int bound(const void* fn) {
  if (!fn) PyErr_SetString(PyExc_RuntimeError, "no library bound");
  return fn != NULL;
}

static PyObject* store_q8(PyObject* self, PyObject* const* args, Py_ssize_t given) {
  call_args a;
  int rc;
  if (!bound(lib.store_q8) || take(args, given, "ppllippiiiilpp", &a) < 0) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = lib.store_q8(P(0), P(1), I64(2), I64(3), I32(4), P(5), P(6), I32(7), I32(8), I32(9), I32(10),
                    I64(11), P(12), P(13));
  Py_END_ALLOW_THREADS
  return status(rc);
}

static PyObject* load_q8(PyObject* self, PyObject* const* args, Py_ssize_t given) {
  call_args a;
  int rc;
  if (!bound(lib.load_q8) || take(args, given, "ppippiiiilpp", &a) < 0) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = lib.load_q8(P(0), P(1), I32(2), P(3), P(4), I32(5), I32(6), I32(7), I32(8), I64(9), P(10),
                   P(11));
  Py_END_ALLOW_THREADS
  return status(rc);
}

static PyObject* decode_q8(PyObject* self, PyObject* const* args, Py_ssize_t given) {
  call_args a;
  int rc;
  if (!bound(lib.decode_q8) || take(args, given, "ppppipiiiiiilfipzpp", &a) < 0) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = lib.decode_q8(P(0), P(1), P(2), P(3), I32(4), P(5), I32(6), I32(7), I32(8), I32(9), I32(10),
                     I32(11), I64(12), a.f, I32(14), P(15), (size_t)a.v[16], P(17), P(18));
  Py_END_ALLOW_THREADS
  return status(rc);
}

static PyObject* rotary_store(PyObject* self, PyObject* const* args, Py_ssize_t given) {
  call_args a;
  int rc;
  if (!bound(lib.rotary) || take(args, given, "ppppllll" "iplpppp" "iiiiilpp", &a) < 0)
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = lib.rotary(P(0), P(1), P(2), P(3), I64(4), I64(5), I64(6), I64(7), I32(8), P(9), I64(10),
                  P(11), P(12), P(13), P(14), I32(15), I32(16), I32(17), I32(18), I32(19), I64(20),
                  P(21), P(22));
  Py_END_ALLOW_THREADS
  return status(rc);
}

static PyObject* rotary_store_q8(PyObject* self, PyObject* const* args, Py_ssize_t given) {
  call_args a;
  int rc;
  if (!bound(lib.rotary_q8) || take(args, given, "ppppllll" "iplppp" "iiiiilpp", &a) < 0)
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = lib.rotary_q8(P(0), P(1), P(2), P(3), I64(4), I64(5), I64(6), I64(7), I32(8), P(9), I64(10),
                     P(11), P(12), P(13), I32(14), I32(15), I32(16), I32(17), I32(18), I64(19),
                     P(20), P(21));
  Py_END_ALLOW_THREADS
  return status(rc);
}

/* bind(store_q8, load_q8, decode_q8, rotary_store, rotary_store_q8): the functions' addresses. */
static PyObject* bind_library(PyObject* self, PyObject* const* args, Py_ssize_t given) {
  call_args a;
  if (take(args, given, "ppppp", &a) < 0) return NULL;
  lib.store_q8 = (__typeof__(lib.store_q8))P(0);
  lib.load_q8 = (__typeof__(lib.load_q8))P(1);
  lib.decode_q8 = (__typeof__(lib.decode_q8))P(2);
  lib.rotary = (__typeof__(lib.rotary))P(3);
  lib.rotary_q8 = (__typeof__(lib.rotary_q8))P(4);
  Py_RETURN_NONE;
}

#define METHOD(name, fn, doc) {name, (PyCFunction)(void (*)(void))fn, METH_FASTCALL, doc}
static PyMethodDef methods[] = {
    METHOD("bind", bind_library, "Sets the library's functions by address."),
    METHOD("pa_store_kvcache_q8", store_q8, "pa_store_kvcache_q8 of pa.h."),
    METHOD("pa_load_kvcache_q8", load_q8, "pa_load_kvcache_q8 of pa.h."),
    METHOD("pa_decode_q8", decode_q8, "pa_decode_q8 of pa.h."),
    METHOD("pa_rotary_store", rotary_store, "pa_rotary_store of pa.h."),
    METHOD("pa_rotary_store_q8", rotary_store_q8, "pa_rotary_store_q8 of pa.h."),
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_call", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pa_call(void) { return PyModule_Create(&module); }
