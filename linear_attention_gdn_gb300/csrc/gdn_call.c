/*
 * gdn_call.c -- the short way from Python to the entry points that take single tokens.
 *
 * Such a call lasts a few microseconds on the GPU, and ctypes' conversion of a dozen arguments is of that order (a
 * call of gdn_step without its launch: 1.9 us through ctypes, 1.0 this way).  This module marshals only: it takes the
 * entry's address, the problem's address, the size argument (None: the entry has none), the stream and the pointer arguments
 * (None, an address, or an object with data_ptr()), calls the entry without the interpreter's lock and returns its status.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stddef.h>

#define MOST 14

typedef const void *P;
typedef int (*entry9)(P, P, P, P, P, P, P, P, P, P, P);
typedef int (*entry11)(P, P, P, P, P, P, P, P, P, P, P, P, P);
typedef int (*entry14)(P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, size_t, P);

static PyObject *data_ptr_name;

static int address(PyObject *o, P *out) {
  if (o == Py_None) {
    *out = NULL;
    return 1;
  }
  if (PyLong_Check(o)) {
    *out = PyLong_AsVoidPtr(o);
    return *out || !PyErr_Occurred();
  }
  PyObject *a = PyObject_CallMethodNoArgs(o, data_ptr_name);
  if (!a) return 0;
  *out = PyLong_AsVoidPtr(a);
  Py_DECREF(a);
  return *out || !PyErr_Occurred();
}

static PyObject *call(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  const Py_ssize_t count = n - 4;
  P entry, prob, stream, p[MOST];
  size_t size = 0;
  int status;
  (void)self;
  if (count != 9 && count != 11 && count != 14)
    return PyErr_Format(PyExc_TypeError, "call() takes 9, 11 or 14 pointers (%zd given)", count);
  if ((count == 14) != (args[2] != Py_None)) return PyErr_Format(PyExc_TypeError, "a size goes with 14 pointers");
  if (!address(args[0], &entry) || !address(args[1], &prob) || !address(args[3], &stream)) return NULL;
  if (args[2] != Py_None) {
    size = PyLong_AsSize_t(args[2]);
    if (size == (size_t)-1 && PyErr_Occurred()) return NULL;
  }
  for (Py_ssize_t i = 0; i < count; ++i)
    if (!address(args[4 + i], &p[i])) return NULL;
  Py_BEGIN_ALLOW_THREADS
  if (count == 9)
    status = ((entry9)entry)(prob, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], stream);
  else if (count == 11)
    status = ((entry11)entry)(prob, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], p[10], stream);
  else
    status = ((entry14)entry)(prob, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11], p[12],
                              p[13], size, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

static PyMethodDef methods[] = {
    {"call", (PyCFunction)(void (*)(void))call, METH_FASTCALL, "call(entry, problem, size or None, stream, *pointers)"},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdn_call", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__gdn_call(void) {
  data_ptr_name = PyUnicode_InternFromString("data_ptr");
  return data_ptr_name ? PyModule_Create(&module) : NULL;
}
