/* Python entry of the calls made once a token: the same C functions that the
 * ctypes binding reaches, with their (up to 35) arguments converted here, which
 * takes 0.5 us instead of 3.  Only the stable ABI is used, so that one build
 * serves every interpreter from 3.10 on.  Each takes its C function's arguments by
 * position (None: a NULL pointer) and returns the status. */
#define PY_SSIZE_T_CLEAN
#define Py_LIMITED_API 0x030A0000
#include <Python.h>
#include <limits.h>
#include <string.h>

#include "../../include/oidnx.h"

/* One letter an argument: p pointer, l long long, i int, f float. */
typedef union {
  void* p;
  long long l;
  int i;
  float f;
} Arg;

static int convert(const char* name, const char* kinds, PyObject* const* args, Py_ssize_t n, Arg* out) {
  const Py_ssize_t want = (Py_ssize_t)strlen(kinds);
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", name, want, n);
    return 0;
  }
  for (Py_ssize_t k = 0; k < n; ++k) {
    PyObject* a = args[k];
    if (kinds[k] == 'f') {
      const double v = PyFloat_AsDouble(a);
      if (v == -1.0 && PyErr_Occurred()) return 0;
      out[k].f = (float)v;
      continue;
    }
    if (kinds[k] == 'p') {
      if (a == Py_None) {
        out[k].p = NULL;
        continue;
      }
      const unsigned long long v = PyLong_AsUnsignedLongLong(a);
      if (v == (unsigned long long)-1 && PyErr_Occurred()) return 0;
      out[k].p = (void*)(uintptr_t)v;
      continue;
    }
    const long long v = PyLong_AsLongLong(a);
    if (v == -1 && PyErr_Occurred()) return 0;
    if (kinds[k] == 'i') {
      if (v < INT_MIN || v > INT_MAX) {
        PyErr_Format(PyExc_OverflowError, "%s: argument %zd is beyond a C int", name, k + 1);
        return 0;
      }
      out[k].i = (int)v;
    } else {
      out[k].l = v;
    }
  }
  return 1;
}

static PyObject* linear(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  Arg a[15];
  oidnx_status s;
  (void)self;
  if (!convert("oidnx_linear", "plplpplpliiiiip", args, n, a)) return NULL;
  Py_BEGIN_ALLOW_THREADS;
  s = oidnx_linear(a[0].p, a[1].l, a[2].p, a[3].l, a[4].p, a[5].p, a[6].l, a[7].p, a[8].l, a[9].i, a[10].i, a[11].i,
                   a[12].i, a[13].i, a[14].p);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(s);
}

static PyObject* qk_norm_rope(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  Arg a[35];
  oidnx_status s;
  (void)self;
  if (!convert("oidnx_qk_norm_rope", "pllpllpllpllpllpllppfpplppliiiiiiip", args, n, a)) return NULL;
  Py_BEGIN_ALLOW_THREADS;
  s = oidnx_qk_norm_rope(a[0].p, a[1].l, a[2].l, a[3].p, a[4].l, a[5].l, a[6].p, a[7].l, a[8].l, a[9].p, a[10].l,
                         a[11].l, a[12].p, a[13].l, a[14].l, a[15].p, a[16].l, a[17].l, a[18].p, a[19].p, a[20].f,
                         a[21].p, a[22].p, a[23].l, a[24].p, a[25].p, a[26].l, a[27].i, a[28].i, a[29].i, a[30].i,
                         a[31].i, a[32].i, a[33].i, a[34].p);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(s);
}

static PyObject* window_attention(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  Arg a[30];
  oidnx_status s;
  (void)self;
  if (!convert("oidnx_window_attention", "plllplllplllplllpppiiiiiiiifip", args, n, a)) return NULL;
  Py_BEGIN_ALLOW_THREADS;
  s = oidnx_window_attention(a[0].p, a[1].l, a[2].l, a[3].l, a[4].p, a[5].l, a[6].l, a[7].l, a[8].p, a[9].l, a[10].l,
                             a[11].l, a[12].p, a[13].l, a[14].l, a[15].l, a[16].p, a[17].p, a[18].p, a[19].i, a[20].i,
                             a[21].i, a[22].i, a[23].i, a[24].i, a[25].i, a[26].i, a[27].f, a[28].i, a[29].p);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(s);
}

static PyMethodDef methods[] = {
    {"oidnx_linear", (PyCFunction)(void (*)(void))linear, METH_FASTCALL, NULL},
    {"oidnx_qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, NULL},
    {"oidnx_window_attention", (PyCFunction)(void (*)(void))window_attention, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
