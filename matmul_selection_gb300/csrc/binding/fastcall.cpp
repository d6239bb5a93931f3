// Python entry of the operators that are called once a layer and token: the
// same C functions as through ctypes (include/mm.h), with the arguments
// converted here.  A call of mm_rmsnorm on one row takes 2 us on the device;
// through ctypes its 16 arguments alone took 3 us to convert.
//
// Each function takes its C function's arguments in order: pointers as None,
// an address, or an object with data_ptr(); the types as a tuple of three; the
// stream as None, a handle, or an object with cuda_stream.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../../include/mm.h"

namespace {

PyObject *g_data_ptr, *g_cuda_stream;  // interned names

bool address(PyObject *o, void **out) {
  if (o == Py_None) {
    *out = nullptr;
    return true;
  }
  if (PyLong_Check(o)) {
    *out = PyLong_AsVoidPtr(o);
    return !PyErr_Occurred();
  }
  PyObject *p = PyObject_CallMethodNoArgs(o, g_data_ptr);
  if (!p) return false;
  *out = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  return !PyErr_Occurred();
}
bool integer(PyObject *o, int64_t *out) {
  *out = PyLong_AsLongLong(o);
  return *out != -1 || !PyErr_Occurred();
}
bool types(PyObject *o, mm_dtypes *out) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3) {
    PyErr_SetString(PyExc_TypeError, "types: a tuple of three");
    return false;
  }
  int64_t v[3];
  for (int i = 0; i < 3; ++i) {
    if (!integer(PyTuple_GET_ITEM(o, i), &v[i])) return false;
    if (v[i] < INT32_MIN || v[i] > INT32_MAX) v[i] = -1;  // no type: refused by the call
  }
  out->a = (int32_t)v[0];
  out->b = (int32_t)v[1];
  out->c = (int32_t)v[2];
  return true;
}
bool stream_of(PyObject *o, void **out) {
  if (o == Py_None || PyLong_Check(o)) return address(o, out);
  PyObject *p = PyObject_GetAttr(o, g_cuda_stream);
  if (!p) return false;
  *out = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  return !PyErr_Occurred();
}

// P pointers, then I integers.
template <int P, int I>
bool convert(const char *name, PyObject *const *args, Py_ssize_t n, int more, void *(&p)[P], int64_t (&i)[I]) {
  if (n != P + I + more) {
    PyErr_Format(PyExc_TypeError, "%s takes %d arguments (%d given)", name, P + I + more, (int)n);
    return false;
  }
  for (int k = 0; k < P; ++k)
    if (!address(args[k], &p[k])) return false;
  for (int k = 0; k < I; ++k)
    if (!integer(args[P + k], &i[k])) return false;
  return true;
}

PyObject *rmsnorm(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void *p[7], *s;
  int64_t i[6];
  mm_dtypes t;
  if (!convert("mm_rmsnorm", args, n, 3, p, i) || !types(args[13], &t)) return nullptr;
  const double eps = PyFloat_AsDouble(args[14]);
  if ((eps == -1.0 && PyErr_Occurred()) || !stream_of(args[15], &s)) return nullptr;
  mm_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = mm_rmsnorm(p[0], p[1], p[2], p[3], p[4], (float *)p[5], (float *)p[6], i[0], i[1], i[2], i[3], i[4], i[5], t,
                  (float)eps, s);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

PyObject *rmsnorm_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void *p[7], *s;
  int64_t i[6];
  mm_dtypes t;
  if (!convert("mm_rmsnorm_backward", args, n, 3, p, i) || !types(args[13], &t)) return nullptr;
  const double eps = PyFloat_AsDouble(args[14]);
  if ((eps == -1.0 && PyErr_Occurred()) || !stream_of(args[15], &s)) return nullptr;
  mm_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = mm_rmsnorm_backward(p[0], p[1], p[2], p[3], (const float *)p[4], p[5], p[6], i[0], i[1], i[2], i[3], i[4],
                           i[5], t, (float)eps, s);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

PyObject *gemm_w4(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void *p[5], *s;
  int64_t i[8];
  mm_dtypes t;
  if (!convert("mm_gemm_w4", args, n, 2, p, i) || !types(args[13], &t) || !stream_of(args[14], &s)) return nullptr;
  if (i[7] < INT32_MIN || i[7] > INT32_MAX) i[7] = 0;  // no group: refused by the call
  mm_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = mm_gemm_w4(p[0], p[1], p[2], p[3], p[4], i[0], i[1], i[2], i[3], i[4], i[5], i[6], (int32_t)i[7], t, s);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

PyObject *gemm_q8(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void *p[5], *s;
  int64_t i[6];
  mm_dtypes t;
  if (!convert("mm_gemm_q8", args, n, 2, p, i) || !types(args[11], &t) || !stream_of(args[12], &s)) return nullptr;
  mm_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = mm_gemm_q8(p[0], p[1], (const float *)p[2], (const float *)p[3], p[4], i[0], i[1], i[2], i[3], i[4], i[5], t, s);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

PyObject *embedding(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void *p[3], *s;
  int64_t i[5];
  mm_dtypes t;
  if (!convert("mm_embedding", args, n, 3, p, i) || !types(args[8], &t)) return nullptr;
  const double scale = PyFloat_AsDouble(args[9]);
  if ((scale == -1.0 && PyErr_Occurred()) || !stream_of(args[10], &s)) return nullptr;
  mm_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = mm_embedding(p[0], p[1], p[2], i[0], i[1], i[2], i[3], i[4], t, (float)scale, s);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

PyObject *embedding_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void *p[4], *s;
  int64_t i[6];
  mm_dtypes t;
  if (!convert("mm_embedding_backward", args, n, 3, p, i) || !types(args[10], &t)) return nullptr;
  const double scale = PyFloat_AsDouble(args[11]);
  if ((scale == -1.0 && PyErr_Occurred()) || !stream_of(args[12], &s)) return nullptr;
  mm_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = mm_embedding_backward(p[0], p[1], p[2], p[3], i[0], i[1], i[2], i[3], i[4], i[5], t, (float)scale, s);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

PyObject *cross_entropy(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void *p[5], *s;
  int64_t i[5];
  mm_dtypes t;
  if (!convert("mm_cross_entropy", args, n, 2, p, i) || !types(args[10], &t) || !stream_of(args[11], &s))
    return nullptr;
  mm_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = mm_cross_entropy(p[0], p[1], p[2], (float *)p[3], (float *)p[4], i[0], i[1], i[2], i[3], i[4], t, s);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

PyObject *cross_entropy_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void *p[7], *s;
  int64_t i[7];
  mm_dtypes t;
  if (!convert("mm_cross_entropy_backward", args, n, 2, p, i) || !types(args[14], &t) || !stream_of(args[15], &s))
    return nullptr;
  mm_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = mm_cross_entropy_backward(p[0], p[1], p[2], (const float *)p[3], (const float *)p[4], p[5], p[6], i[0], i[1],
                                 i[2], i[3], i[4], i[5], i[6], t, s);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

#define MM_FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {MM_FAST(rmsnorm), MM_FAST(rmsnorm_backward), MM_FAST(gemm_w4), MM_FAST(gemm_q8),
                           MM_FAST(embedding), MM_FAST(embedding_backward), MM_FAST(cross_entropy),
                           MM_FAST(cross_entropy_backward),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "mm_fastcall", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mm_fastcall(void) {
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  g_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (!g_data_ptr || !g_cuda_stream) return nullptr;
  return PyModule_Create(&g_module);
}
