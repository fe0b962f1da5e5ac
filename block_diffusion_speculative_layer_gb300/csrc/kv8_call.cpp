// The three 8-bit cache calls as CPython functions.
//
// A decode step's call is a few microseconds of GPU work, and converting its
// 27 arguments through ctypes costs 2 us of host time; here it costs a tenth
// of that.  The functions take the C calls' arguments in their order and
// return the status; the library's entry points are handed over by bind(), so
// this module links against nothing.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "dflash.h"

static decltype(&df_op_kv8_write) g_write = nullptr;
static decltype(&df_op_kv8_read) g_read = nullptr;
static decltype(&df_op_attention_kv8) g_attention = nullptr;

namespace {

// Reads positional arguments one after the other; stops at the first bad one.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, i = 0;
  bool ok = true;
  Args(PyObject* const* args, Py_ssize_t count, Py_ssize_t want) : a(args), n(count) {
    if (count != want) {
      PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, count);
      ok = false;
    }
  }
  void* ptr() {
    if (!ok) return nullptr;
    PyObject* o = a[i++];
    if (o == Py_None) return nullptr;
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) ok = false;
    return p;
  }
  int64_t i64() {
    if (!ok) return 0;
    const long long v = PyLong_AsLongLong(a[i++]);
    if (v == -1 && PyErr_Occurred()) ok = false;
    return v;
  }
  int32_t i32() {
    const int64_t v = i64();
    if (ok && (v > INT32_MAX || v < INT32_MIN)) {
      PyErr_SetString(PyExc_OverflowError, "argument does not fit 32 bits");
      ok = false;
    }
    return (int32_t)v;
  }
  float f32() {
    if (!ok) return 0.f;
    const double v = PyFloat_AsDouble(a[i++]);
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return (float)v;
  }
};

PyObject* finish(bool bound) {
  if (!bound && !PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
  return nullptr;
}

}  // namespace

static PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Args r(a, n, 3);
  void *w = r.ptr(), *d = r.ptr(), *t = r.ptr();
  if (!r.ok) return nullptr;
  g_write = reinterpret_cast<decltype(g_write)>(w);
  g_read = reinterpret_cast<decltype(g_read)>(d);
  g_attention = reinterpret_cast<decltype(g_attention)>(t);
  Py_RETURN_NONE;
}

static PyObject* py_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Args r(a, n, 19);
  const void *k = r.ptr(), *v = r.ptr();
  const int32_t dtype = r.i32(), rows = r.i32();
  const int64_t ks = r.i64(), vs = r.i64();
  void *codes = r.ptr(), *exps = r.ptr();
  const int32_t pages = r.i32(), page = r.i32(), heads = r.i32(), hd = r.i32();
  const int32_t* table = (const int32_t*)r.ptr();
  const int32_t entries = r.i32();
  const int32_t *start = (const int32_t*)r.ptr(), *len = (const int32_t*)r.ptr();
  const int32_t nseq = r.i32();
  int32_t* err = (int32_t*)r.ptr();
  void* stream = r.ptr();
  if (!r.ok || !g_write) return finish(g_write != nullptr);
  df_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_write(k, v, dtype, rows, ks, vs, codes, exps, pages, page, heads, hd, table, entries, start, len, nseq, err,
               stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

static PyObject* py_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Args r(a, n, 17);
  const void *codes = r.ptr(), *exps = r.ptr();
  const int32_t pages = r.i32(), page = r.i32(), heads = r.i32(), hd = r.i32();
  const int32_t* table = (const int32_t*)r.ptr();
  const int32_t entries = r.i32();
  const int32_t *start = (const int32_t*)r.ptr(), *len = (const int32_t*)r.ptr();
  const int32_t nseq = r.i32(), rows = r.i32(), dtype = r.i32();
  void *k = r.ptr(), *v = r.ptr();
  int32_t* err = (int32_t*)r.ptr();
  void* stream = r.ptr();
  if (!r.ok || !g_read) return finish(g_read != nullptr);
  df_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_read(codes, exps, pages, page, heads, hd, table, entries, start, len, nseq, rows, dtype, k, v, err, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

static PyObject* py_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Args r(a, n, 26);
  const void* q = r.ptr();
  const int64_t qs = r.i64();
  void* out = r.ptr();
  const int64_t os = r.i64();
  float* lse = (float*)r.ptr();
  const int32_t rows = r.i32(), hq = r.i32();
  const void *codes = r.ptr(), *exps = r.ptr();
  const int32_t pages = r.i32(), page = r.i32(), heads = r.i32(), hd = r.i32();
  const int32_t* table = (const int32_t*)r.ptr();
  const int32_t entries = r.i32();
  const int32_t *start = (const int32_t*)r.ptr(), *len = (const int32_t*)r.ptr();
  const int32_t nseq = r.i32(), max_rows = r.i32(), max_len = r.i32();
  const float scale = r.f32();
  const int32_t causal = r.i32(), window = r.i32(), cluster = r.i32();
  int32_t* err = (int32_t*)r.ptr();
  void* stream = r.ptr();
  if (!r.ok || !g_attention) return finish(g_attention != nullptr);
  df_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_attention(q, qs, out, os, lse, rows, hq, codes, exps, pages, page, heads, hd, table, entries, start, len, nseq,
                   max_rows, max_len, scale, causal, window, cluster, err, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))py_bind, METH_FASTCALL, "bind(write, read, attention): entry point addresses"},
    {"write", (PyCFunction)(void (*)(void))py_write, METH_FASTCALL, "df_op_kv8_write"},
    {"read", (PyCFunction)(void (*)(void))py_read, METH_FASTCALL, "df_op_kv8_read"},
    {"attention", (PyCFunction)(void (*)(void))py_attention, METH_FASTCALL, "df_op_attention_kv8"},
    {nullptr, nullptr, 0, nullptr}};
static PyModuleDef module = {PyModuleDef_HEAD_INIT, "kv8_call", "8-bit cache calls", -1, methods,
                             nullptr, nullptr, nullptr, nullptr};
PyMODINIT_FUNC PyInit_kv8_call(void) { return PyModule_Create(&module); }
