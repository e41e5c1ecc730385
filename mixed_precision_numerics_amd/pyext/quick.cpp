// The common case of the norm, gated-activation and requantization calls from
// Python, in C: operands that are contiguous torch tensors on the current GPU
// with room for what the call spans.  A call of one token spends most of its
// time in the checks and conversions, not in the kernel.
//
// Each function takes its Python counterpart's arguments in order, then the
// stream's handle and the current device's index, and returns the entry
// point's status; None where an operand is anything else (an integer pointer,
// a view, a tensor that is too small, elsewhere, or no longer where an
// Fp8Tiles points): the caller then takes its own path, which names and refuses
// the operand or makes the call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "amp.h"

namespace {

PyTypeObject* g_tensor;   // torch.Tensor
PyTypeObject* g_tiles;    // Fp8Tiles
PyObject *g_get_device, *g_nbytes, *g_is_contiguous, *g_data_ptr, *g_tensors;

decltype(&amp_rmsnorm) g_rmsnorm;
decltype(&amp_rmsnorm_backward) g_rmsnorm_backward;
decltype(&amp_swiglu) g_swiglu;
decltype(&amp_swiglu_backward) g_swiglu_backward;
decltype(&amp_requantize_blockwise) g_requantize;

typedef __int128 wide;

int bytes_of(int64_t dt) {
  return dt == AMP_F32 ? 4 : dt == AMP_F16 || dt == AMP_BF16 ? 2 : dt == AMP_E4M3 || dt == AMP_E5M2 ? 1 : 0;
}
// Bytes that a matrix with row stride ld spans.
wide span(int64_t rows, int64_t cols, int64_t ld, int64_t dt) {
  return rows > 0 && cols > 0 ? (static_cast<wide>(rows - 1) * ld + cols) * bytes_of(dt) : 0;
}
int64_t blocks(int64_t n) { return n / 128 + (n % 128 > 0); }

// The arguments of a call; `ok` turns false at the first that is not plain.
struct Args {
  PyObject* const* v;
  int64_t dev;
  bool ok = true;

  int64_t num(PyObject* o) {
    if (!ok) return 0;
    if (!PyLong_Check(o)) { ok = false; return 0; }
    const long long n = PyLong_AsLongLong(o);
    if (n == -1 && PyErr_Occurred()) { PyErr_Clear(); ok = false; }
    return n;
  }
  int64_t num(int i) { return num(v[i]); }
  int type(int i) {
    const int64_t n = num(v[i]);
    if (n != static_cast<int>(n)) ok = false;
    return static_cast<int>(n);
  }
  // What a method (call) or an attribute of o gives, as a number.
  int64_t ask(PyObject* o, PyObject* name, bool call) {
    if (!ok) return 0;
    PyObject* r = call ? PyObject_CallMethodNoArgs(o, name) : PyObject_GetAttr(o, name);
    if (!r) { PyErr_Clear(); ok = false; return 0; }
    const int64_t n = num(r);   // True and False are 1 and 0
    Py_DECREF(r);
    return n;
  }
  void* mem(PyObject* o, wide need) {
    if (!ok || o == Py_None) return nullptr;
    if (!PyObject_TypeCheck(o, g_tensor) || ask(o, g_get_device, true) != dev || ask(o, g_nbytes, false) < need ||
        ask(o, g_is_contiguous, true) != 1) {
      ok = false;
      return nullptr;
    }
    return reinterpret_cast<void*>(ask(o, g_data_ptr, true));
  }
  void* mem(int i, wide need) { return mem(v[i], need); }
  template <typename T>
  T* mem(int i, wide need) { return static_cast<T*>(mem(v[i], need)); }
  // An Fp8Tiles [rows, cols] of nb tiles along K, copied to t.
  const amp_fp8_tiles* tiles(int i, int64_t rows, int64_t cols, int64_t nb, amp_fp8_tiles& t) {
    PyObject* o = v[i];
    if (!ok || o == Py_None) return nullptr;
    Py_buffer b;
    if (!PyObject_TypeCheck(o, g_tiles) || PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
      PyErr_Clear();
      ok = false;
      return nullptr;
    }
    ok = b.len == sizeof(t);
    if (ok) t = *static_cast<const amp_fp8_tiles*>(b.buf);
    PyBuffer_Release(&b);
    PyObject* qs = ok ? PyObject_GetAttr(o, g_tensors) : nullptr;
    if (!qs) PyErr_Clear();
    if (!qs || !PyTuple_Check(qs) || PyTuple_GET_SIZE(qs) != 2) {
      Py_XDECREF(qs);
      ok = false;
      return nullptr;
    }
    const bool some = rows > 0 && cols > 0;
    // where the structure was filled from them, and they have not moved since
    ok = mem(PyTuple_GET_ITEM(qs, 0), some ? static_cast<wide>(rows - 1) * t.ldq + cols : 0) == t.q && ok;
    ok = mem(PyTuple_GET_ITEM(qs, 1), some ? 4 * (static_cast<wide>(nb - 1) * t.lds + rows) : 0) == t.s && ok;
    Py_DECREF(qs);
    return ok ? &t : nullptr;
  }
};

#define AMP_OPEN(count)                                                            \
  if (n != (count) + 2) { PyErr_SetString(PyExc_TypeError, "argument count"); return nullptr; } \
  Args a{v, 0};                                                                    \
  void* const stream = reinterpret_cast<void*>(a.num(count));                      \
  a.dev = a.num((count) + 1)
#define AMP_CALL(expr)                  \
  if (!a.ok) Py_RETURN_NONE;            \
  int st;                               \
  Py_BEGIN_ALLOW_THREADS st = (expr);   \
  Py_END_ALLOW_THREADS return PyLong_FromLong(st)

PyObject* rmsnorm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  AMP_OPEN(20);
  const int xt = a.type(1), gt = a.type(8), yt = a.type(13);
  const int64_t rows = a.num(2), cols = a.num(3), ldx = a.num(4), ldr = a.num(6), ldh = a.num(11), ldy = a.num(14);
  if (!PyFloat_Check(v[9])) Py_RETURN_NONE;
  const float eps = static_cast<float>(PyFloat_AS_DOUBLE(v[9]));
  amp_fp8_tiles q, c;
  const void *x = a.mem(0, span(rows, cols, ldx, xt)), *res = a.mem(5, span(rows, cols, ldr, xt)),
             *gamma = a.mem(7, span(1, cols, cols, gt));
  void *h = a.mem(10, span(rows, cols, ldh, xt)), *y = a.mem(12, span(rows, cols, ldy, yt));
  const float* scale = a.mem<float>(15, 4);
  float* amax = a.mem<float>(16, 4);
  const amp_fp8_tiles *yq = a.tiles(17, rows, cols, blocks(cols), q), *ck = a.tiles(18, rows, cols, blocks(cols), c);
  float* rstd = a.mem<float>(19, span(1, rows, rows, AMP_F32));
  AMP_CALL(g_rmsnorm(x, xt, rows, cols, ldx, res, ldr, gamma, gt, eps, h, ldh, y, yt, ldy, scale, amax, yq, ck, rstd, stream));
}

PyObject* rmsnorm_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  AMP_OPEN(17);
  const int dt = a.type(1), gt = a.type(9);
  const int64_t rows = a.num(2), cols = a.num(3), lddy = a.num(4), ldh = a.num(6), lddr = a.num(12), lddx = a.num(14);
  amp_fp8_tiles c;
  const void *dy = a.mem(0, span(rows, cols, lddy, dt)), *h = a.mem(5, span(rows, cols, ldh, dt));
  const amp_fp8_tiles* ck = a.tiles(7, rows, cols, blocks(cols), c);
  const void* gamma = a.mem(8, span(1, cols, cols, gt));
  const float* rstd = a.mem<float>(10, span(1, rows, rows, AMP_F32));
  const void* dres = a.mem(11, span(rows, cols, lddr, dt));
  void* dx = a.mem(13, span(rows, cols, lddx, dt));
  float* dgamma = a.mem<float>(15, span(1, cols, cols, AMP_F32));
  float* work = a.mem<float>(16, dgamma ? span(rows < AMP_RMSNORM_PARTIALS ? rows : AMP_RMSNORM_PARTIALS, cols, cols, AMP_F32) : 0);
  AMP_CALL(g_rmsnorm_backward(dy, dt, rows, cols, lddy, h, ldh, ck, gamma, gt, rstd, dres, lddr, dx, lddx, dgamma, work, stream));
}

PyObject* swiglu(PyObject*, PyObject* const* v, Py_ssize_t n) {
  AMP_OPEN(12);
  const int xt = a.type(1), yt = a.type(6);
  const int64_t rows = a.num(2), cols = a.num(3), ldx = a.num(4), ldy = a.num(7);
  if (cols < 0 || cols > INT64_MAX / 4) Py_RETURN_NONE;
  amp_fp8_tiles q, c;
  const void* x = a.mem(0, span(rows, 2 * cols, ldx, xt));
  void* y = a.mem(5, span(rows, cols, ldy, yt));
  const float* scale = a.mem<float>(8, 4);
  float* amax = a.mem<float>(9, 4);
  const amp_fp8_tiles *yq = a.tiles(10, rows, cols, blocks(cols), q), *ck = a.tiles(11, rows, 2 * cols, 2 * blocks(cols), c);
  AMP_CALL(g_swiglu(x, xt, rows, cols, ldx, y, yt, ldy, scale, amax, yq, ck, stream));
}

PyObject* swiglu_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  AMP_OPEN(13);
  const int dt = a.type(1);
  const int64_t rows = a.num(2), cols = a.num(3), lddy = a.num(4), ldx = a.num(6), lddx = a.num(9);
  if (cols < 0 || cols > INT64_MAX / 4) Py_RETURN_NONE;
  amp_fp8_tiles c, q, qt, yt;
  const void *dy = a.mem(0, span(rows, cols, lddy, dt)), *x = a.mem(5, span(rows, 2 * cols, ldx, dt));
  const amp_fp8_tiles* ck = a.tiles(7, rows, 2 * cols, 2 * blocks(cols), c);
  void* dx = a.mem(8, span(rows, 2 * cols, lddx, dt));
  const amp_fp8_tiles *dxq = a.tiles(10, rows, 2 * cols, blocks(2 * cols), q), *dxqt = a.tiles(11, 2 * cols, rows, blocks(rows), qt),
                      *yqt = a.tiles(12, cols, rows, blocks(rows), yt);
  AMP_CALL(g_swiglu_backward(dy, dt, rows, cols, lddy, x, ldx, ck, dx, lddx, dxq, dxqt, yqt, stream));
}

PyObject* requantize(PyObject*, PyObject* const* v, Py_ssize_t n) {
  AMP_OPEN(7);
  const int64_t rows = a.num(1), cols = a.num(2);
  const int ct = a.type(5);
  amp_fp8_tiles x, q;
  const amp_fp8_tiles* xq = a.tiles(0, rows, cols, blocks(cols), x);
  const float* row = a.mem<float>(3, span(1, rows, rows, AMP_F32));
  const void* col = a.mem(4, span(1, cols, cols, ct));
  const amp_fp8_tiles* qt = a.tiles(6, cols, rows, blocks(rows), q);
  AMP_CALL(g_requantize(xq, rows, cols, row, col, ct, qt, stream));
}

// bind(torch.Tensor, Fp8Tiles, addresses of the five entry points)
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 7 || !PyType_Check(v[0]) || !PyType_Check(v[1])) { PyErr_SetString(PyExc_TypeError, "bind"); return nullptr; }
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(v[2 + i]);
    if (!p[i]) { if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind"); return nullptr; }
  }
  Py_INCREF(v[0]);
  Py_INCREF(v[1]);
  g_tensor = reinterpret_cast<PyTypeObject*>(v[0]);
  g_tiles = reinterpret_cast<PyTypeObject*>(v[1]);
  g_rmsnorm = reinterpret_cast<decltype(g_rmsnorm)>(p[0]);
  g_rmsnorm_backward = reinterpret_cast<decltype(g_rmsnorm_backward)>(p[1]);
  g_swiglu = reinterpret_cast<decltype(g_swiglu)>(p[2]);
  g_swiglu_backward = reinterpret_cast<decltype(g_swiglu_backward)>(p[3]);
  g_requantize = reinterpret_cast<decltype(g_requantize)>(p[4]);
  Py_RETURN_NONE;
}

#define AMP_DEF(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {AMP_DEF(bind), AMP_DEF(rmsnorm), AMP_DEF(rmsnorm_backward), AMP_DEF(swiglu), AMP_DEF(swiglu_backward),
                           AMP_DEF(requantize), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_quick", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__quick(void) {
  g_get_device = PyUnicode_InternFromString("get_device");
  g_nbytes = PyUnicode_InternFromString("nbytes");
  g_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  g_tensors = PyUnicode_InternFromString("tensors");
  return PyModule_Create(&g_module);
}
