// The common case of the norm, gated-activation and requantization calls, of the
// gated feed-forward block and of the calls over lists of tensors from Python, in
// C: operands that are contiguous torch tensors on the current GPU with room for
// what the call spans.  A call of one token spends most of its time in the checks
// and conversions, not in the kernel.
//
// Each function takes its Python counterpart's arguments in order, then the
// stream's handle and the current device's index, and returns the entry
// point's status; None where an operand is anything else (an integer pointer,
// a view, a tensor that is too small, elsewhere, or no longer where an
// Fp8Tiles points): the caller then takes its own path, which names and refuses
// the operand or makes the call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#if __has_include(<ATen/dlpack.h>)
#include <ATen/dlpack.h>
#endif

#include <algorithm>
#include <new>
#include <vector>

#include "amp.h"

namespace {

PyTypeObject* g_tensor;   // torch.Tensor
PyTypeObject* g_tiles;    // Fp8Tiles
PyTypeObject* g_list;     // TensorList
PyObject *g_get_device, *g_nbytes, *g_is_contiguous, *g_data_ptr, *g_tensors, *g_array, *g_held, *g_where, *g_apart, *g_serial, *g_beside;
PyObject* g_where_is;      // torch.Tensor.data_ptr

typedef __int128 wide;

// Where torch offers DLPack's exchange functions, what a call needs to know of a
// tensor is one plain call instead of four of its methods (clipping of 700 tensors
// into others 90 -> 71 us, 60 since what they are compared with is one
// buffer; the norm of four tensors 11.3 -> 10.6).
enum Look { kUnseen, kPlain, kOther };
#if defined(DLPACK_MAJOR_VERSION) && (DLPACK_MAJOR_VERSION > 1 || (DLPACK_MAJOR_VERSION == 1 && DLPACK_MINOR_VERSION >= 3))
DLPackDLTensorFromPyObjectNoSync g_view;
void bind_view() {
  PyObject* c = PyObject_GetAttrString(reinterpret_cast<PyObject*>(g_tensor), "__dlpack_c_exchange_api__");
  const auto* api = c ? static_cast<const DLPackExchangeAPI*>(PyCapsule_GetPointer(c, "dlpack_exchange_api")) : nullptr;
  g_view = api && api->header.version.major == DLPACK_MAJOR_VERSION ? api->dltensor_from_py_object_no_sync : nullptr;
  Py_XDECREF(c);             // the functions are static
  PyErr_Clear();
}
bool view(PyObject* t, DLTensor& v) {
  if (g_view && g_view(t, &v) == 0) return true;
  PyErr_Clear();
  return false;
}
wide bytes_per(const DLTensor& v) { return (static_cast<wide>(v.dtype.bits) * v.dtype.lanes + 7) / 8; }
// A tensor's address and the bytes of its elements.
bool place(PyObject* t, uint64_t& p, wide& bytes) {
  DLTensor v;
  if (!view(t, v)) return false;
  p = reinterpret_cast<uint64_t>(v.data) + v.byte_offset;
  bytes = bytes_per(v);
  for (int32_t i = 0; i < v.ndim; ++i) bytes *= v.shape[i];
  return true;
}
// Whether t is contiguous, on GPU dev and holds `need` bytes; its address.
Look look(PyObject* t, int64_t dev, wide need, void*& p) {
  DLTensor v;
  if (!view(t, v)) return kUnseen;
  if ((v.device.device_type != kDLROCM && v.device.device_type != kDLCUDA) || v.device.device_id != dev) return kOther;
  wide n = 1;
  for (int32_t i = v.ndim - 1; i >= 0; --i) {
    if (v.strides && v.shape[i] != 1 && v.strides[i] != n) return kOther;      // (an empty tensor may count as one with gaps)
    n *= v.shape[i];
  }
  if (n * bytes_per(v) < need) return kOther;
  p = static_cast<char*>(v.data) + v.byte_offset;
  return kPlain;
}
#else
void bind_view() {}
bool place(PyObject*, uint64_t&, wide&) { return false; }
Look look(PyObject*, int64_t, wide, void*&) { return kUnseen; }
#endif

decltype(&amp_rmsnorm) g_rmsnorm;
decltype(&amp_rmsnorm_backward) g_rmsnorm_backward;
decltype(&amp_swiglu) g_swiglu;
decltype(&amp_swiglu_backward) g_swiglu_backward;
decltype(&amp_requantize_blockwise) g_requantize;
decltype(&amp_gemm_swiglu) g_gemm_swiglu;
decltype(&amp_gemm_swiglu_backward) g_gemm_swiglu_backward;
decltype(&amp_grad_norm_list) g_norm_list;
decltype(&amp_grad_clip_list) g_clip_list;

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
    void* p = nullptr;
    const Look seen = PyObject_TypeCheck(o, g_tensor) ? look(o, dev, need, p) : kOther;
    if (seen == kPlain) return p;
    if (seen == kOther || ask(o, g_get_device, true) != dev || ask(o, g_nbytes, false) < need ||
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
  // The array of a TensorList whose tensors are where they were and still hold the
  // elements.
  const amp_tensor* list(int i, int32_t& count) {
    PyObject* o = v[i];
    count = 0;
    if (!ok || o == Py_None) return nullptr;
    PyObject *a = nullptr, *ts = nullptr, *held = nullptr;
    Py_buffer b{}, h{};
    if (!PyObject_TypeCheck(o, g_list) || !(a = PyObject_GetAttr(o, g_array)) || !(ts = PyObject_GetAttr(o, g_tensors)) ||
        !(held = PyObject_GetAttr(o, g_held)) || !PyList_Check(ts) || PyObject_GetBuffer(a, &b, PyBUF_SIMPLE) != 0 ||
        PyObject_GetBuffer(held, &h, PyBUF_SIMPLE) != 0 || h.len != 16 * PyList_GET_SIZE(ts))
      ok = false;
    const int64_t* was = static_cast<const int64_t*>(h.buf);      // address and bytes of each tensor
    const amp_tensor* p = ok ? static_cast<const amp_tensor*>(b.buf) : nullptr;
    if (ok) count = static_cast<int32_t>(b.len / static_cast<Py_ssize_t>(sizeof(amp_tensor)));
    if (ok && PyList_GET_SIZE(ts) > 0) ok = ask(o, g_where, false) == dev && ok;
    for (Py_ssize_t k = 0; ok && k < PyList_GET_SIZE(ts); ++k, was += 2) {
      PyObject* t = PyList_GET_ITEM(ts, k);
      uint64_t p;
      wide bytes;
      if (!PyObject_TypeCheck(t, g_tensor)) {
        ok = false;
      } else if (place(t, p, bytes)) {
        ok = static_cast<int64_t>(p) == was[0] && bytes >= was[1];
      } else if (ask(t, g_nbytes, false) < was[1]) {
        ok = false;
      } else {
        PyObject* r = PyObject_Vectorcall(g_where_is, &t, 1, nullptr);
        ok = r && num(r) == was[0] && ok;
        Py_XDECREF(r);
      }
    }
    PyErr_Clear();
    if (b.obj) PyBuffer_Release(&b);
    if (h.obj) PyBuffer_Release(&h);
    Py_XDECREF(a);                     // the list keeps its array
    Py_XDECREF(ts);
    Py_XDECREF(held);
    return ok ? p : nullptr;
  }
  // TensorList.clear_of: whether the lists are known to lie clear of each other, or
  // found to (700 outputs: 4 us in order of their addresses, 8 in any, once a pair).
  static bool clear_of(PyObject* outs, PyObject* grads, const amp_tensor* o, const amp_tensor* g, int32_t count) {
    PyObject *known = PyObject_GetAttr(outs, g_beside), *serial = PyObject_GetAttr(grads, g_serial);
    bool yes = known && serial && PySet_Check(known);
    if (yes && PySet_Contains(known, serial) != 1) {
      yes = apart(o, g, count);
      if (yes && PySet_GET_SIZE(known) >= 64) PySet_Clear(known);
      if (yes) PySet_Add(known, serial);
    }
    Py_XDECREF(known);
    Py_XDECREF(serial);
    PyErr_Clear();
    return yes;
  }
  // Outputs that lie over none of one another, beside all gradients but their own.
  static bool apart(const amp_tensor* o, const amp_tensor* g, int32_t count) {
    auto begin = [](const amp_tensor& t) { return reinterpret_cast<uintptr_t>(t.p); };
    auto end = [&](const amp_tensor& t) { return begin(t) + static_cast<uintptr_t>(t.n) * bytes_of(t.type); };
    auto lower = [&](int32_t i, int32_t j) { return begin(o[i]) < begin(o[j]); };
    std::vector<int32_t> at;
    try {
      at.reserve(count);
    } catch (const std::bad_alloc&) {
      return false;
    }
    for (int32_t i = 0; i < count; ++i)
      if (o[i].n > 0 && o[i].p) at.push_back(i);
    if (!std::is_sorted(at.begin(), at.end(), lower)) std::sort(at.begin(), at.end(), lower);
    for (int32_t i = 0; i < count; ++i) {
      if (g[i].n <= 0 || !g[i].p) continue;
      // the last output that begins before the gradient's end
      auto k = std::lower_bound(at.begin(), at.end(), end(g[i]), [&](int32_t j, uintptr_t e) { return begin(o[j]) < e; });
      if (k == at.begin()) continue;
      const int32_t j = *--k;
      if (end(o[j]) > begin(g[i]) && (j != i || o[j].p != g[i].p || o[j].type != g[i].type)) return false;
    }
    return true;
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

PyObject* gemm_swiglu(PyObject*, PyObject* const* v, Py_ssize_t n) {
  AMP_OPEN(12);
  const int64_t M = a.num(0), F = a.num(1), K = a.num(2), ldx = a.num(5), ldw = a.num(7), ldy = a.num(9), ldgu = a.num(11);
  const int t = a.type(4);
  if (F < 0 || F > INT64_MAX / 4) Py_RETURN_NONE;
  const void *x = a.mem(3, span(M, K, ldx, t)), *w = a.mem(6, span(2 * F, K, ldw, t));
  void *y = a.mem(8, span(M, F, ldy, t)), *gu = a.mem(10, span(M, 2 * F, ldgu, t));
  AMP_CALL(g_gemm_swiglu(M, F, K, x, t, ldx, w, ldw, y, ldy, gu, ldgu, stream));
}

PyObject* gemm_swiglu_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  AMP_OPEN(22);
  const int64_t M = a.num(0), F = a.num(1), K = a.num(2), lddy = a.num(5), ldx = a.num(7), ldw = a.num(9), ldgu = a.num(11),
                lddgu = a.num(13), ldy = a.num(15), lddx = a.num(17), lddw = a.num(20);
  const int t = a.type(4), dwt = a.type(19);
  if (F < 0 || F > INT64_MAX / 4) Py_RETURN_NONE;
  const void *dy = a.mem(3, span(M, F, lddy, t)), *x = a.mem(6, span(M, K, ldx, t)), *w = a.mem(8, span(2 * F, K, ldw, t)),
             *gu = a.mem(10, span(M, 2 * F, ldgu, t));
  void *dgu = a.mem(12, span(M, 2 * F, lddgu, t)), *y = a.mem(14, span(M, F, ldy, t)), *dx = a.mem(16, span(M, K, lddx, t)),
       *dw = a.mem(18, span(2 * F, K, lddw, dwt));
  float* work = a.mem<float>(21, span(1, AMP_GEMM_SWIGLU_WORK, AMP_GEMM_SWIGLU_WORK, AMP_F32));
  AMP_CALL(g_gemm_swiglu_backward(M, F, K, dy, t, lddy, x, ldx, w, ldw, gu, ldgu, dgu, lddgu, y, ldy, dx, lddx, dw, dwt, lddw, work,
                                  stream));
}

PyObject* norm_list(PyObject*, PyObject* const* v, Py_ssize_t n) {
  AMP_OPEN(6);
  int32_t count;
  const amp_tensor* grads = a.list(0, count);
  const int first = PyObject_IsTrue(v[1]);
  amp_scaler_state* state = a.mem<amp_scaler_state>(2, sizeof(amp_scaler_state));
  amp_grad_norm_state* norm = a.mem<amp_grad_norm_state>(3, sizeof(amp_grad_norm_state));
  float* out = a.mem<float>(5, 8);
  if (first < 0) PyErr_Clear();
  if (first < 0 || !grads || !PyFloat_Check(v[4])) Py_RETURN_NONE;
  const float max_norm = static_cast<float>(PyFloat_AS_DOUBLE(v[4]));
  AMP_CALL(g_norm_list(grads, count, first, state, norm, max_norm, out, stream));
}

PyObject* clip_list(PyObject*, PyObject* const* v, Py_ssize_t n) {
  AMP_OPEN(4);
  int32_t count, as_many;
  const amp_tensor *grads = a.list(0, count), *outs = a.list(1, as_many);
  const amp_scaler_state* state = a.mem<amp_scaler_state>(2, sizeof(amp_scaler_state));
  const float* coef = a.mem<float>(3, 4);
  if (!a.ok || !grads || (outs && as_many != count) || a.ask(v[outs ? 1 : 0], g_apart, false) != 1) Py_RETURN_NONE;
  if (outs && !a.clear_of(v[1], v[0], outs, grads, count)) Py_RETURN_NONE;
  AMP_CALL(g_clip_list(grads, outs, count, state, coef, stream));
}

// bind_block(TensorList, addresses of the four entry points above), after bind
PyObject* bind_block(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 5 || !PyType_Check(v[0]) || !g_tensor) { PyErr_SetString(PyExc_TypeError, "bind_block"); return nullptr; }
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(v[1 + i]);
    if (!p[i]) { if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind_block"); return nullptr; }
  }
  Py_INCREF(v[0]);
  g_where_is = PyObject_GetAttr(reinterpret_cast<PyObject*>(g_tensor), g_data_ptr);
  if (!g_where_is) return nullptr;
  bind_view();
  g_list = reinterpret_cast<PyTypeObject*>(v[0]);
  g_gemm_swiglu = reinterpret_cast<decltype(g_gemm_swiglu)>(p[0]);
  g_gemm_swiglu_backward = reinterpret_cast<decltype(g_gemm_swiglu_backward)>(p[1]);
  g_norm_list = reinterpret_cast<decltype(g_norm_list)>(p[2]);
  g_clip_list = reinterpret_cast<decltype(g_clip_list)>(p[3]);
  Py_RETURN_NONE;
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
                           AMP_DEF(requantize), AMP_DEF(bind_block), AMP_DEF(gemm_swiglu), AMP_DEF(gemm_swiglu_backward), AMP_DEF(norm_list),
                           AMP_DEF(clip_list), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_quick", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__quick(void) {
  g_get_device = PyUnicode_InternFromString("get_device");
  g_nbytes = PyUnicode_InternFromString("nbytes");
  g_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  g_tensors = PyUnicode_InternFromString("tensors");
  g_array = PyUnicode_InternFromString("array");
  g_held = PyUnicode_InternFromString("held");
  g_where = PyUnicode_InternFromString("where");
  g_apart = PyUnicode_InternFromString("apart");
  g_serial = PyUnicode_InternFromString("serial");
  g_beside = PyUnicode_InternFromString("beside");
  return PyModule_Create(&g_module);
}
