// The quick form of kdn.py's calls of the linear recurrence, the residual norm
// and the 8-bit projections: the same checks, output allocations and call of the
// C entry point, in one C++ function each (a small call is bound by its host
// side: scan step 10.4 us through ctypes, norm of 256 rows 13.8).  A function
// returns None for anything out of the ordinary, an argument that a check
// refuses, and has then enqueued nothing; kdn.py goes on in Python, which finds
// the words for it.  An error of the CUDA runtime is raised here: something may
// have been enqueued before it, and is not enqueued again.
#include <Python.h>

#include <ATen/Functions.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "../../include/kdn.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Unusual {};
struct Failed {
  kdn_status status;
  const char* where;
};

constexpr ScalarType F32 = ScalarType::Float, BF16 = ScalarType::BFloat16,
                     E4M3 = ScalarType::Float8_e4m3fn;

void usual(bool ok) {
  if (!ok) throw Unusual();
}
// An entry point's call, without the interpreter's lock (a launch waits when
// the stream's queue is full).
template <typename F, typename... A>
void call(const char* name, F f, A... args) {
  PyThreadState* s = PyEval_SaveThread();
  const kdn_status st = f(args...);
  PyEval_RestoreThread(s);
  usual(st != KDN_ERR_INVALID_ARG && st != KDN_ERR_UNSUPPORTED && st != KDN_ERR_WORKSPACE);
  if (st != KDN_OK) throw Failed{st, name};
}
#define KDN_CALL(f, ...) call(#f, f, __VA_ARGS__)
// kdn.KdnError
void raise(const Failed& e) {
  PyObject* module = PyImport_ImportModule("kalman_filter_linear_b200.kdn");
  PyObject* type = module ? PyObject_GetAttrString(module, "KdnError") : nullptr;
  PyObject* error = type ? PyObject_CallFunction(type, "is", (int)e.status, e.where) : nullptr;
  if (error) PyErr_SetObject(type, error);
  Py_XDECREF(error);
  Py_XDECREF(type);
  Py_XDECREF(module);
}
const Tensor* opt(PyObject* o) {
  if (o == Py_None) return nullptr;
  usual(THPVariable_Check(o));
  return &THPVariable_Unpack(o);
}
const Tensor& need(PyObject* o) {
  const Tensor* t = opt(o);
  usual(t != nullptr);
  return *t;
}
kdn_dtype code(const Tensor& t) {
  usual(t.scalar_type() == F32 || t.scalar_type() == BF16);
  return t.scalar_type() == F32 ? KDN_F32 : KDN_BF16;
}
// The device that a call runs on, which has to be the current one.
struct Place {
  at::Device device;
  explicit Place(const Tensor& t) : device(t.device()) {
    usual(device.is_cuda() && device.index() == c10::cuda::current_device());
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
  Tensor empty(at::IntArrayRef shape, ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(device));
  }
  void* arg(const Tensor* t, ScalarType type, at::IntArrayRef shape) const {
    if (!t) return nullptr;
    usual(t->scalar_type() == type && t->device() == device && t->sizes() == shape &&
          t->is_contiguous());
    return t->data_ptr();
  }
  // an output: the caller's, checked, or a new one
  Tensor out(PyObject* given, ScalarType type, at::IntArrayRef shape) const {
    const Tensor* t = opt(given);
    if (!t) return empty(shape, type);
    arg(t, type, shape);
    return *t;
  }
  // an 8-bit matrix and the distance of its rows
  void* fp8(const Tensor& t, int64_t rows, int64_t cols, int64_t* ld) const {
    usual(t.dim() == 2 && t.scalar_type() == E4M3 && t.device() == device && t.size(0) == rows &&
          t.size(1) == cols);
    *ld = rows > 1 ? t.stride(0) : (cols + 15) / 16 * 16;
    usual((cols <= 1 || t.stride(1) == 1) && *ld % 16 == 0 && *ld >= cols);
    return t.data_ptr();
  }
  Tensor fp8_empty(int64_t rows, int64_t cols) const {
    const int64_t ld = (cols + 15) / 16 * 16;
    Tensor q = empty({rows, ld}, E4M3);
    return ld == cols ? q : q.narrow(1, 0, cols);
  }
};

// The scan's workspace: a word that nobody reads where it needs no more (as
// kdn.py's), else new memory.
Tensor scan_workspace(const Place& p, size_t bytes) {
  static Tensor* words[64];  // (under the interpreter's lock; kept for good)
  const int i = p.device.index();
  if (bytes > 256 || i >= 64) return p.empty({(int64_t)bytes}, ScalarType::Byte);
  if (!words[i]) words[i] = new Tensor(p.empty({256}, ScalarType::Byte));
  return *words[i];
}
struct Scan {
  int64_t B, T, D;
  size_t bytes;
  Scan(const Tensor& a, const Tensor* cu) {
    usual(a.dim() == (cu ? 2 : 3) && a.is_contiguous());
    B = cu ? cu->numel() - 1 : a.size(0);
    T = a.size(cu ? 0 : 1);
    D = a.size(cu ? 1 : 2);
    usual(B >= 1 && B < 0x7fffffff && T < 0x7fffffff && D < 0x7fffffff);
    bytes = kdn_linear_scan_workspace_size(cu ? 1 : (int)B, (int)T, (int)D);
    usual(bytes > 0);
  }
};

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
void put(PyObject* dict, const char* key, PyObject* value) {
  PyDict_SetItemString(dict, key, value);
  Py_DECREF(value);
}

// a, x, h, b, y
PyObject* scan_step(PyObject* const* v) {
  const Tensor &a = need(v[0]), &x = need(v[1]), &h = need(v[2]), *b = opt(v[3]);
  const Place p(a);
  usual(a.dim() == 2 && a.size(0) < 0x7fffffff && a.size(1) < 0x7fffffff);
  const auto shape = a.sizes();
  const kdn_dtype gate = code(a), in = code(x);
  void *pa = p.arg(&a, a.scalar_type(), shape), *pb = p.arg(b, a.scalar_type(), shape);
  void *px = p.arg(&x, x.scalar_type(), shape), *ph = p.arg(&h, F32, shape);
  Tensor y = p.out(v[4], x.scalar_type(), shape);
  KDN_CALL(kdn_linear_scan_step, pa, pb, gate, px, in, static_cast<float*>(ph), y.data_ptr(),
                             (int)shape[0], (int)shape[1], p.stream());
  return wrap(y);
}

// a, x, b, h0, cu_seqlens, y, h_out
PyObject* scan_forward(PyObject* const* v) {
  const Tensor &a = need(v[0]), &x = need(v[1]), *b = opt(v[2]), *h0 = opt(v[3]), *cu = opt(v[4]);
  const Place p(a);
  const Scan d(a, cu);
  const auto shape = a.sizes();
  const ScalarType gt = a.scalar_type(), xt = x.scalar_type();
  const kdn_dtype gate = code(a), in = code(x);
  void *pb = p.arg(b, gt, shape), *px = p.arg(&x, xt, shape), *p0 = p.arg(h0, F32, {d.B, d.D});
  void* pc = p.arg(cu, ScalarType::Int, {d.B + 1});
  Tensor y = p.out(v[5], xt, shape), h = p.out(v[6], F32, {d.B, d.D});
  Tensor ws = scan_workspace(p, d.bytes);
  KDN_CALL(kdn_linear_scan_forward, a.data_ptr(), pb, gate, px, in, static_cast<float*>(p0),
                                static_cast<int32_t*>(pc), y.data_ptr(), h.data_ptr<float>(),
                                (int)d.B, (int)d.T, (int)d.D, ws.data_ptr(), (size_t)ws.numel(),
                                p.stream());
  return Py_BuildValue("(NN)", wrap(y), wrap(h));
}

// a, x, y, dy, b, h0, dh_T, cu_seqlens, da, dx, db, dh0
PyObject* scan_backward(PyObject* const* v) {
  const Tensor &a = need(v[0]), *x = opt(v[1]), &y = need(v[2]), &dy = need(v[3]), *b = opt(v[4]);
  const Tensor *h0 = opt(v[5]), *dh = opt(v[6]), *cu = opt(v[7]);
  usual(!b || x);
  const Place p(a);
  const Scan d(a, cu);
  const auto shape = a.sizes();
  const ScalarType gt = a.scalar_type(), yt = y.scalar_type();
  const kdn_dtype gate = code(a), in = code(y);
  void *pb = p.arg(b, gt, shape), *px = p.arg(x, yt, shape), *py = p.arg(&y, yt, shape);
  void *pdy = p.arg(&dy, yt, shape), *p0 = p.arg(h0, F32, {d.B, d.D});
  void *pT = p.arg(dh, F32, {d.B, d.D}), *pc = p.arg(cu, ScalarType::Int, {d.B + 1});
  Tensor da = p.out(v[8], gt, shape), dx = p.out(v[9], yt, shape), db;
  if (b) db = p.out(v[10], gt, shape);
  Tensor dh0 = p.out(v[11], F32, {d.B, d.D}), ws = scan_workspace(p, d.bytes);
  KDN_CALL(kdn_linear_scan_backward, a.data_ptr(), pb, gate, px, py, pdy, in, static_cast<float*>(p0),
            static_cast<float*>(pT), static_cast<int32_t*>(pc), da.data_ptr(),
            b ? db.data_ptr() : nullptr, dx.data_ptr(), dh0.data_ptr<float>(), (int)d.B, (int)d.T,
            (int)d.D, ws.data_ptr(), (size_t)ws.numel(), p.stream());
  PyObject* r = PyDict_New();
  put(r, "a", wrap(da));
  put(r, "x", wrap(dx));
  put(r, "h0", wrap(dh0));
  if (b) put(r, "b", wrap(db));
  return r;
}

ScalarType type_of(long c) {
  usual(c >= 0 && c <= 2);
  return c == KDN_F32 ? F32 : c == KDN_BF16 ? BF16 : E4M3;
}
long whole(PyObject* o) {
  const long c = PyLong_AsLong(o);
  if (c == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Unusual();
  }
  return c;
}
float real(PyObject* o) {
  const double c = PyFloat_AsDouble(o);
  if (c == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Unusual();
  }
  return (float)c;
}

// x, weight, residual, eps, output code, y, scale, h
PyObject* norm_forward(PyObject* const* v) {
  const Tensor &x = need(v[0]), &w = need(v[1]), *res = opt(v[2]);
  const Place p(x);
  const ScalarType out = type_of(whole(v[4]));
  usual(x.dim() >= 1 && x.numel() > 0 && (res || v[7] == Py_None) &&
        (out == E4M3 || v[6] == Py_None));
  const auto shape = x.sizes();
  const int64_t D = shape.back(), rows = x.numel() / D;
  usual(D < 0x7fffffff);
  const kdn_dtype xt = code(x), rt = res ? code(*res) : KDN_F32;
  void *px = p.arg(&x, x.scalar_type(), shape), *pw = p.arg(&w, F32, {D});
  void* pr = res ? p.arg(res, res->scalar_type(), shape) : nullptr;
  Tensor h, y, scale;
  if (res) h = p.out(v[7], res->scalar_type(), shape);
  int64_t ld = 0;
  if (out == E4M3) {
    y = v[5] == Py_None ? p.fp8_empty(rows, D) : need(v[5]);
    p.fp8(y, rows, D, &ld);
    scale = p.out(v[6], F32, {rows, (D + 127) / 128});
  } else {
    y = p.out(v[5], out, shape);
  }
  KDN_CALL(kdn_rmsnorm_forward, px, xt, pr, rt, static_cast<float*>(pw), res ? h.data_ptr() : nullptr,
                            y.data_ptr(), (kdn_dtype)whole(v[4]), ld,
                            out == E4M3 ? scale.data_ptr<float>() : nullptr, rows, (int)D,
                            real(v[3]), p.stream());
  PyObject *ps = Py_None, *ph = Py_None;
  if (out == E4M3) ps = wrap(scale);
  else Py_INCREF(ps);
  if (res) ph = wrap(h);
  else Py_INCREF(ph);
  return Py_BuildValue("(NNN)", wrap(y), ps, ph);
}

// h, weight, dy, dh, eps, dx code or -1, whether the residual's gradient is
// wanted, dx, dresidual, dweight
PyObject* norm_backward(PyObject* const* v) {
  const Tensor &h = need(v[0]), &w = need(v[1]), &dy = need(v[2]), *dh = opt(v[3]);
  const Place p(h);
  usual(h.dim() >= 1 && h.numel() > 0);
  const auto shape = h.sizes();
  const int64_t D = shape.back(), rows = h.numel() / D;
  usual(D < 0x7fffffff);
  const ScalarType ht = h.scalar_type();
  const long c = whole(v[5]);
  const ScalarType xt = c < 0 ? ht : type_of(c);
  usual(xt != E4M3);
  const kdn_dtype hc = code(h), yc = code(dy);
  void *ph = p.arg(&h, ht, shape), *pw = p.arg(&w, F32, {D});
  void *pdy = p.arg(&dy, dy.scalar_type(), shape), *pdh = p.arg(dh, ht, shape);
  const bool want = whole(v[6]) != 0;
  Tensor dx = p.out(v[7], xt, shape), dres, dw = p.out(v[9], F32, {D});
  if (want) dres = p.out(v[8], ht, shape);
  const size_t bytes = kdn_rmsnorm_backward_workspace_size(rows, (int)D);
  Tensor ws = p.empty({(int64_t)bytes}, ScalarType::Byte);
  KDN_CALL(kdn_rmsnorm_backward, ph, hc, static_cast<float*>(pw), pdy, yc, pdh, dx.data_ptr(),
                             xt == F32 ? KDN_F32 : KDN_BF16, want ? dres.data_ptr() : nullptr,
                             dw.data_ptr<float>(), rows, (int)D, real(v[4]), ws.data_ptr(), bytes,
                             p.stream());
  PyObject *r = PyDict_New(), *pr = Py_None;
  if (want) pr = wrap(dres);
  else Py_INCREF(pr);
  put(r, "x", wrap(dx));
  put(r, "weight", wrap(dw));
  put(r, "residual", pr);
  return r;
}

// x, tile, transpose, q, scale
PyObject* quantize(PyObject* const* v) {
  const Tensor& x = need(v[0]);
  const Place p(x);
  usual(x.dim() == 2 && x.numel() > 0);
  const int64_t rows = x.size(0), cols = x.size(1);
  const int tile = PyObject_IsTrue(v[1]), tr = PyObject_IsTrue(v[2]);
  usual(tile >= 0 && tr >= 0);
  const int64_t R = tr ? cols : rows, C = tr ? rows : cols;
  const kdn_dtype xt = code(x);
  void* px = p.arg(&x, x.scalar_type(), x.sizes());
  Tensor q = v[3] == Py_None ? p.fp8_empty(R, C) : need(v[3]);
  int64_t ld = 0;
  void* pq = p.fp8(q, R, C, &ld);
  Tensor s = p.out(v[4], F32, {tile ? (R + 127) / 128 : R, (C + 127) / 128});
  KDN_CALL(kdn_fp8_quantize, px, xt, rows, cols, tile, tr, pq, ld, s.data_ptr<float>(), p.stream());
  return Py_BuildValue("(NN)", wrap(q), wrap(s));
}

// x, x_scale, w, w_scale, output code, out, status
PyObject* matmul(PyObject* const* v) {
  const Tensor &x = need(v[0]), &xs = need(v[1]), &w = need(v[2]), &ws = need(v[3]);
  const Place p(x);
  usual(x.dim() == 2 && w.dim() == 2 && ws.dim() == 2 && x.size(0) > 0);
  const int64_t M = x.size(0), K = x.size(1), N = w.size(0), kb = (K + 127) / 128;
  usual(M < 0x7fffffff && N < 0x7fffffff && K < 0x7fffffff);
  int64_t ldx = 0, ldw = 0;
  void *px = p.fp8(x, M, K, &ldx), *pw = p.fp8(w, N, K, &ldw);
  const bool tile = ws.size(0) != N;  // (the two forms agree for N = 1)
  void *psx = p.arg(&xs, F32, {M, kb}), *psw = p.arg(&ws, F32, {tile ? (N + 127) / 128 : N, kb});
  const ScalarType ot = type_of(whole(v[4]));
  usual(ot != E4M3);
  Tensor out = p.out(v[5], ot, {M, N});
  void* st = p.arg(opt(v[6]), ScalarType::Int, {1});
  KDN_CALL(kdn_fp8_matmul, px, ldx, static_cast<float*>(psx), pw, ldw, static_cast<float*>(psw), tile,
                       out.data_ptr(), ot == F32 ? KDN_F32 : KDN_BF16, (int)M, (int)N, (int)K,
                       static_cast<uint32_t*>(st), p.stream());
  return wrap(out);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n == N) {
    try {
      return F(args);
    } catch (const Failed& e) {
      raise(e);
      return nullptr;
    } catch (...) {
    }
    PyErr_Clear();
  }
  Py_RETURN_NONE;
}
#define KDN_ENTRY(name, count) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<name, count>)), \
   METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KDN_ENTRY(scan_step, 5),      KDN_ENTRY(scan_forward, 7),
                         KDN_ENTRY(scan_backward, 12), KDN_ENTRY(norm_forward, 8),
                         KDN_ENTRY(norm_backward, 10), KDN_ENTRY(quantize, 5),
                         KDN_ENTRY(matmul, 7),         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kdn_quick", nullptr, -1, methods,
                      nullptr,               nullptr,      nullptr, nullptr};

}  // namespace

// (kdn.py leaves a module that was built against another torch unused)
PyMODINIT_FUNC PyInit__kdn_quick() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
