// Python entry points of the norm and MXFP4 operators for torch tensors: checks of types, shapes, layout
// and device, then one call of the C ABI on the current stream. Argument marshalling only, like the
// package's ctypes wrappers, which spend more time on a decoded token's call than its kernels run.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "../../include/qe.h"

namespace {

PyObject* g_raise = nullptr;  // raise(status, what, detail): raises the package's QEError

struct Refused {
  int status;
  std::string what, detail;
};

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

// A call's tensors: the first one sets the device, the others have to be on it.
struct Call {
  const char* what;
  int device = -1;

  [[noreturn]] void refuse(const char* name, const std::string& detail) const {
    throw Refused{QE_ERR_INVALID_ARG, name, std::string(what) + ": " + detail};
  }
  const at::Tensor& tensor(PyObject* o, const char* name) const {
    if (!THPVariable_Check(o)) refuse(name, "expected a tensor");
    return THPVariable_Unpack(o);
  }
  const at::Tensor& matrix(PyObject* o, const char* name) const {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 2) refuse(name, "expected [rows, channels], got " + shape_text(t.sizes()));
    return t;
  }
  qe_dtype dtype(const at::Tensor& t, const char* name) const {
    if (t.scalar_type() == at::kBFloat16) return QE_BF16;
    if (t.scalar_type() == at::kFloat) return QE_F32;
    refuse(name, std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
  }
  void expect(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    if (t.scalar_type() != type || t.sizes() != shape)
      refuse(name, std::string("expected ") + c10::toString(type) + " " + shape_text(shape) + ", got " +
                       c10::toString(t.scalar_type()) + " " + shape_text(t.sizes()));
  }
  void expect_bytes(const at::Tensor& t, const char* name, size_t n) const {
    if (t.scalar_type() != at::kByte || static_cast<size_t>(t.numel()) < n)
      refuse(name, "expected uint8 of at least " + std::to_string(n) + " elements, got " +
                       c10::toString(t.scalar_type()) + " " + shape_text(t.sizes()));
  }
  void* pointer(const at::Tensor& t, const char* name) {
    if (!t.is_cuda() || !t.is_contiguous()) refuse(name, "tensors passed to the QE library must be contiguous CUDA tensors");
    const int d = t.get_device();
    if (device < 0) device = d;
    else if (d != device) refuse(name, "tensors on devices " + std::to_string(device) + " and " + std::to_string(d));
    return t.data_ptr();
  }
  // An optional tensor of the given type and shape.
  void* maybe(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    expect(t, name, type, shape);
    return pointer(t, name);
  }
};

// Runs f(stream) on the call's device, with its current stream unless one is given (a raw handle).
template <class F>
PyObject* launch(const Call& c, PyObject* stream, F f) {
  void* given = stream == Py_None ? nullptr : PyLong_AsVoidPtr(stream);
  if (PyErr_Occurred()) return nullptr;
  qe_status rc;
  auto run = [&] { return f(stream == Py_None ? static_cast<void*>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream()) : given); };
  if (c.device == c10::cuda::current_device()) {
    rc = run();
  } else {
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device));
    rc = run();
  }
  if (rc != QE_OK) throw Refused{rc, c.what, rc == QE_ERR_CUDA ? qe_last_cuda_error() : ""};
  Py_RETURN_NONE;
}

// No C++ exception reaches Python's C code.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused& e) {
    PyObject* r = g_raise ? PyObject_CallFunction(g_raise, "iss", e.status, e.what.c_str(), e.detail.c_str()) : nullptr;
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.detail.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

int32_t i32(const Call& c, const char* name, int64_t v) {
  if (v > INT32_MAX) c.refuse(name, "more than 2^31 - 1 rows or channels");
  return static_cast<int32_t>(v);
}

// X, gamma, eps, a_bits, codes, scales, residual, residual_out, Y, s_inv, stream
PyObject* add_rmsnorm_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    Call c{"qe_add_rmsnorm_quant"};
    const double eps = PyFloat_AsDouble(a[2]);
    const long bits = PyLong_AsLong(a[3]);
    if (PyErr_Occurred()) return nullptr;
    const at::Tensor& X = c.matrix(a[0], "X");
    const at::Tensor& gamma = c.tensor(a[1], "gamma");
    const qe_dtype xd = c.dtype(X, "X"), gd = c.dtype(gamma, "gamma");
    const int64_t T = X.size(0), d = X.size(1);
    void* x = c.pointer(X, "X");
    c.expect(gamma, "gamma", gamma.scalar_type(), {d});
    void* g = c.pointer(gamma, "gamma");
    void* r = c.maybe(a[6], "residual", X.scalar_type(), {T, d});
    void* h = c.maybe(a[7], "residual_out", X.scalar_type(), {T, d});
    void* y = c.maybe(a[8], "Y", X.scalar_type(), {T, d});
    void* s = c.maybe(a[9], "s_inv", at::kFloat, {d});
    void *codes = nullptr, *scales = nullptr;
    if (bits == 4) {
      codes = c.maybe(a[4], "codes", at::kByte, {T, d / 2});
      if (a[5] != Py_None) {
        const at::Tensor& sc = c.tensor(a[5], "scales");
        c.expect_bytes(sc, "scales", qe_mx4_scale_bytes(i32(c, "X", T), i32(c, "X", d)));
        scales = c.pointer(sc, "scales");
      }
    } else if (bits == 6 || bits == 8) {
      codes = c.maybe(a[4], "codes", at::kChar, {T, d});
      scales = c.maybe(a[5], "scales", at::kFloat, {T});
    }
    return launch(c, a[10], [&](void* st) {
      return qe_add_rmsnorm_quant(x, xd, r, g, gd, eps, i32(c, "X", T), i32(c, "X", d), static_cast<const float*>(s),
                                  static_cast<int32_t>(bits), h, y, codes, scales, st);
    });
  });
}

// codes, sa, out, stream
PyObject* act_dequant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 4)) return nullptr;
  return guarded([&] {
    Call c{"qe_act_dequant"};
    const at::Tensor& codes = c.matrix(a[0], "codes");
    const at::Tensor& sa = c.tensor(a[1], "sa");
    const at::Tensor& out = c.matrix(a[2], "out");
    const int64_t T = codes.size(0), d = codes.size(1);
    c.expect(codes, "codes", at::kChar, {T, d});
    c.expect(sa, "sa", at::kFloat, {T});
    const qe_dtype od = c.dtype(out, "out");
    c.expect(out, "out", out.scalar_type(), {T, d});
    void *q = c.pointer(codes, "codes"), *s = c.pointer(sa, "sa"), *o = c.pointer(out, "out");
    return launch(c, a[3], [&](void* st) {
      return qe_act_dequant(static_cast<const int8_t*>(q), static_cast<const float*>(s), i32(c, "codes", T), i32(c, "codes", d), o,
                            od, st);
    });
  });
}

// X, codes, scales, s, s_inv, stream
PyObject* mx4_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 6)) return nullptr;
  return guarded([&] {
    Call c{"qe_mx4_quantize"};
    const at::Tensor& X = c.matrix(a[0], "X");
    const at::Tensor& codes = c.tensor(a[1], "codes");
    const at::Tensor& scales = c.tensor(a[2], "scales");
    const qe_dtype xd = c.dtype(X, "X");
    const int32_t rows = i32(c, "X", X.size(0)), cols = i32(c, "X", X.size(1));
    c.expect(codes, "codes", at::kByte, {rows, cols / 2});
    c.expect_bytes(scales, "scales", qe_mx4_scale_bytes(rows, cols));
    void *x = c.pointer(X, "X"), *q = c.pointer(codes, "codes"), *sc = c.pointer(scales, "scales");
    void* s = c.maybe(a[3], "s", at::kFloat, {cols});
    void* si = c.maybe(a[4], "s_inv", at::kFloat, {cols});
    return launch(c, a[5], [&](void* st) {
      return qe_mx4_quantize(x, xd, static_cast<const float*>(s), rows, cols, q, sc, static_cast<float*>(si), st);
    });
  });
}

// codes, scales, out, stream
PyObject* mx4_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 4)) return nullptr;
  return guarded([&] {
    Call c{"qe_mx4_dequantize"};
    const at::Tensor& codes = c.tensor(a[0], "codes");
    const at::Tensor& scales = c.tensor(a[1], "scales");
    const at::Tensor& out = c.matrix(a[2], "out");
    const qe_dtype od = c.dtype(out, "out");
    const int32_t rows = i32(c, "out", out.size(0)), cols = i32(c, "out", out.size(1));
    c.expect(codes, "codes", at::kByte, {rows, cols / 2});
    c.expect_bytes(scales, "scales", qe_mx4_scale_bytes(rows, cols));
    void *q = c.pointer(codes, "codes"), *sc = c.pointer(scales, "scales"), *o = c.pointer(out, "out");
    return launch(c, a[3], [&](void* st) { return qe_mx4_dequantize(q, sc, rows, cols, o, od, st); });
  });
}

// x_codes, x_scales, w_codes, w_scales, Y, stream
PyObject* mx4_product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 6)) return nullptr;
  return guarded([&] {
    Call c{"qe_mx4_product"};
    const at::Tensor& xc = c.tensor(a[0], "x_codes");
    const at::Tensor& xs = c.tensor(a[1], "x_scales");
    const at::Tensor& wc = c.matrix(a[2], "w_codes");
    const at::Tensor& ws = c.tensor(a[3], "w_scales");
    const at::Tensor& Y = c.matrix(a[4], "Y");
    const qe_dtype yd = c.dtype(Y, "Y");
    const int32_t T = i32(c, "Y", Y.size(0)), N = i32(c, "Y", Y.size(1)), K = i32(c, "w_codes", 2 * wc.size(1));
    c.expect(xc, "x_codes", at::kByte, {T, K / 2});
    c.expect(wc, "w_codes", at::kByte, {N, K / 2});
    c.expect_bytes(xs, "x_scales", qe_mx4_scale_bytes(T, K));
    c.expect_bytes(ws, "w_scales", qe_mx4_scale_bytes(N, K));
    void *p = c.pointer(xc, "x_codes"), *ps = c.pointer(xs, "x_scales"), *q = c.pointer(wc, "w_codes"),
         *qs = c.pointer(ws, "w_scales"), *y = c.pointer(Y, "Y");
    return launch(c, a[5], [&](void* st) { return qe_mx4_product(p, ps, q, qs, T, K, N, y, yd, st); });
  });
}

// w_codes, w_scales, X, Y, workspace, s_inv, stream
PyObject* mx4_linear_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 7)) return nullptr;
  return guarded([&] {
    Call c{"qe_mx4_linear_forward"};
    const at::Tensor& wc = c.tensor(a[0], "w_codes");
    const at::Tensor& ws = c.tensor(a[1], "w_scales");
    const at::Tensor& X = c.matrix(a[2], "X");
    const at::Tensor& Y = c.matrix(a[3], "Y");
    const at::Tensor& work = c.tensor(a[4], "workspace");
    const qe_dtype xd = c.dtype(X, "X"), yd = c.dtype(Y, "Y");
    const int32_t T = i32(c, "X", X.size(0)), K = i32(c, "X", X.size(1)), N = i32(c, "Y", Y.size(1));
    c.expect(Y, "Y", Y.scalar_type(), {T, N});
    c.expect(wc, "w_codes", at::kByte, {N, K / 2});
    c.expect_bytes(ws, "w_scales", qe_mx4_scale_bytes(N, K));
    void *x = c.pointer(X, "X"), *y = c.pointer(Y, "Y"), *q = c.pointer(wc, "w_codes"), *qs = c.pointer(ws, "w_scales"),
         *w = c.pointer(work, "workspace");
    void* s = c.maybe(a[5], "s_inv", at::kFloat, {K});
    return launch(c, a[6], [&](void* st) {
      return qe_mx4_linear_forward(q, qs, static_cast<const float*>(s), x, xd, T, K, N, y, yd, w, work.nbytes(), st);
    });
  });
}

PyObject* set_raise(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_raise, f);
  Py_RETURN_NONE;
}

#define QE_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {QE_FAST(add_rmsnorm_quant),  QE_FAST(act_dequant), QE_FAST(mx4_quantize),
                           QE_FAST(mx4_dequantize),     QE_FAST(mx4_product), QE_FAST(mx4_linear_forward),
                           {"set_raise", set_raise, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_qe_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qe_torch() { return PyModule_Create(&g_module); }
