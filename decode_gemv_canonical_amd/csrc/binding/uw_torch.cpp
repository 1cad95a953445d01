// Python's side of the 8-bit activation path's entry points: the tensors'
// checks and the call into libuw.so in one step of C++.  A decode step makes
// these calls on kernels of a few microseconds, so the caller's time per call
// counts: the same checks written in Python and a ctypes call took 2.9 us on
// top of the launch's 4.
//
// Nothing is computed here.  Each function checks what the C side cannot know
// (types, shapes, strides, devices), raises TypeError or ValueError naming
// the operand, and returns the entry point's status.  The entry points'
// addresses are handed over once, by bind().
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <stdexcept>
#include <string>

#include "../../../include/uw.h"

namespace {

decltype(&uw_rmsnorm) f_rmsnorm = nullptr;
decltype(&uw_silu_mul) f_silu_mul = nullptr;
decltype(&uw_i8_quantize) f_quantize = nullptr;
decltype(&uw_i8_dequantize) f_dequantize = nullptr;
decltype(&uw_i8_gemm) f_gemm = nullptr;
decltype(&uw_i8_gemm_shaped) f_gemm_shaped = nullptr;

struct ValueProblem : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct TypeProblem : std::runtime_error {
  using std::runtime_error::runtime_error;
};

[[noreturn]] void value_error(const std::string& what) { throw ValueProblem(what); }

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw TypeProblem(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int float_code(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kFloat) return UW_F32;
  if (t.scalar_type() == at::kBFloat16) return UW_BF16;
  throw TypeProblem(std::string(name) + ": unsupported dtype " + c10::toString(t.scalar_type()) +
                    "; use float32 or bfloat16");
}

void want_i8(const at::Tensor& t, const char* name) {
  if (t.scalar_type() != at::kChar)
    throw TypeProblem(std::string(name) + " must be int8, got " + c10::toString(t.scalar_type()));
}

// The device of a call: the first operand's, which has to be the current one.
int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
  const int dev = t.get_device(), now = c10::hip::current_device();
  if (dev != now)
    value_error(std::string(name) + " is on cuda:" + std::to_string(dev) + ", the current device is cuda:" +
                std::to_string(now));
  return dev;
}

void want_device(const at::Tensor& t, int dev, const char* name) {
  if (!t.is_cuda() || t.get_device() != dev) value_error(std::string(name) + " must be on cuda:" + std::to_string(dev));
}

// A row-major [n, cols] operand on the device: its row stride.
int64_t want_rows(const at::Tensor& t, int64_t n, int64_t cols, int dev, const char* name) {
  if (t.dim() != 2 || t.size(0) != n || t.size(1) != cols)
    value_error(std::string(name) + " must have shape (" + std::to_string(n) + ", " + std::to_string(cols) + "), got " +
                shape_of(t));
  const int64_t ld = t.stride(0);
  if ((t.stride(1) != 1 && cols > 1) || (ld < cols && n > 1))
    value_error(std::string(name) + " must have a unit inner stride and rows that do not overlap");
  want_device(t, dev, name);
  return ld;
}

void want_2d(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) value_error(std::string(name) + " must be 2-D, got shape " + shape_of(t));
}

float* want_scale(const at::Tensor& t, int64_t n, int dev, const char* name) {
  if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    value_error(std::string(name) + " must be a contiguous float32 vector of " + std::to_string(n) + " values");
  want_device(t, dev, name);
  return static_cast<float*>(t.data_ptr());
}

// The type code of a row operator's output, and its scales.
int out_code(const at::Tensor& y, PyObject* scale, int64_t n, int dev, float** sp) {
  *sp = nullptr;
  if (y.scalar_type() != at::kChar) {
    if (scale != Py_None) value_error("scale goes with an int8 output");
    return float_code(y, "Y");
  }
  if (scale == Py_None) value_error("an int8 output needs a scale vector");
  *sp = want_scale(tensor(scale, "scale"), n, dev, "scale");
  return UW_I8;
}

// None: the current stream; an int: a raw stream; else an object with cuda_stream.
void* stream_of(PyObject* o, int dev) {
  if (o == Py_None) return c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(dev)).stream();
  if (!PyLong_Check(o)) {
    PyObject* on = PyObject_GetAttrString(o, "device_index");
    const long at = on ? PyLong_AsLong(on) : dev;
    Py_XDECREF(on);
    PyErr_Clear();
    if (at != dev) value_error("the stream is on cuda:" + std::to_string(at) + ", the operands on cuda:" + std::to_string(dev));
  }
  PyObject* raw = PyLong_Check(o) ? (Py_INCREF(o), o) : PyObject_GetAttrString(o, "cuda_stream");
  if (!raw) {
    PyErr_Clear();
    throw TypeProblem("stream must be a torch.cuda.Stream, a raw stream or None");
  }
  void* s = PyLong_AsVoidPtr(raw);
  Py_DECREF(raw);
  if (!s && PyErr_Occurred()) {
    PyErr_Clear();
    throw TypeProblem("stream must be a torch.cuda.Stream, a raw stream or None");
  }
  return s;
}

template <class F>
PyObject* guarded(const char* name, bool bound, Py_ssize_t got, Py_ssize_t want, F f) {
  try {
    if (!bound) throw std::runtime_error("not bound to libuw.so");
    if (got != want) throw TypeProblem("takes " + std::to_string(want) + " arguments");
    return PyLong_FromLong(f());
  } catch (const ValueProblem& e) {
    PyErr_Format(PyExc_ValueError, "%s: %s", name, e.what());
  } catch (const TypeProblem& e) {
    PyErr_Format(PyExc_TypeError, "%s: %s", name, e.what());
  } catch (const std::exception& e) {
    PyErr_Format(PyExc_RuntimeError, "%s: %s", name, e.what());
  } catch (...) {
    PyErr_Format(PyExc_RuntimeError, "%s: unknown C++ exception", name);
  }
  return nullptr;
}

// rmsnorm(X, gain, Y, scale, residual, residual_out, eps, stream)
PyObject* py_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded("uw_rmsnorm", f_rmsnorm, n_args, 8, [&] {
    const at::Tensor& X = tensor(a[0], "X");
    const int dev = device_of(X, "X");
    want_2d(X, "X");
    const int64_t n = X.size(0), cols = X.size(1), ldx = want_rows(X, n, cols, dev, "X");
    const at::Tensor& Y = tensor(a[2], "Y");
    const int64_t ldy = want_rows(Y, n, cols, dev, "Y");
    float* sp;
    const int yt = out_code(Y, a[3], n, dev, &sp);
    const void *rp = nullptr, *gp = nullptr;
    void* hp = nullptr;
    int64_t ldr = 0, ldh = 0;
    int rt = UW_F32, gt = UW_F32;
    if (a[4] != Py_None) {
      const at::Tensor& R = tensor(a[4], "residual");
      ldr = want_rows(R, n, cols, dev, "residual");
      rt = float_code(R, "residual");
      rp = R.data_ptr();
    }
    if (a[5] != Py_None) {
      const at::Tensor& H = tensor(a[5], "residual_out");
      if (a[4] == Py_None) value_error("residual_out needs a residual");
      ldh = want_rows(H, n, cols, dev, "residual_out");
      if (float_code(H, "residual_out") != rt) value_error("residual_out must have the residual's dtype");
      hp = H.data_ptr();
    }
    if (a[1] != Py_None) {
      const at::Tensor& g = tensor(a[1], "gain");
      if (g.dim() != 1 || g.size(0) != cols || (cols > 1 && g.stride(0) != 1))
        value_error("gain must be a contiguous vector of " + std::to_string(cols) + " elements, got shape " + shape_of(g));
      want_device(g, dev, "gain");
      gt = float_code(g, "gain");
      gp = g.data_ptr();
    }
    const double eps = PyFloat_AsDouble(a[6]);
    if (eps == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      throw TypeProblem("eps must be a number");
    }
    return f_rmsnorm(X.data_ptr(), n, cols, ldx, float_code(X, "X"), rp, ldr, rt, hp, ldh, gp, gt,
                     static_cast<float>(eps), Y.data_ptr(), ldy, yt, sp, stream_of(a[7], dev));
  });
}

// silu_mul(G, U, Y, scale, stream)
PyObject* py_silu_mul(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded("uw_silu_mul", f_silu_mul, n_args, 5, [&] {
    const at::Tensor &G = tensor(a[0], "G"), &U = tensor(a[1], "U"), &Y = tensor(a[2], "Y");
    const int dev = device_of(G, "G");
    want_2d(G, "G");
    const int64_t n = G.size(0), cols = G.size(1), ldg = want_rows(G, n, cols, dev, "G");
    const int64_t ldu = want_rows(U, n, cols, dev, "U"), ldy = want_rows(Y, n, cols, dev, "Y");
    if (U.scalar_type() != G.scalar_type()) throw TypeProblem("G and U must have the same dtype");
    float* sp;
    const int yt = out_code(Y, a[3], n, dev, &sp);
    return f_silu_mul(G.data_ptr(), ldg, U.data_ptr(), ldu, float_code(G, "G"), n, cols, Y.data_ptr(), ldy, yt, sp,
                      stream_of(a[4], dev));
  });
}

// quantize(X, Q, scale, stream)
PyObject* py_quantize(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded("uw_i8_quantize", f_quantize, n_args, 4, [&] {
    const at::Tensor &X = tensor(a[0], "X"), &Q = tensor(a[1], "Q");
    const int dev = device_of(X, "X");
    want_2d(X, "X");
    const int64_t n = X.size(0), cols = X.size(1), ldx = want_rows(X, n, cols, dev, "X");
    want_i8(Q, "Q");
    const int64_t ldq = want_rows(Q, n, cols, dev, "Q");
    float* sp = want_scale(tensor(a[2], "scale"), n, dev, "scale");
    return f_quantize(X.data_ptr(), n, cols, ldx, float_code(X, "X"), static_cast<int8_t*>(Q.data_ptr()), ldq, sp,
                      stream_of(a[3], dev));
  });
}

// dequantize(Q, scale, Y, stream)
PyObject* py_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded("uw_i8_dequantize", f_dequantize, n_args, 4, [&] {
    const at::Tensor &Q = tensor(a[0], "Q"), &Y = tensor(a[2], "Y");
    const int dev = device_of(Q, "Q");
    want_i8(Q, "Q");
    want_2d(Q, "Q");
    const int64_t n = Q.size(0), cols = Q.size(1), ldq = want_rows(Q, n, cols, dev, "Q");
    const int64_t ldy = want_rows(Y, n, cols, dev, "Y");
    const float* sp = want_scale(tensor(a[1], "scale"), n, dev, "scale");
    return f_dequantize(static_cast<const int8_t*>(Q.data_ptr()), n, cols, ldq, sp, Y.data_ptr(), ldy,
                        float_code(Y, "Y"), stream_of(a[3], dev));
  });
}

// gemm(W, w_scale, X, x_scale, Y, bias, stream) and, with a shape and ks
// before the stream, gemm_shaped.
PyObject* call_gemm(PyObject* const* a, Py_ssize_t n_args, bool shaped) {
  return guarded(shaped ? "uw_i8_gemm_shaped" : "uw_i8_gemm", f_gemm && f_gemm_shaped, n_args, shaped ? 9 : 7, [&] {
    const at::Tensor &W = tensor(a[0], "W"), &X = tensor(a[2], "X"), &Y = tensor(a[4], "Y");
    const int dev = device_of(W, "W");
    want_i8(W, "W");
    want_i8(X, "X");
    want_2d(W, "W");
    want_2d(X, "X");
    const int64_t rows = W.size(0), cols = W.size(1), n = X.size(0);
    const int64_t ldw = want_rows(W, rows, cols, dev, "W"), ldx = want_rows(X, n, cols, dev, "X");
    const int64_t ldy = want_rows(Y, n, rows, dev, "Y");
    const float* ws = want_scale(tensor(a[1], "w_scale"), rows, dev, "w_scale");
    const float* xs = want_scale(tensor(a[3], "x_scale"), n, dev, "x_scale");
    const float* bias = a[5] == Py_None ? nullptr : want_scale(tensor(a[5], "bias"), rows, dev, "bias");
    const auto* w = static_cast<const int8_t*>(W.data_ptr());
    const auto* x = static_cast<const int8_t*>(X.data_ptr());
    const int yt = float_code(Y, "Y");
    if (!shaped)
      return f_gemm(w, rows, cols, ldw, ws, x, n, ldx, xs, bias, Y.data_ptr(), ldy, yt, stream_of(a[6], dev));
    const long shape = PyLong_AsLong(a[6]), ks = PyLong_AsLong(a[7]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw TypeProblem("shape and ks must be integers");
    }
    return f_gemm_shaped(w, rows, cols, ldw, ws, x, n, ldx, xs, bias, Y.data_ptr(), ldy, yt,
                         static_cast<int>(std::min(std::max(shape, -1L), 1000000L)),
                         static_cast<int>(std::min(std::max(ks, -1L), 1000000L)), stream_of(a[8], dev));
  });
}

PyObject* py_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) { return call_gemm(a, n, false); }
PyObject* py_gemm_shaped(PyObject*, PyObject* const* a, Py_ssize_t n) { return call_gemm(a, n, true); }

// bind(rmsnorm, silu_mul, quantize, dequantize, gemm, gemm_shaped): addresses
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  void* p[6];
  if (n_args != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes 6 addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null address");
      return nullptr;
    }
  }
  f_rmsnorm = reinterpret_cast<decltype(f_rmsnorm)>(p[0]);
  f_silu_mul = reinterpret_cast<decltype(f_silu_mul)>(p[1]);
  f_quantize = reinterpret_cast<decltype(f_quantize)>(p[2]);
  f_dequantize = reinterpret_cast<decltype(f_dequantize)>(p[3]);
  f_gemm = reinterpret_cast<decltype(f_gemm)>(p[4]);
  f_gemm_shaped = reinterpret_cast<decltype(f_gemm_shaped)>(p[5]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<py_bind>("bind"),           method<py_rmsnorm>("rmsnorm"),       method<py_silu_mul>("silu_mul"),
    method<py_quantize>("quantize"),   method<py_dequantize>("dequantize"), method<py_gemm>("gemm"),
    method<py_gemm_shaped>("gemm_shaped"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_uw_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__uw_torch() { return PyModule_Create(&module_def); }
