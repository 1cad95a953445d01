// Python's side of the entry points of the 8-bit activation path, the block
// norm and the 4-bit weights: the tensors'
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
decltype(&uw_block_norm) f_block_norm = nullptr;
decltype(&uw_i4_quantize) f_quantize4 = nullptr;
decltype(&uw_i4_dequantize) f_dequantize4 = nullptr;
decltype(&uw_i4_gemm) f_gemm4 = nullptr;
decltype(&uw_i4_gemm_shaped) f_gemm4_shaped = nullptr;

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

// A vector of cols gains, or None (null): its address, and its type code.
const void* want_gain(PyObject* o, int64_t cols, int dev, const char* name, int* code) {
  if (o == Py_None) return nullptr;
  const at::Tensor& g = tensor(o, name);
  if (g.dim() != 1 || g.size(0) != cols || (cols > 1 && g.stride(0) != 1))
    value_error(std::string(name) + " must be a contiguous vector of " + std::to_string(cols) + " elements, got shape " +
                shape_of(g));
  want_device(g, dev, name);
  *code = float_code(g, name);
  return g.data_ptr();
}

float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw TypeProblem(std::string(name) + " must be a number");
  }
  return static_cast<float>(v);
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
    gp = want_gain(a[1], cols, dev, "gain", &gt);
    const float eps = number(a[6], "eps");
    return f_rmsnorm(X.data_ptr(), n, cols, ldx, float_code(X, "X"), rp, ldr, rt, hp, ldh, gp, gt,
                     eps, Y.data_ptr(), ldy, yt, sp, stream_of(a[7], dev));
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

// block_norm(X, residual, post_norm, post_gain, post_eps, gate, block_scale, residual_scale, residual_out, gain, eps,
//            Y, scale, stream)
PyObject* py_block_norm(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded("uw_block_norm", f_block_norm, n_args, 14, [&] {
    const at::Tensor &X = tensor(a[0], "X"), &R = tensor(a[1], "residual");
    const int dev = device_of(X, "X");
    want_2d(X, "X");
    const int64_t n = X.size(0), cols = X.size(1), ldx = want_rows(X, n, cols, dev, "X");
    const int64_t ldr = want_rows(R, n, cols, dev, "residual");
    const int rt = float_code(R, "residual");
    const int post_norm = PyObject_IsTrue(a[2]);
    if (post_norm < 0) {
      PyErr_Clear();
      throw TypeProblem("post_norm must be a truth value");
    }
    int pt = UW_F32, gt = UW_F32, nt = UW_F32, yt = UW_F32;
    const void* post = want_gain(a[3], cols, dev, "post_gain", &pt);
    const void *gate = nullptr, *gain = want_gain(a[9], cols, dev, "gain", &nt);
    int64_t ldg = 0, ldh = 0, ldy = 0;
    if (a[5] != Py_None) {
      const at::Tensor& g = tensor(a[5], "gate");
      if (g.dim() == 1) {
        gate = want_gain(a[5], cols, dev, "gate", &gt);
      } else if (g.dim() == 2 && g.size(0) == n && g.size(1) == cols && n > 1 && g.stride(0) == 0) {
        // one row, expanded
        if (cols > 1 && g.stride(1) != 1) value_error("gate must have a unit inner stride");
        want_device(g, dev, "gate");
        gt = float_code(g, "gate");
        gate = g.data_ptr();
      } else {
        ldg = want_rows(g, n, cols, dev, "gate");
        gt = float_code(g, "gate");
        gate = g.data_ptr();
      }
    }
    void *hp = nullptr, *yp = nullptr;
    if (a[8] != Py_None) {
      const at::Tensor& H = tensor(a[8], "residual_out");
      ldh = want_rows(H, n, cols, dev, "residual_out");
      if (float_code(H, "residual_out") != rt) value_error("residual_out must have the residual's dtype");
      hp = H.data_ptr();
    }
    float* sp = nullptr;
    if (a[11] != Py_None) {
      const at::Tensor& Y = tensor(a[11], "Y");
      ldy = want_rows(Y, n, cols, dev, "Y");
      yt = out_code(Y, a[12], n, dev, &sp);
      yp = Y.data_ptr();
    } else if (a[12] != Py_None || a[9] != Py_None) {
      value_error("gain and scale go with Y");
    }
    if (a[8] == Py_None && a[11] == Py_None) value_error("nothing to write: residual_out and Y are both None");
    return f_block_norm(X.data_ptr(), n, cols, ldx, float_code(X, "X"), post_norm, post, pt,
                        post_norm ? number(a[4], "post_eps") : 1.f, gate, ldg, gt, number(a[6], "block_scale"), R.data_ptr(),
                        ldr, rt, number(a[7], "residual_scale"), hp, ldh, gain, nt, yp ? number(a[10], "eps") : 1.f, yp, ldy, yt,
                        sp, stream_of(a[13], dev));
  });
}

// Packed 4-bit rows of `cols` integers: their stride in bytes.
int64_t want_packed(const at::Tensor& t, int64_t rows, int64_t cols, int dev, const char* name) {
  if (t.scalar_type() != at::kByte)
    throw TypeProblem(std::string(name) + " must be uint8, got " + c10::toString(t.scalar_type()));
  const int64_t ld = want_rows(t, rows, (cols + 1) / 2, dev, name), words = (cols + 31) / 32 * 16;
  if (reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 || (rows > 1 && (ld % 16 || ld < words)))
    value_error(std::string(name) + " must have rows that start at multiples of 16 bytes and hold whole 16-byte words");
  // the words of the last row have to be there
  const int64_t end = (t.storage_offset() + (rows > 0 ? (rows - 1) * ld : 0)) + words;
  if (rows > 0 && end > static_cast<int64_t>(t.storage().nbytes()))
    value_error(std::string(name) + ": its last row's 16-byte words pass the end of its memory");
  return ld;
}

struct Groups {
  void *scale = nullptr, *offset = nullptr;
  int64_t lds = 0, ldo = 0;
  int st = UW_F32, group = 0;
};

// Scales, offsets (or None) and the group's size.
Groups want_groups(PyObject* scale, PyObject* offset, PyObject* group, int64_t rows, int64_t cols, int dev) {
  Groups g;
  const long size = PyLong_AsLong(group);
  if (size == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw TypeProblem("group must be an integer");
  }
  if (size != 32 && size != 64 && size != 128) value_error("group must be 32, 64 or 128, got " + std::to_string(size));
  g.group = static_cast<int>(size);
  const int64_t n = (cols + size - 1) / size;
  const at::Tensor& s = tensor(scale, "scale");
  g.lds = want_rows(s, n, rows, dev, "scale");
  g.st = float_code(s, "scale");
  g.scale = s.data_ptr();
  if (offset != Py_None) {
    const at::Tensor& m = tensor(offset, "offset");
    g.ldo = want_rows(m, n, rows, dev, "offset");
    if (float_code(m, "offset") != g.st) value_error("offset must have the scale's dtype");
    g.offset = m.data_ptr();
  }
  return g;
}

// quantize4(X, Q, scale, offset, group, stream)
PyObject* py_quantize4(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded("uw_i4_quantize", f_quantize4, n_args, 6, [&] {
    const at::Tensor &X = tensor(a[0], "X"), &Q = tensor(a[1], "Q");
    const int dev = device_of(X, "X");
    want_2d(X, "X");
    const int64_t n = X.size(0), cols = X.size(1), ldx = want_rows(X, n, cols, dev, "X");
    const int64_t ldq = want_packed(Q, n, cols, dev, "Q");
    const Groups g = want_groups(a[2], a[3], a[4], n, cols, dev);
    return f_quantize4(X.data_ptr(), n, cols, ldx, float_code(X, "X"), g.group, static_cast<uint8_t*>(Q.data_ptr()), ldq,
                       g.scale, g.lds, g.offset, g.ldo, g.st, stream_of(a[5], dev));
  });
}

// dequantize4(Q, scale, Y, offset, group, stream)
PyObject* py_dequantize4(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded("uw_i4_dequantize", f_dequantize4, n_args, 6, [&] {
    const at::Tensor &Q = tensor(a[0], "Q"), &Y = tensor(a[2], "Y");
    const int dev = device_of(Q, "Q");
    want_2d(Y, "Y");
    const int64_t n = Y.size(0), cols = Y.size(1), ldy = want_rows(Y, n, cols, dev, "Y");
    const int64_t ldq = want_packed(Q, n, cols, dev, "Q");
    const Groups g = want_groups(a[1], a[3], a[4], n, cols, dev);
    return f_dequantize4(static_cast<const uint8_t*>(Q.data_ptr()), n, cols, ldq, g.group, g.scale, g.lds, g.offset, g.ldo,
                         g.st, Y.data_ptr(), ldy, float_code(Y, "Y"), stream_of(a[5], dev));
  });
}

// gemm4(W, scale, X, Y, offset, group, bias, stream) and, with a shape before
// the stream, gemm4_shaped.
PyObject* call_gemm4(PyObject* const* a, Py_ssize_t n_args, bool shaped) {
  return guarded(shaped ? "uw_i4_gemm_shaped" : "uw_i4_gemm", f_gemm4 && f_gemm4_shaped, n_args, shaped ? 9 : 8, [&] {
    const at::Tensor &W = tensor(a[0], "W"), &X = tensor(a[2], "X"), &Y = tensor(a[3], "Y");
    const int dev = device_of(W, "W");
    want_2d(W, "W");
    want_2d(X, "X");
    const int64_t rows = W.size(0), n = X.size(0), cols = X.size(1);
    if (X.scalar_type() != at::kBFloat16)
      throw TypeProblem(std::string("X must be bfloat16, got ") + c10::toString(X.scalar_type()));
    const int64_t ldx = want_rows(X, n, cols, dev, "X"), ldw = want_packed(W, rows, cols, dev, "W");
    const int64_t ldy = want_rows(Y, n, rows, dev, "Y");
    const Groups g = want_groups(a[1], a[4], a[5], rows, cols, dev);
    const float* bias = a[6] == Py_None ? nullptr : want_scale(tensor(a[6], "bias"), rows, dev, "bias");
    const auto* w = static_cast<const uint8_t*>(W.data_ptr());
    const auto* x = static_cast<const uint16_t*>(X.data_ptr());
    const int yt = float_code(Y, "Y");
    if (!shaped)
      return f_gemm4(w, rows, cols, ldw, g.group, g.scale, g.lds, g.offset, g.ldo, g.st, x, n, ldx, bias, Y.data_ptr(), ldy,
                     yt, stream_of(a[7], dev));
    const long shape = PyLong_AsLong(a[7]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw TypeProblem("shape must be an integer");
    }
    return f_gemm4_shaped(w, rows, cols, ldw, g.group, g.scale, g.lds, g.offset, g.ldo, g.st, x, n, ldx, bias, Y.data_ptr(),
                          ldy, yt, static_cast<int>(std::min(std::max(shape, -1L), 1000000L)), stream_of(a[8], dev));
  });
}

PyObject* py_gemm4(PyObject*, PyObject* const* a, Py_ssize_t n) { return call_gemm4(a, n, false); }
PyObject* py_gemm4_shaped(PyObject*, PyObject* const* a, Py_ssize_t n) { return call_gemm4(a, n, true); }

// bind(rmsnorm, silu_mul, quantize, dequantize, gemm, gemm_shaped, block_norm, quantize4, dequantize4, gemm4,
// gemm4_shaped): addresses
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  constexpr int kEntries = 11;
  void* p[kEntries];
  if (n_args != kEntries) {
    PyErr_SetString(PyExc_TypeError, "bind takes 11 addresses");
    return nullptr;
  }
  for (int i = 0; i < kEntries; ++i) {
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
  f_block_norm = reinterpret_cast<decltype(f_block_norm)>(p[6]);
  f_quantize4 = reinterpret_cast<decltype(f_quantize4)>(p[7]);
  f_dequantize4 = reinterpret_cast<decltype(f_dequantize4)>(p[8]);
  f_gemm4 = reinterpret_cast<decltype(f_gemm4)>(p[9]);
  f_gemm4_shaped = reinterpret_cast<decltype(f_gemm4_shaped)>(p[10]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<py_bind>("bind"),           method<py_rmsnorm>("rmsnorm"),       method<py_silu_mul>("silu_mul"),
    method<py_quantize>("quantize"),   method<py_dequantize>("dequantize"), method<py_gemm>("gemm"),
    method<py_gemm_shaped>("gemm_shaped"), method<py_block_norm>("block_norm"), method<py_quantize4>("quantize4"),
    method<py_dequantize4>("dequantize4"), method<py_gemm4>("gemm4"),     method<py_gemm4_shaped>("gemm4_shaped"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_uw_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__uw_torch() { return PyModule_Create(&module_def); }
