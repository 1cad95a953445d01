// Entry points of the 8-bit activation path: argument checks, then the
// launchers of uw_rows.hip and uw_i8.hip.
#include <cmath>
#include <string>

#include "uw_checks.h"

using namespace uw;

namespace {

int check_i8_gemm(const char* where, const int8_t* W, int64_t rows, int64_t cols, int64_t ldw, const float* ws,
                  const int8_t* X, int64_t batch, int64_t ldx, const float* xs, const float* bias, const void* Y,
                  int64_t ldy, int yt) {
  if (int rc = check_sizes(where, batch, cols)) return rc;
  if (rows < 1 || rows >= kMaxExtent) return bad(where, "rows out of range");
  if (!float_type(yt)) return bad(where, "Y must be UW_F32 or UW_BF16");
  if (cols > 131071)
    return fail(UW_ERR_UNSUPPORTED, std::string(where) + ": cols > 131071 could overflow the 32-bit sum");
  if (batch == 0) return UW_OK;
  if (int rc = check_rows(where, "W", W, UW_I8, rows, cols, ldw)) return rc;
  if (int rc = check_rows(where, "X", X, UW_I8, batch, cols, ldx)) return rc;
  if (int rc = check_rows(where, "Y", Y, yt, batch, rows, ldy)) return rc;
  if (int rc = check_scale(where, "the weight scales", ws)) return rc;
  if (int rc = check_scale(where, "the activation scales", xs)) return rc;
  if (reinterpret_cast<uintptr_t>(bias) % 4) return bad(where, "bias not aligned");
  return UW_OK;
}

int check_i8_gemm_apart(const char* where, const int8_t* W, int64_t rows, int64_t cols, int64_t ldw, const float* ws,
                        const int8_t* X, int64_t batch, int64_t ldx, const float* xs, const float* bias, const void* Y,
                        int64_t ldy, int yt) {
  return check_apart(where, rows_of("Y", Y, yt, batch, rows, ldy),
                     {rows_of("W", W, UW_I8, rows, cols, ldw), rows_of("X", X, UW_I8, batch, cols, ldx),
                      vector_of("the weight scales", ws, rows), vector_of("the activation scales", xs, batch),
                      vector_of("the bias", bias, rows)},
                     false);
}

}  // namespace

extern "C" {

int uw_rmsnorm(const void* d_X, int64_t batch, int64_t cols, int64_t ldx, int xt, const void* d_R, int64_t ldr, int rt,
               void* d_H, int64_t ldh, const void* d_gain, int gt, float eps, void* d_Y, int64_t ldy, int yt,
               float* d_scale, void* stream) {
  const char* where = "uw_rmsnorm";
  if (int rc = check_sizes(where, batch, cols)) return rc;
  if (!float_type(xt)) return bad(where, "X must be UW_F32 or UW_BF16");
  if (!(eps > 0.f) || !std::isfinite(eps)) return bad(where, "eps must be positive and finite");
  if (d_R && !float_type(rt)) return bad(where, "the residual must be UW_F32 or UW_BF16");
  if (d_H && !d_R) return bad(where, "an output for x + r needs a residual");
  if (d_gain && !float_type(gt)) return bad(where, "the gain must be UW_F32 or UW_BF16");
  if (batch == 0) return UW_OK;
  if (int rc = check_rows(where, "X", d_X, xt, batch, cols, ldx)) return rc;
  if (d_R)
    if (int rc = check_rows(where, "the residual", d_R, rt, batch, cols, ldr)) return rc;
  if (d_H)
    if (int rc = check_rows(where, "the residual's output", d_H, rt, batch, cols, ldh)) return rc;
  if (d_gain)
    if (int rc = check_rows(where, "the gain", d_gain, gt, 1, cols, cols)) return rc;
  if (int rc = check_out(where, d_Y, yt, batch, cols, ldy, d_scale)) return rc;
  const Region x = rows_of("X", d_X, xt, batch, cols, ldx), r = rows_of("the residual", d_R, rt, batch, cols, ldr),
               h = rows_of("the residual's output", d_H, rt, batch, cols, ldh), y = rows_of("Y", d_Y, yt, batch, cols, ldy),
               gain = vector_of("the gain", d_gain, cols, esize(gt)),
               scale = vector_of("the scales", yt == UW_I8 ? d_scale : nullptr, batch);
  if (int rc = check_apart(where, y, {x, r}, true)) return rc;
  if (int rc = check_apart(where, y, {h, gain}, false)) return rc;
  if (int rc = check_apart(where, h, {x, r}, true)) return rc;
  if (int rc = check_apart(where, h, {gain}, false)) return rc;
  if (int rc = check_apart(where, scale, {x, r, gain, h, y}, false)) return rc;
  return launch_rmsnorm(d_X, batch, cols, ldx, xt, d_R, ldr, rt, d_H, ldh, d_gain, gt, eps, d_Y, ldy, yt, d_scale, stream);
}

int uw_silu_mul(const void* d_G, int64_t ldg, const void* d_U, int64_t ldu, int xt, int64_t batch, int64_t cols,
                void* d_Y, int64_t ldy, int yt, float* d_scale, void* stream) {
  const char* where = "uw_silu_mul";
  if (int rc = check_sizes(where, batch, cols)) return rc;
  if (!float_type(xt)) return bad(where, "G and U must be UW_F32 or UW_BF16");
  if (batch == 0) return UW_OK;
  if (int rc = check_rows(where, "G", d_G, xt, batch, cols, ldg)) return rc;
  if (int rc = check_rows(where, "U", d_U, xt, batch, cols, ldu)) return rc;
  if (int rc = check_out(where, d_Y, yt, batch, cols, ldy, d_scale)) return rc;
  const Region g = rows_of("G", d_G, xt, batch, cols, ldg), u = rows_of("U", d_U, xt, batch, cols, ldu),
               y = rows_of("Y", d_Y, yt, batch, cols, ldy),
               scale = vector_of("the scales", yt == UW_I8 ? d_scale : nullptr, batch);
  if (int rc = check_apart(where, y, {g, u}, true)) return rc;
  if (int rc = check_apart(where, scale, {g, u, y}, false)) return rc;
  return launch_silu_mul(d_G, ldg, d_U, ldu, xt, batch, cols, d_Y, ldy, yt, d_scale, stream);
}

int uw_i8_quantize(const void* d_X, int64_t rows, int64_t cols, int64_t ldx, int xt, int8_t* d_Q, int64_t ldq,
                   float* d_scale, void* stream) {
  const char* where = "uw_i8_quantize";
  if (int rc = check_sizes(where, rows, cols)) return rc;
  if (!float_type(xt)) return bad(where, "X must be UW_F32 or UW_BF16");
  if (rows == 0) return UW_OK;
  if (int rc = check_rows(where, "X", d_X, xt, rows, cols, ldx)) return rc;
  if (int rc = check_rows(where, "Q", d_Q, UW_I8, rows, cols, ldq)) return rc;
  if (int rc = check_scale(where, "the scales", d_scale)) return rc;
  const Region x = rows_of("X", d_X, xt, rows, cols, ldx), q = rows_of("Q", d_Q, UW_I8, rows, cols, ldq),
               scale = vector_of("the scales", d_scale, rows);
  if (int rc = check_apart(where, q, {x}, false)) return rc;
  if (int rc = check_apart(where, scale, {x, q}, false)) return rc;
  return launch_i8_quantize(d_X, rows, cols, ldx, xt, d_Q, ldq, d_scale, stream);
}

int uw_i8_dequantize(const int8_t* d_Q, int64_t rows, int64_t cols, int64_t ldq, const float* d_scale, void* d_Y,
                     int64_t ldy, int yt, void* stream) {
  const char* where = "uw_i8_dequantize";
  if (int rc = check_sizes(where, rows, cols)) return rc;
  if (!float_type(yt)) return bad(where, "Y must be UW_F32 or UW_BF16");
  if (rows == 0) return UW_OK;
  if (int rc = check_rows(where, "Q", d_Q, UW_I8, rows, cols, ldq)) return rc;
  if (int rc = check_rows(where, "Y", d_Y, yt, rows, cols, ldy)) return rc;
  if (int rc = check_scale(where, "the scales", d_scale)) return rc;
  if (int rc = check_apart(where, rows_of("Y", d_Y, yt, rows, cols, ldy),
                           {rows_of("Q", d_Q, UW_I8, rows, cols, ldq), vector_of("the scales", d_scale, rows)}, false))
    return rc;
  return launch_i8_dequantize(d_Q, rows, cols, ldq, d_scale, d_Y, ldy, yt, stream);
}

int uw_i8_gemm(const int8_t* d_W, int64_t rows, int64_t cols, int64_t ldw, const float* d_ws, const int8_t* d_X,
               int64_t batch, int64_t ldx, const float* d_xs, const float* d_bias, void* d_Y, int64_t ldy, int yt,
               void* stream) {
  const char* where = "uw_i8_gemm";
  if (int rc = check_i8_gemm(where, d_W, rows, cols, ldw, d_ws, d_X, batch, ldx, d_xs, d_bias, d_Y, ldy, yt)) return rc;
  if (batch == 0) return UW_OK;
  if (int rc = check_i8_gemm_apart(where, d_W, rows, cols, ldw, d_ws, d_X, batch, ldx, d_xs, d_bias, d_Y, ldy, yt)) return rc;
  return launch_i8_gemm(d_W, rows, cols, ldw, d_ws, d_X, batch, ldx, d_xs, d_bias, d_Y, ldy, yt, 0, 0, stream);
}

int uw_i8_gemm_shaped(const int8_t* d_W, int64_t rows, int64_t cols, int64_t ldw, const float* d_ws, const int8_t* d_X,
                      int64_t batch, int64_t ldx, const float* d_xs, const float* d_bias, void* d_Y, int64_t ldy,
                      int yt, int shape, int ks, void* stream) {
  const char* where = "uw_i8_gemm_shaped";
  if (int rc = check_i8_gemm(where, d_W, rows, cols, ldw, d_ws, d_X, batch, ldx, d_xs, d_bias, d_Y, ldy, yt)) return rc;
  if (shape < 1 || shape >= i8_gemm_shape_count() || ks < 0 || ks > 8) return bad(where, "unknown shape or ks");
  if (batch == 0) return UW_OK;
  if (!i8_gemm_shape_ok(d_W, rows, ldw, d_X, batch, ldx, shape))
    return fail(UW_ERR_UNSUPPORTED, std::string(where) + ": a staged shape needs 16-byte aligned operands and strides");
  if (int rc = check_i8_gemm_apart(where, d_W, rows, cols, ldw, d_ws, d_X, batch, ldx, d_xs, d_bias, d_Y, ldy, yt)) return rc;
  return launch_i8_gemm(d_W, rows, cols, ldw, d_ws, d_X, batch, ldx, d_xs, d_bias, d_Y, ldy, yt, shape, ks, stream);
}

int uw_i8_gemm_shape_count(void) { return i8_gemm_shape_count(); }

}  // extern "C"
