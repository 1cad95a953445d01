// Entry points of the 8-bit activation path: argument checks, then the
// launchers of uw_rows.hip and uw_i8.hip.
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <string>

#include "uw_internal.h"

using namespace uw;

namespace {

// Strides and sizes stay below 2^40 elements, so byte offsets fit in 63 bits.
constexpr int64_t kMaxExtent = int64_t(1) << 40;

size_t esize(int t) { return t == UW_F32 ? 4 : t == UW_BF16 ? 2 : 1; }
bool float_type(int t) { return t == UW_F32 || t == UW_BF16; }

int bad(const char* where, const char* what) { return fail(UW_ERR_INVALID, std::string(where) + ": " + what); }

int check_sizes(const char* where, int64_t batch, int64_t cols) {
  if (batch < 0 || batch >= kMaxExtent) return bad(where, "batch out of range");
  if (cols < 1 || cols >= kMaxExtent) return bad(where, "cols out of range");
  return UW_OK;
}

// `batch` rows of `cols` elements of type t with stride ld.
int check_rows(const char* where, const char* name, const void* p, int t, int64_t batch, int64_t cols, int64_t ld) {
  if (!p) return bad(where, (std::string("null ") + name).c_str());
  if (reinterpret_cast<uintptr_t>(p) % esize(t))
    return bad(where, (std::string(name) + " not aligned to its element size").c_str());
  if (batch > 1 && (ld < cols || ld >= kMaxExtent))
    return bad(where, (std::string(name) + ": row stride smaller than a row, or out of range").c_str());
  return UW_OK;
}

// The output of a row operator: fp32, bf16, or integers with scales.
int check_out(const char* where, const void* Y, int yt, int64_t batch, int64_t cols, int64_t ldy, const float* scale) {
  if (!float_type(yt) && yt != UW_I8) return bad(where, "the output type must be UW_F32, UW_BF16 or UW_I8");
  if (int rc = check_rows(where, "Y", Y, yt, batch, cols, ldy)) return rc;
  if (yt == UW_I8 && (!scale || reinterpret_cast<uintptr_t>(scale) % 4)) return bad(where, "UW_I8 outputs need a scale buffer");
  return UW_OK;
}

int check_scale(const char* where, const char* name, const float* p) {
  if (!p || reinterpret_cast<uintptr_t>(p) % 4) return bad(where, (std::string(name) + " null or not aligned").c_str());
  return UW_OK;
}

// An operand in memory: n rows of `width` elements of `size` bytes, `ld` elements apart.
struct Region {
  const char* name;
  const void* p;  // null: not given
  int64_t n, width, ld;
  size_t size;
};

Region rows_of(const char* name, const void* p, int t, int64_t n, int64_t cols, int64_t ld) {
  return {name, p, n, cols, n > 1 ? ld : cols, esize(t)};
}
Region vector_of(const char* name, const void* p, int64_t n, size_t size = 4) { return {name, p, 1, n, n, size}; }

int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }  // b > 0

// Whether any byte belongs to both (rows of one may lie between rows of the other).
bool overlap(const Region& a, const Region& b) {
  // past 2^56 bytes there is no such memory, and the offsets below would not fit
  constexpr double kMost = 72057594037927936.0;
  if (double(a.n) * double(a.ld) * double(a.size) > kMost || double(b.n) * double(b.ld) * double(b.size) > kMost) return false;
  const int64_t as = a.ld * int64_t(a.size), bs = b.ld * int64_t(b.size);
  const int64_t aw = a.width * int64_t(a.size), bw = b.width * int64_t(b.size);
  const int64_t off = reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p);
  if (off >= (a.n - 1) * as + aw || -off >= (b.n - 1) * bs + bw) return false;
  // rows of b that start less than bw before row i of a, or inside it
  auto meets = [&](int64_t i, int64_t j_min, int64_t j_max) {
    const int64_t at = i * as - off;
    return std::max(j_min, floor_div(at - bw, bs) + 1) <= std::min(j_max, floor_div(at + aw - 1, bs));
  };
  if (as == bs) return meets(0, -(a.n - 1), b.n - 1);  // only the difference of the rows' numbers counts
  for (int64_t i = 0; i < a.n; ++i)
    if (meets(i, 0, b.n - 1)) return true;
  return false;
}

// An output against inputs (and other outputs).  twin: inputs that the output
// may replace element for element, where type and stride are the same.
int check_apart(const char* where, const Region& out, std::initializer_list<Region> others, bool twin) {
  for (const Region& in : others) {
    if (!out.p || !in.p || !overlap(out, in)) continue;
    if (twin && out.p == in.p && out.size == in.size && out.ld == in.ld) continue;
    return bad(where, (std::string(out.name) + " overlaps " + in.name + (twin ? " without being the same rows" : "")).c_str());
  }
  return UW_OK;
}

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
