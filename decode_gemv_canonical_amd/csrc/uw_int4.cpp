// Entry points of the 4-bit weights and of the block norm: argument checks,
// then the launchers of uw_i4.hip and uw_rows.hip.
#include <cmath>
#include <string>

#include "uw_checks.h"

using namespace uw;

namespace {

int64_t groups_of(int64_t cols, int group) { return (cols + group - 1) / group; }

// Packed 4-bit rows: 16-byte aligned, whole 16-byte words.
int check_packed(const char* where, const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld) {
  if (!p) return bad(where, (std::string("null ") + name).c_str());
  if (reinterpret_cast<uintptr_t>(p) % 16) return bad(where, (std::string(name) + " not 16-byte aligned").c_str());
  if (rows > 1 && (ld % 16 || ld < (cols + 31) / 32 * 16 || ld >= kMaxExtent))
    return bad(where, (std::string(name) + ": the row stride must be a multiple of 16 bytes that holds a row's 16-byte words").c_str());
  return UW_OK;
}

// Scales (and offsets, where given): `groups` rows of `rows` values of type st.
int check_groups4(const char* where, int64_t rows, int64_t cols, int group, const void* scale, int64_t lds,
                  const void* offset, int64_t ldo, int st) {
  const int64_t n = groups_of(cols, group);
  if (int rc = check_rows(where, "the scales", scale, st, n, rows, lds)) return rc;
  if (offset)
    if (int rc = check_rows(where, "the offsets", offset, st, n, rows, ldo)) return rc;
  return UW_OK;
}

int check_form4(const char* where, int64_t rows, int64_t cols, int group, int st) {
  if (int rc = check_sizes(where, rows, cols)) return rc;
  if (group != 32 && group != 64 && group != 128) return bad(where, "the group must be 32, 64 or 128 columns");
  if (!float_type(st)) return bad(where, "the scales must be UW_F32 or UW_BF16");
  return UW_OK;
}

Region packed_of(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return {name, p, rows, (cols + 1) / 2, rows > 1 ? ld : (cols + 1) / 2, 1};
}

int check_i4_gemm(const char* where, const uint8_t* W, int64_t rows, int64_t cols, int64_t ldw, int group,
                  const void* scale, int64_t lds, const void* offset, int64_t ldo, int st, const uint16_t* X,
                  int64_t batch, int64_t ldx, const float* bias, const void* Y, int64_t ldy, int yt) {
  if (int rc = check_form4(where, rows, cols, group, st)) return rc;
  if (rows < 1) return bad(where, "rows out of range");
  if (batch < 0 || batch >= kMaxExtent) return bad(where, "batch out of range");
  if (!float_type(yt)) return bad(where, "Y must be UW_F32 or UW_BF16");
  if (batch == 0) return UW_OK;
  if (int rc = check_packed(where, "W", W, rows, cols, ldw)) return rc;
  if (int rc = check_groups4(where, rows, cols, group, scale, lds, offset, ldo, st)) return rc;
  if (int rc = check_rows(where, "X", X, UW_BF16, batch, cols, ldx)) return rc;
  if (int rc = check_rows(where, "Y", Y, yt, batch, rows, ldy)) return rc;
  if (reinterpret_cast<uintptr_t>(bias) % 4) return bad(where, "bias not aligned");
  const int64_t n = groups_of(cols, group);
  return check_apart(where, rows_of("Y", Y, yt, batch, rows, ldy),
                     {packed_of("W", W, rows, cols, ldw), rows_of("X", X, UW_BF16, batch, cols, ldx),
                      rows_of("the scales", scale, st, n, rows, lds), rows_of("the offsets", offset, st, n, rows, ldo),
                      vector_of("the bias", bias, rows)},
                     false);
}

}  // namespace

extern "C" {

int uw_i4_quantize(const void* d_X, int64_t rows, int64_t cols, int64_t ldx, int xt, int group, uint8_t* d_Q, int64_t ldq,
                   void* d_scale, int64_t lds, void* d_offset, int64_t ldo, int st, void* stream) {
  const char* where = "uw_i4_quantize";
  if (int rc = check_form4(where, rows, cols, group, st)) return rc;
  if (!float_type(xt)) return bad(where, "X must be UW_F32 or UW_BF16");
  if (rows == 0) return UW_OK;
  if (int rc = check_rows(where, "X", d_X, xt, rows, cols, ldx)) return rc;
  if (int rc = check_packed(where, "Q", d_Q, rows, cols, ldq)) return rc;
  if (int rc = check_groups4(where, rows, cols, group, d_scale, lds, d_offset, ldo, st)) return rc;
  const int64_t n = groups_of(cols, group);
  const Region x = rows_of("X", d_X, xt, rows, cols, ldx), q = packed_of("Q", d_Q, rows, cols, ldq),
               s = rows_of("the scales", d_scale, st, n, rows, lds), m = rows_of("the offsets", d_offset, st, n, rows, ldo);
  if (int rc = check_apart(where, q, {x}, false)) return rc;
  if (int rc = check_apart(where, s, {x, q}, false)) return rc;
  if (int rc = check_apart(where, m, {x, q, s}, false)) return rc;
  return launch_i4_quantize(d_X, rows, cols, ldx, xt, group, d_Q, ldq, d_scale, lds, d_offset, ldo, st, stream);
}

int uw_i4_dequantize(const uint8_t* d_Q, int64_t rows, int64_t cols, int64_t ldq, int group, const void* d_scale,
                     int64_t lds, const void* d_offset, int64_t ldo, int st, void* d_Y, int64_t ldy, int yt, void* stream) {
  const char* where = "uw_i4_dequantize";
  if (int rc = check_form4(where, rows, cols, group, st)) return rc;
  if (!float_type(yt)) return bad(where, "Y must be UW_F32 or UW_BF16");
  if (rows == 0) return UW_OK;
  if (int rc = check_packed(where, "Q", d_Q, rows, cols, ldq)) return rc;
  if (int rc = check_groups4(where, rows, cols, group, d_scale, lds, d_offset, ldo, st)) return rc;
  if (int rc = check_rows(where, "Y", d_Y, yt, rows, cols, ldy)) return rc;
  const int64_t n = groups_of(cols, group);
  if (int rc = check_apart(where, rows_of("Y", d_Y, yt, rows, cols, ldy),
                           {packed_of("Q", d_Q, rows, cols, ldq), rows_of("the scales", d_scale, st, n, rows, lds),
                            rows_of("the offsets", d_offset, st, n, rows, ldo)},
                           false))
    return rc;
  return launch_i4_dequantize(d_Q, rows, cols, ldq, group, d_scale, lds, d_offset, ldo, st, d_Y, ldy, yt, stream);
}

int uw_i4_gemm(const uint8_t* d_W, int64_t rows, int64_t cols, int64_t ldw, int group, const void* d_scale, int64_t lds,
               const void* d_offset, int64_t ldo, int st, const uint16_t* d_X, int64_t batch, int64_t ldx,
               const float* d_bias, void* d_Y, int64_t ldy, int yt, void* stream) {
  if (int rc = check_i4_gemm("uw_i4_gemm", d_W, rows, cols, ldw, group, d_scale, lds, d_offset, ldo, st, d_X, batch, ldx,
                             d_bias, d_Y, ldy, yt))
    return rc;
  if (batch == 0) return UW_OK;
  return launch_i4_gemm(d_W, rows, cols, ldw, group, d_scale, lds, d_offset, ldo, st, d_X, batch, ldx, d_bias, d_Y, ldy, yt,
                        0, stream);
}

int uw_i4_gemm_shaped(const uint8_t* d_W, int64_t rows, int64_t cols, int64_t ldw, int group, const void* d_scale,
                      int64_t lds, const void* d_offset, int64_t ldo, int st, const uint16_t* d_X, int64_t batch,
                      int64_t ldx, const float* d_bias, void* d_Y, int64_t ldy, int yt, int shape, void* stream) {
  const char* where = "uw_i4_gemm_shaped";
  if (int rc = check_i4_gemm(where, d_W, rows, cols, ldw, group, d_scale, lds, d_offset, ldo, st, d_X, batch, ldx, d_bias, d_Y,
                             ldy, yt))
    return rc;
  if (shape < 1 || shape >= i4_gemm_shape_count()) return bad(where, "unknown shape");
  if (batch == 0) return UW_OK;
  if (!i4_gemm_shape_ok(rows, cols, ldw, group, lds, d_offset ? ldo : 0, st, d_X, batch, ldx, shape))
    return fail(UW_ERR_UNSUPPORTED, std::string(where) + ": the shape does not take these operands (their alignment, strides or number of tokens)");
  return launch_i4_gemm(d_W, rows, cols, ldw, group, d_scale, lds, d_offset, ldo, st, d_X, batch, ldx, d_bias, d_Y, ldy, yt,
                        shape, stream);
}

int uw_i4_gemm_shape_count(void) { return i4_gemm_shape_count(); }

int uw_block_norm(const void* d_X, int64_t batch, int64_t cols, int64_t ldx, int xt, int post_norm, const void* d_post,
                  int pt, float post_eps, const void* d_gate, int64_t ldg, int gt, float block_scale, const void* d_R,
                  int64_t ldr, int rt, float residual_scale, void* d_H, int64_t ldh, const void* d_gain, int nt, float eps,
                  void* d_Y, int64_t ldy, int yt, float* d_scale, void* stream) {
  const char* where = "uw_block_norm";
  if (int rc = check_sizes(where, batch, cols)) return rc;
  if (!float_type(xt)) return bad(where, "X must be UW_F32 or UW_BF16");
  if (!float_type(rt)) return bad(where, "the residual must be UW_F32 or UW_BF16");
  if (post_norm && (!(post_eps > 0.f) || !std::isfinite(post_eps))) return bad(where, "post_eps must be positive and finite");
  if (d_Y && (!(eps > 0.f) || !std::isfinite(eps))) return bad(where, "eps must be positive and finite");
  if (!std::isfinite(block_scale) || !std::isfinite(residual_scale)) return bad(where, "block_scale and residual_scale must be finite");
  if (d_post && !post_norm) return bad(where, "a post gain without the post norm");
  if (d_gain && !d_Y && batch) return bad(where, "a gain without Y");
  if (d_post && !float_type(pt)) return bad(where, "the post gain must be UW_F32 or UW_BF16");
  if (d_gate && !float_type(gt)) return bad(where, "the gate must be UW_F32 or UW_BF16");
  if (d_gain && !float_type(nt)) return bad(where, "the gain must be UW_F32 or UW_BF16");
  if (batch == 0) return UW_OK;
  if (!d_H && !d_Y) return bad(where, "nothing to write: H and Y are both null");
  if (int rc = check_rows(where, "X", d_X, xt, batch, cols, ldx)) return rc;
  if (int rc = check_rows(where, "the residual", d_R, rt, batch, cols, ldr)) return rc;
  if (d_H)
    if (int rc = check_rows(where, "the residual's output", d_H, rt, batch, cols, ldh)) return rc;
  if (d_post)
    if (int rc = check_rows(where, "the post gain", d_post, pt, 1, cols, cols)) return rc;
  if (d_gate)  // stride 0: one row for every token
    if (int rc = check_rows(where, "the gate", d_gate, gt, ldg ? batch : 1, cols, ldg)) return rc;
  if (d_gain)
    if (int rc = check_rows(where, "the gain", d_gain, nt, 1, cols, cols)) return rc;
  if (d_Y)
    if (int rc = check_out(where, d_Y, yt, batch, cols, ldy, d_scale)) return rc;
  const Region x = rows_of("X", d_X, xt, batch, cols, ldx), r = rows_of("the residual", d_R, rt, batch, cols, ldr),
               h = rows_of("the residual's output", d_H, rt, batch, cols, ldh),
               y = rows_of("Y", d_Y, d_Y ? yt : UW_F32, batch, cols, ldy),
               gate = rows_of("the gate", d_gate, gt, ldg ? batch : 1, cols, ldg),
               post = vector_of("the post gain", d_post, cols, esize(pt)), gain = vector_of("the gain", d_gain, cols, esize(nt)),
               scale = vector_of("the scales", d_Y && yt == UW_I8 ? d_scale : nullptr, batch);
  if (int rc = check_apart(where, y, {x, r}, true)) return rc;
  if (int rc = check_apart(where, y, {h, post, gate, gain}, false)) return rc;
  if (int rc = check_apart(where, h, {x, r}, true)) return rc;
  if (int rc = check_apart(where, h, {post, gate, gain}, false)) return rc;
  if (int rc = check_apart(where, scale, {x, r, post, gate, gain, h, y}, false)) return rc;
  return launch_block_norm(d_X, batch, cols, ldx, xt, post_norm != 0, d_post, pt, post_eps, d_gate, ldg, gt, block_scale, d_R,
                           ldr, rt, residual_scale, d_H, ldh, d_gain, nt, eps, d_Y, ldy, yt, d_scale, stream);
}

}  // extern "C"
