// Argument checks that the entry points of the row operators and of the 8-bit
// and 4-bit paths share: sizes, rows, scales, and operands that overlap.
#pragma once

#include <algorithm>
#include <initializer_list>
#include <string>

#include "uw_internal.h"

namespace uw {

// Strides and sizes stay below 2^40 elements, so byte offsets fit in 63 bits.
constexpr int64_t kMaxExtent = int64_t(1) << 40;

inline size_t esize(int t) { return t == UW_F32 ? 4 : t == UW_BF16 ? 2 : 1; }
inline bool float_type(int t) { return t == UW_F32 || t == UW_BF16; }

inline int bad(const char* where, const char* what) { return fail(UW_ERR_INVALID, std::string(where) + ": " + what); }

inline int check_sizes(const char* where, int64_t batch, int64_t cols) {
  if (batch < 0 || batch >= kMaxExtent) return bad(where, "batch out of range");
  if (cols < 1 || cols >= kMaxExtent) return bad(where, "cols out of range");
  return UW_OK;
}

// `batch` rows of `cols` elements of type t with stride ld.
inline int check_rows(const char* where, const char* name, const void* p, int t, int64_t batch, int64_t cols, int64_t ld) {
  if (!p) return bad(where, (std::string("null ") + name).c_str());
  if (reinterpret_cast<uintptr_t>(p) % esize(t))
    return bad(where, (std::string(name) + " not aligned to its element size").c_str());
  if (batch > 1 && (ld < cols || ld >= kMaxExtent))
    return bad(where, (std::string(name) + ": row stride smaller than a row, or out of range").c_str());
  return UW_OK;
}

// The output of a row operator: fp32, bf16, or integers with scales.
inline int check_out(const char* where, const void* Y, int yt, int64_t batch, int64_t cols, int64_t ldy, const float* scale) {
  if (!float_type(yt) && yt != UW_I8) return bad(where, "the output type must be UW_F32, UW_BF16 or UW_I8");
  if (int rc = check_rows(where, "Y", Y, yt, batch, cols, ldy)) return rc;
  if (yt == UW_I8 && (!scale || reinterpret_cast<uintptr_t>(scale) % 4)) return bad(where, "UW_I8 outputs need a scale buffer");
  return UW_OK;
}

inline int check_scale(const char* where, const char* name, const float* p) {
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

inline Region rows_of(const char* name, const void* p, int t, int64_t n, int64_t cols, int64_t ld) {
  return {name, p, n, cols, n > 1 ? ld : cols, esize(t)};
}
inline Region vector_of(const char* name, const void* p, int64_t n, size_t size = 4) { return {name, p, 1, n, n, size}; }

inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }  // b > 0

// Whether any byte belongs to both (rows of one may lie between rows of the other).
inline bool overlap(const Region& a, const Region& b) {
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
inline int check_apart(const char* where, const Region& out, std::initializer_list<Region> others, bool twin) {
  for (const Region& in : others) {
    if (!out.p || !in.p || !overlap(out, in)) continue;
    if (twin && out.p == in.p && out.size == in.size && out.ld == in.ld) continue;
    return bad(where, (std::string(out.name) + " overlaps " + in.name + (twin ? " without being the same rows" : "")).c_str());
  }
  return UW_OK;
}

}  // namespace uw
