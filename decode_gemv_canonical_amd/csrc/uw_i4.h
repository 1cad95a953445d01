// What the files of the 4-bit weights share: the operands of their product, and
// its launchers, one for each size of a group.
#pragma once

#include <algorithm>

#include "uw_device.h"

namespace uw {

constexpr int kXcds = 8;
constexpr int kCus = 256;

struct I4Args {
  const uint8_t* W;
  const char* scale;
  const char* offset;  // null: none
  const uint16_t* X;
  const float* bias;  // may be null
  char* Y;
  int64_t rows, cols, ldw, lds, ldo, batch, ldx, ldy;  // ldw in bytes, the others in elements
  int32_t st, yt;                                      // types of the scales and of Y
};

// shape: an index below i4_gemm_shape_count() that takes the operands.
int i4_gemm_g32(const I4Args& a, int shape, hipStream_t s);
int i4_gemm_g64(const I4Args& a, int shape, hipStream_t s);
int i4_gemm_g128(const I4Args& a, int shape, hipStream_t s);

// LDS of the stream kernel.
inline uint32_t stream_pitch(int64_t cols) { return uint32_t((cols + 127) / 128 * 256 + 16); }
inline int64_t stream_lds(const I4Args& a, int kw) {
  return a.batch * int64_t(stream_pitch(a.cols)) + int64_t(2) * kw * ((a.batch + 3) / 4) * 256;
}
inline bool stream_ok(const I4Args& a, int kw) {
  return a.batch <= 16 && a.cols <= 65536 && (a.rows + 16) * a.ldw < (int64_t(1) << 31) && stream_lds(a, kw) <= kLdsLimit;
}

__device__ __forceinline__ float load_scale(const char* p, int64_t i, int st) {
  if (st == UW_F32) return reinterpret_cast<const float*>(p)[i];
  return bits_f32(uint32_t(reinterpret_cast<const uint16_t*>(p)[i]) << 16);
}

}  // namespace uw
