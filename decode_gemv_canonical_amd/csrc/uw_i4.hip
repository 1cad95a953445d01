// Weights in 4-bit integers with a scale (and, in the affine form, an offset)
// per group of G = 32, 64 or 128 columns: from rows of bf16 or fp32, back, and
// their product with bf16 activations on the gfx950 matrix cores.
//
//   W[n, k] = s[g, n] q[n, k] (+ m[g, n]),   g = k / G,  q in -8 .. 7
//   Y[b, n] = sum_g s[g, n] (sum_k q[n, k] X[b, k]) + m[g, n] (sum_k X[b, k]) (+ bias[n])
//
// A row's integers lie two to a byte as q + 8, the even column in the low
// half; rows start at multiples of 16 bytes, and the last 16-byte word of a
// row may be read whole.  Scales and offsets lie group by group, [groups,
// rows], so that the rows of a tile find theirs side by side.  The product's
// kernels are in uw_i4_gemm.h; here is the choice among them.
#include <algorithm>
#include <cmath>

#include "uw_i4.h"

namespace uw {
namespace {

constexpr float kTiny = 1.17549435e-38f;  // 2^-126

__device__ __forceinline__ u32x4 load16_any(const void* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// -- rows in 4 bits and back ----------------------------------------------------

// Values [i, i + 8) of a row of n as fp32; those past the end read as `pad`.
template <bool F32>
__device__ __forceinline__ void load_f8(const char* row, int64_t i, int64_t n, float pad, float (&f)[8]) {
  if (i + 8 <= n) {
    if (F32) {
      const u32x4 a = load16_any(row + 4 * i), b = load16_any(row + 4 * i + 16);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = bits_f32(e < 4 ? a[e] : b[e - 4]);
    } else {
      const u32x4 a = load16_any(row + 2 * i);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = bits_f32((e & 1) ? (a[e / 2] & 0xFFFF0000u) : (a[e / 2] << 16));
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    f[e] = pad;
    if (i + e < n) {
      if (F32) f[e] = reinterpret_cast<const float*>(row)[i + e];
      else f[e] = bits_f32(uint32_t(reinterpret_cast<const uint16_t*>(row)[i + e]) << 16);
    }
  }
}

struct Q4Args {
  const char* X;
  uint8_t* Q;
  char* scale;
  char* offset;
  int64_t rows, cols, ldx, ldq, lds, ldo;
  int32_t st;
  uint32_t per_row;  // workgroups of a row
};

__device__ __forceinline__ void store_scale(char* p, int64_t i, int st, float v) {
  if (st == UW_F32) reinterpret_cast<float*>(p)[i] = v;
  else reinterpret_cast<__bf16*>(p)[i] = static_cast<__bf16>(v);
}

__device__ __forceinline__ float as_kept(float v, int st) {
  return st == UW_F32 ? v : static_cast<float>(static_cast<__bf16>(v));
}

// The integer nearest to the fp32 quotient t / s (ties to even), held to -8 ..
// 7, plus 8.  inv is 1 / s rounded: the quotient is corrected by its residual,
// which gives the rounded quotient, and where t itself is infinite (p - m past
// the fp32 range) stays as it is.  Adding 1.5 * 2^23 + 8 rounds to the nearest
// integer and leaves it in the low bits.
__device__ __forceinline__ uint32_t nibble(float t, float s, float inv) {
#pragma clang fp contract(off)
  const float q0 = t * inv, q1 = fmaf(fmaf(-q0, s, t), inv, q0);
  const float q = fminf(fmaxf(fabsf(q0) < 64.f ? q1 : q0, -8.f), 7.f);
  return f32_bits(q + 12582920.f) & 15u;
}

// One thread holds 8 columns, G / 8 neighbouring lanes a group.
template <bool F32, int G, bool OFF>
__global__ __launch_bounds__(256) void quantize4_kernel(Q4Args a) {
  const int64_t row = blockIdx.x / a.per_row;
  const int64_t i = 8 * (int64_t(blockIdx.x % a.per_row) * 256 + threadIdx.x);
  const char* x = a.X + row * a.ldx * (F32 ? 4 : 2);
  float f[8];
  load_f8<F32>(x, i, a.cols, 0.f, f);
  uint32_t top = 0u;
  float most = -INFINITY, least = INFINITY;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    top = max(top, f32_bits(f[e]) & 0x7FFFFFFFu);
    if (OFF && i + e < a.cols) {
      most = fmaxf(most, f[e]);
      least = fminf(least, f[e]);
    }
  }
#pragma unroll
  for (int d = 1; d < G / 8; d *= 2) {
    top = max(top, uint32_t(__shfl_xor(int(top), d, kWave)));
    if (OFF) {
      most = fmaxf(most, __shfl_xor(most, d, kWave));
      least = fminf(least, __shfl_xor(least, d, kWave));
    }
  }
  if (i >= a.cols) return;
  const bool fine = top < 0x7F800000u;
  float s, m = 0.f;
  {
#pragma clang fp contract(off)
    if (OFF) {
      s = as_kept(fmaxf(most / 15.f - least / 15.f, kTiny), a.st);
      m = as_kept((least * 0.5f + most * 0.5f) + s * 0.5f, a.st);
    } else {
      s = as_kept(fmaxf(bits_f32(top) / 7.f, kTiny), a.st);
    }
  }
  // where s nears the denormal range the residual would leave it: both are scaled up (t is at most 8 s)
  const float up = s < 0x1p-60f ? 0x1p64f : 1.f;
  const float su = s * up, inv = 1.f / su;
  uint32_t w = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = (OFF ? f[e] - m : f[e]) * up;
    w |= (fine ? nibble(t, su, inv) : 8u) << (4 * e);
  }
  uint8_t* q = a.Q + row * a.ldq + i / 2;
  if (i + 8 <= a.cols) {
    *reinterpret_cast<uint32_t*>(q) = w;
  } else {
    const int left = int(a.cols - i);
    if (left & 1) w = (w & ~(15u << (4 * left))) | 8u << (4 * left);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (2 * e < left) q[e] = uint8_t(w >> (8 * e));
  }
  if (i % G == 0) {
    const int64_t g = i / G;
    const float nan = bits_f32(0x7FC00000u);
    store_scale(a.scale, g * a.lds + row, a.st, fine ? s : nan);
    if (OFF) store_scale(a.offset, g * a.ldo + row, a.st, fine ? m : nan);
  }
}

struct D4Args {
  const uint8_t* Q;
  const char* scale;
  const char* offset;
  char* Y;
  int64_t rows, cols, ldq, lds, ldo, ldy;
  int32_t st, yt, log_group;
  uint32_t per_row;
};

// One thread, 8 columns: s q rounded to fp32, the offset added in a rounding
// of its own, then rounded to Y's type.
__global__ __launch_bounds__(256) void dequantize4_kernel(D4Args a) {
#pragma clang fp contract(off)
  const int64_t row = blockIdx.x / a.per_row;
  const int64_t i = 8 * (int64_t(blockIdx.x % a.per_row) * 256 + threadIdx.x);
  if (i >= a.cols) return;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(a.Q + row * a.ldq + i / 2) ^ 0x88888888u;
  const int64_t g = i >> a.log_group;
  const float s = load_scale(a.scale, g * a.lds + row, a.st);
  const float m = a.offset ? load_scale(a.offset, g * a.ldo + row, a.st) : 0.f;
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    f[e] = float(int32_t(w << (28 - 4 * e)) >> 28) * s;
    if (a.offset) f[e] = f[e] + m;
  }
  if (a.yt == UW_F32) {
    float* y = reinterpret_cast<float*>(a.Y) + row * a.ldy + i;
    if (i + 8 <= a.cols) {
      __builtin_memcpy(y, f, 32);
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (i + e < a.cols) y[e] = f[e];
    }
    return;
  }
  uint16_t* y = reinterpret_cast<uint16_t*>(a.Y) + row * a.ldy + i;
  const uint32_t v[4] = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
  if (i + 8 <= a.cols) {
    __builtin_memcpy(y, v, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (i + e < a.cols) y[e] = uint16_t(v[e / 2] >> (16 * (e & 1)));
  }
}

// Rows that a launch takes where each is spread over per_row workgroups of
// 256: a launch holds fewer than 2^32 threads.
int64_t band_rows(int64_t per_row) { return ((int64_t(1) << 24) - 1) / per_row; }

template <bool F32, int G, bool OFF>
int run_quantize(const Q4Args& a, hipStream_t s) {
  const int64_t per_row = (a.cols + 2047) / 2048, band = band_rows(per_row);
  if (band == 0) return fail(UW_ERR_UNSUPPORTED, "uw_i4_quantize: a row wider than a launch holds");
  for (int64_t row0 = 0; row0 < a.rows; row0 += band) {
    Q4Args b = a;
    const int64_t es = a.st == UW_F32 ? 4 : 2;
    b.rows = std::min(band, a.rows - row0);
    b.per_row = uint32_t(per_row);
    b.X += row0 * a.ldx * (F32 ? 4 : 2);
    b.Q += row0 * a.ldq;
    b.scale += row0 * es;
    if (OFF) b.offset += row0 * es;
    hipLaunchKernelGGL((quantize4_kernel<F32, G, OFF>), dim3(unsigned(b.rows * per_row)), dim3(256), 0, s, b);
    if (int rc = hip_check(hipGetLastError(), "quantize4_kernel launch")) return rc;
  }
  return UW_OK;
}

template <bool F32, int G>
int run_quantize_form(const Q4Args& a, hipStream_t s) {
  return a.offset ? run_quantize<F32, G, true>(a, s) : run_quantize<F32, G, false>(a, s);
}

template <bool F32>
int run_quantize_group(const Q4Args& a, int group, hipStream_t s) {
  return group == 32   ? run_quantize_form<F32, 32>(a, s)
         : group == 64 ? run_quantize_form<F32, 64>(a, s)
                       : run_quantize_form<F32, 128>(a, s);
}

// 32-bit offsets inside a tile of 256 rows, and over the scales.
bool offsets_ok(const I4Args& a, int group) {
  const int64_t span = (a.cols + group - 1) / group * (a.st == UW_F32 ? 4 : 2), most = int64_t(1) << 31;
  return a.ldx < (int64_t(1) << 21) && a.ldw < (int64_t(1) << 22) && span * a.lds < most && span * a.ldo < most &&
         a.rows * 4 < most;
}
// 16-byte chunks of the activations.
bool aligned_ok(const I4Args& a) { return reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && a.ldx % 8 == 0; }

// Shapes: weight and batch rows of a workgroup's tile (at groups of 128), and
// the kernel (uw_i4_gemm.h).  per_cu, start, alone, shared, lead and loose are
// for expected_us below.
enum Kind { kDirect, kToken, kStream, kSlice, kDeep, kStage, kLoose };
struct I4Shape {
  int bw, bb;
  Kind kind;
  int per_cu;
  float start, alone, shared, lead, loose;
};
constexpr I4Shape kShapeList[] = {
    {0, 0, kDirect, 1, 0, 0, 0, 0, 0},  // 0: the choice below
    {16, 16, kDirect, 1, 0, 0, 0, 0, 0},
    {32, 4, kToken, 2, 1.20f, 0.0728f, 0.0947f, 0.0053f, 0.0073f},
    {16, 4, kToken, 2, 1.23f, 0.0380f, 0.0481f, 0.0086f, 0.0109f},
    {16, 16, kStream, 4, 2.90f, 0.0236f, 0.0356f, 0.0060f, 0.0094f},
    {64, 16, kSlice, 1, 1.82f, 0.1457f, 0.0004f, 0.0044f, 0.0109f},
    {16, 16, kSlice, 1, 1.78f, 0.0525f, 0.0002f, 0.0043f, 0.0066f},
    {32, 16, kSlice, 1, 1.65f, 0.0847f, 0.0712f, 0.0036f, 0.0090f},
    {16, 16, kDeep, 1, 1.63f, 0.0688f, 0.0590f, 0.0008f, 0},
    {32, 16, kDeep, 1, 1.71f, 0.0960f, 0.0696f, 0.0009f, 0},
    {64, 16, kStage, 1, 2.17f, 0.2215f, 0.0002f, 0.0007f, 0},   // 4 groups of waves
    {64, 32, kStage, 1, 2.80f, 0.2614f, 0.2165f, 0.0014f, 0},   // 4
    {64, 64, kStage, 1, 3.78f, 0.3489f, 0.2762f, 0.0017f, 0},   // 4
    {128, 64, kStage, 1, 3.80f, 0.6068f, 0.5585f, 0.0025f, 0},  // 3
    {128, 128, kStage, 1, 5.01f, 1.2312f, 0.8370f, 0.0009f, 0}, // 2
    {256, 256, kStage, 1, 6.28f, 3.1787f, 2.9768f, 0.0015f, 0},
    {64, 32, kLoose, 1, 2.24f, 0.2958f, 0.2743f, 0.0006f, 0.0015f},   // 4
    {64, 64, kLoose, 1, 3.26f, 0.4365f, 0.3174f, 0.0006f, 0.0022f},   // 4
    {128, 128, kLoose, 1, 5.27f, 1.3357f, 0.9810f, 0.0001f, 0.0030f}, // 2
    {256, 128, kLoose, 1, 4.26f, 1.9368f, 1.9535f, 0.0030f, 0.0071f},
};
constexpr int kShapes = int(sizeof(kShapeList) / sizeof(kShapeList[0]));

bool shape_ok(const I4Args& a, int group, int shape) {
  const Kind kind = kShapeList[shape].kind;
  if (kind == kDirect) return true;
  if (!offsets_ok(a, group)) return false;
  if (kind == kToken) return a.batch <= 4;
  if (kind == kStream) return stream_ok(a, 8);
  return kind == kDeep || kind == kStage ? aligned_ok(a) : true;
}

// What a product takes on a shape, in us: 1.6 for the launch, then rounds of
// workgroups.  Each round costs `start` (first loads, epilogue), `lead` (or
// `loose`, where the rows of X are off 16-byte boundaries) per token and block
// of 128 columns that a workgroup reads, and `alone` per block where it waits on
// its own loads; a compute unit needs `shared` per block and workgroup it holds;
// and the operands' bytes come at 5.4 TB/s.  The three limits of the loop add as
// fourth powers (the largest rules, a near second counts).
// The constants were fitted to the shapes' times on 1993 sizes drawn over 1..4096
// x 64..28672 x 64..14336, all groups, forms and types of scales, half of them
// with rows of X off 16 bytes, each on 3 to 8 rotated operand sets.  Only their
// order counts: the times themselves are up to a quarter off.  On those sizes the
// choice takes 1.03 of the best shape's time in the mean, 95 of 100 under 1.18;
// without any one of the shapes the best would be 0.3 to 3 percent slower in the
// mean and up to 3 times in single sizes.
float expected_us(const I4Shape& s, const I4Args& a, int group, bool aligned) {
  const float blocks = float((a.cols + 127) / 128);
  const int64_t bw = s.kind == kSlice && s.bw == 64 && group == 32 ? 32 : s.bw;
  const int64_t bb = s.bb == 256 && (a.offset || group == 32) ? 192 : s.bb;
  const float n = float((a.rows + bw - 1) / bw) * float((a.batch + bb - 1) / bb) / kCus;
  const float rounds = std::ceil(n / float(s.per_cu));
  const float held = n < 1.f ? n : 0.5f * (n + std::ceil(n));
  const auto p4 = [](float v) { return v * v * v * v; };
  const float loop = p4(blocks * s.alone * rounds) + p4(blocks * s.shared * held) +
                     p4((0.5f * float(a.rows) + 2.f * float(a.batch)) * blocks * (128.f / 5.4e6f));
  return 1.6f + rounds * (s.start + (aligned ? s.lead : s.loose) * blocks * float(std::min(a.batch, bb))) + std::sqrt(std::sqrt(loop));
}

int pick_shape(const I4Args& a, int group) {
  if (!offsets_ok(a, group)) return 1;
  const bool aligned = aligned_ok(a);
  int shape = 1;
  float best = 0.f;
  for (int i = 2; i < kShapes; ++i) {
    if (!shape_ok(a, group, i)) continue;
    // a slice for each 16 tokens reads the weights as often: not past a few of them
    if (kShapeList[i].kind == kSlice && a.batch > 80) continue;
    const float us = expected_us(kShapeList[i], a, group, aligned);
    if (shape == 1 || us < best) {
      best = us;
      shape = i;
    }
  }
  return shape;
}

}  // namespace

int i4_gemm_shape_count() { return kShapes; }

bool i4_gemm_shape_ok(int64_t rows, int64_t cols, int64_t ldw, int group, int64_t lds, int64_t ldo, int st, const uint16_t* X,
                      int64_t batch, int64_t ldx, int shape) {
  I4Args a{};
  a.X = X;
  a.rows = rows;
  a.cols = cols;
  a.batch = batch;
  a.ldw = rows > 1 ? ldw : 0;
  a.ldx = batch > 1 ? ldx : 0;
  a.lds = cols <= group ? 0 : lds;
  a.ldo = cols <= group ? 0 : ldo;
  a.st = st;
  return shape_ok(a, group, shape);
}

int launch_i4_gemm(const uint8_t* W, int64_t rows, int64_t cols, int64_t ldw, int group, const void* scale, int64_t lds,
                   const void* offset, int64_t ldo, int st, const uint16_t* X, int64_t batch, int64_t ldx,
                   const float* bias, void* Y, int64_t ldy, int yt, int shape, void* stream) {
  // a single row has no stride
  const bool one = cols <= group;
  const I4Args a{W, static_cast<const char*>(scale), static_cast<const char*>(offset), X, bias, static_cast<char*>(Y), rows, cols,
                 rows > 1 ? ldw : 0, one ? 0 : lds, one || !offset ? 0 : ldo, batch, batch > 1 ? ldx : 0, ldy, st, yt};
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (shape <= 0) shape = pick_shape(a, group);
  return group == 32 ? i4_gemm_g32(a, shape, s) : group == 64 ? i4_gemm_g64(a, shape, s) : i4_gemm_g128(a, shape, s);
}

int launch_i4_quantize(const void* X, int64_t rows, int64_t cols, int64_t ldx, int xt, int group, uint8_t* Q, int64_t ldq,
                       void* scale, int64_t lds, void* offset, int64_t ldo, int st, void* stream) {
  const Q4Args a{static_cast<const char*>(X), Q, static_cast<char*>(scale), static_cast<char*>(offset), rows, cols, ldx, ldq,
                 lds, ldo, st, 0};
  hipStream_t s = static_cast<hipStream_t>(stream);
  return xt == UW_F32 ? run_quantize_group<true>(a, group, s) : run_quantize_group<false>(a, group, s);
}

int launch_i4_dequantize(const uint8_t* Q, int64_t rows, int64_t cols, int64_t ldq, int group, const void* scale, int64_t lds,
                         const void* offset, int64_t ldo, int st, void* Y, int64_t ldy, int yt, void* stream) {
  const int64_t per_row = (cols + 2047) / 2048, band = band_rows(per_row);
  if (band == 0) return fail(UW_ERR_UNSUPPORTED, "uw_i4_dequantize: a row wider than a launch holds");
  const int64_t es = st == UW_F32 ? 4 : 2;
  for (int64_t row0 = 0; row0 < rows; row0 += band) {
    const D4Args a{Q + row0 * ldq, static_cast<const char*>(scale) + row0 * es,
                   offset ? static_cast<const char*>(offset) + row0 * es : nullptr,
                   static_cast<char*>(Y) + row0 * ldy * int64_t(elem_size(yt)), std::min(band, rows - row0), cols, ldq, lds, ldo,
                   ldy, st, yt, group == 32 ? 5 : group == 64 ? 6 : 7, uint32_t(per_row)};
    hipLaunchKernelGGL(dequantize4_kernel, dim3(unsigned(a.rows * per_row)), dim3(256), 0, static_cast<hipStream_t>(stream), a);
    if (int rc = hip_check(hipGetLastError(), "dequantize4_kernel launch")) return rc;
  }
  return UW_OK;
}

}  // namespace uw
