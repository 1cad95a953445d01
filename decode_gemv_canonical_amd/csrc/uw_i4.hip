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

// Eight values as they lie in memory.
struct Raw8 {
  u32x4 a, b;  // b: of fp32
};
// The first `left` (1 .. 7) of them, the others zero.
template <bool F32>
__device__ __forceinline__ Raw8 load_part(const char* p, int left) {
  Raw8 v{u32x4{0u, 0u, 0u, 0u}, u32x4{0u, 0u, 0u, 0u}};
#pragma unroll
  for (int e = 0; e < 7; ++e) {
    if (e >= left) continue;
    if (F32) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(p)[e];
      if (e < 4) v.a[e] = w;
      else v.b[e - 4] = w;
    } else {
      v.a[e / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(p)[e]) << (16 * (e & 1));
    }
  }
  return v;
}
template <bool F32>
__device__ __forceinline__ void unpack8(const Raw8& v, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (F32) f[e] = bits_f32(e < 4 ? v.a[e] : v.b[e - 4]);
    else f[e] = bits_f32((e & 1) ? (v.a[e / 2] & 0xFFFF0000u) : (v.a[e / 2] << 16));
  }
}

// A workgroup of 256 threads takes 16 rows (8 where those are few) by kTileCols
// columns, a wave a row at a time with all its loads issued first, so that the
// scales of a group go out (and come in) for 16 rows side by side: a row at a
// time they cost as much as the matrix (14336 x 4096, groups of 32 with offsets:
// 55 us, with these tiles 38.4; back 53, 34.2).  Bytes bound the plain forms (groups
// of 128: 33.6 us from bf16, 4.4 TB/s; 50 from fp32, 5.3; back 30.4, 4.9, or 23.6
// right behind the quantisation, while the caches hold the integers), the vector
// ALU the quantisation with offsets (the quotients, and the smallest and largest
// value, of every 8 values).
constexpr int kTileCols = 512;

struct Q4Args {
  const char* X;
  uint8_t* Q;
  char* scale;
  char* offset;
  int64_t rows, cols, ldx, ldq, lds, ldo;
  int32_t st;
  uint32_t across;  // tiles of a row
};

// Over the 4, 8 or 16 lanes of a group: DPP within rows of 16 lanes.
template <int N, class F>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, F f) {
  v = f(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 0xF, 0xF, false)));   // quad_perm 1,0,3,2
  v = f(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x4E, 0xF, 0xF, false)));   // quad_perm 2,3,0,1
  if (N > 4) v = f(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x141, 0xF, 0xF, false)));  // row_half_mirror
  if (N > 8) v = f(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x140, 0xF, 0xF, false)));  // row_mirror
  return v;
}

__device__ __forceinline__ void store_scale(char* p, int64_t i, int st, float v) {
  if (st == UW_F32) reinterpret_cast<float*>(p)[i] = v;
  else reinterpret_cast<__bf16*>(p)[i] = static_cast<__bf16>(v);
}

__device__ __forceinline__ float as_kept(float v, int st) {
  return st == UW_F32 ? v : static_cast<float>(static_cast<__bf16>(v));
}

// The bits of 1.5 * 2^23 + 8 plus the integer nearest to the fp32 quotient t / s
// (ties to even), held to -8 .. 7: the sum rounds, and leaves the integer in the
// low bits.  inv is 1 / s rounded.  The product with it is corrected by its
// residual, which gives the rounded quotient; held to +-16 before, an infinite t
// (p - m past the fp32 range) comes out infinite rather than NaN.
constexpr uint32_t kNibbleBase = 0x4B400000u;
__device__ __forceinline__ uint32_t nibble(float t, float s, float inv) {
#pragma clang fp contract(off)
  const float q0 = __builtin_amdgcn_fmed3f(t * inv, -16.f, 16.f), q1 = fmaf(fmaf(-q0, s, t), inv, q0);
  return f32_bits(__builtin_amdgcn_fmed3f(q1, -8.f, 7.f) + 12582920.f);
}

// A lane holds 8 columns, G / 8 neighbouring lanes a group, a wave STEPS rows.
template <bool F32, int G, bool OFF, int STEPS>
__global__ __launch_bounds__(256) void quantize4_kernel(Q4Args a) {
  constexpr int kGroups = kTileCols / G, kRows = 4 * STEPS;
  __shared__ float s_scale[kGroups][kRows + 1], s_offset[OFF ? kGroups : 1][kRows + 1];
  const int64_t row0 = int64_t(blockIdx.x / a.across) * kRows, col0 = int64_t(blockIdx.x % a.across) * kTileCols;
  const int lane = int(threadIdx.x) % kWave, wave = int(threadIdx.x) / kWave;
  const int64_t i = col0 + 8 * lane;
  const int left = int(std::min<int64_t>(a.cols - i, 8));  // of the lane's columns
  // rows past the last read it again
  const char* x[STEPS];
#pragma unroll
  for (int u = 0; u < STEPS; ++u)
    x[u] = a.X + (std::min<int64_t>(row0 + 4 * u + wave, a.rows - 1) * a.ldx + i) * (F32 ? 4 : 2);
  Raw8 raw[STEPS] = {};
  if (left == 8) {
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      raw[u].a = load16_any(x[u]);
      if (F32) raw[u].b = load16_any(x[u] + 16);
    }
  } else if (left > 0) {
#pragma unroll
    for (int u = 0; u < STEPS; ++u) raw[u] = load_part<F32>(x[u], left);
  }
#pragma unroll
  for (int u = 0; u < STEPS; ++u) {
    const int64_t row = row0 + 4 * u + wave;
    float f[8];
    unpack8<F32>(raw[u], f);
    uint32_t top;
    if (F32) {
      const u32x4 v = raw[u].a & 0x7FFFFFFFu, w = raw[u].b & 0x7FFFFFFFu;
      top = max(max(max(v[0], v[1]), max(v[2], v[3])), max(max(w[0], w[1]), max(w[2], w[3])));
    } else {
      using u16x8 = uint16_t __attribute__((ext_vector_type(8)));
      const u32x4 v = raw[u].a & 0x7FFF7FFFu;
      const u16x8 h = __builtin_bit_cast(u16x8, v);
      const auto m = __builtin_elementwise_max(__builtin_elementwise_max(h.s01, h.s23), __builtin_elementwise_max(h.s45, h.s67));
      top = max(uint32_t(m[0]), uint32_t(m[1])) << 16;
    }
    top = group_reduce<G / 8>(top, [](uint32_t p, uint32_t q) { return max(p, q); });
    float most = -INFINITY, least = INFINITY;
    if (OFF) {
      if (left < 8) {
#pragma unroll
        for (int e = 1; e < 8; ++e) f[e] = e < left ? f[e] : f[0];
      }
      if (left > 0) {
        most = least = f[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) {
          most = fmaxf(most, f[e]);
          least = fminf(least, f[e]);
        }
      }
      most = bits_f32(group_reduce<G / 8>(f32_bits(most), [](uint32_t p, uint32_t q) { return f32_bits(fmaxf(bits_f32(p), bits_f32(q))); }));
      least = bits_f32(group_reduce<G / 8>(f32_bits(least), [](uint32_t p, uint32_t q) { return f32_bits(fminf(bits_f32(p), bits_f32(q))); }));
    }
    if (left <= 0 || row >= a.rows) continue;
    const bool fine = top < 0x7F800000u;
    float s, m = 0.f;
    {
#pragma clang fp contract(off)
      if (OFF) {
        s = as_kept(fmaxf(most * (1.f / 15.f) - least * (1.f / 15.f), kTiny), a.st);
        m = as_kept((least * 0.5f + most * 0.5f) + s * 0.5f, a.st);
      } else {
        s = as_kept(fmaxf(bits_f32(top) * (1.f / 7.f), kTiny), a.st);
      }
    }
    // where s nears the denormal range the residual would leave it: both are scaled up (a t that this takes past the fp32
    // range is many s, and held as an infinite one is)
    const float up = s < 0x1p-60f ? 0x1p64f : 1.f;
    const float su = s * up, inv = 1.f / su;
    uint32_t w = 0u - kNibbleBase * 0x11111111u;
#pragma unroll
    for (int e = 0; e < 8; ++e) w += nibble((OFF ? f[e] - m : f[e]) * up, su, inv) << (4 * e);
    if (!fine) w = 0x88888888u;
    uint8_t* q = a.Q + row * a.ldq + i / 2;
    if (left == 8) {
      *reinterpret_cast<uint32_t*>(q) = w;
    } else {
      if (left & 1) w = (w & ~(15u << (4 * left))) | 8u << (4 * left);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (2 * e < left) q[e] = uint8_t(w >> (8 * e));
    }
    if (lane % (G / 8) == 0) {
      const float nan = bits_f32(0x7FC00000u);
      s_scale[lane / (G / 8)][4 * u + wave] = fine ? s : nan;
      if (OFF) s_offset[lane / (G / 8)][4 * u + wave] = fine ? m : nan;
    }
  }
  __syncthreads();
  for (int at = int(threadIdx.x); at < kGroups * kRows; at += 256) {
    const int g = at / kRows, r = at % kRows;
    if (col0 + int64_t(g) * G >= a.cols || row0 + r >= a.rows) continue;
    const int64_t to = col0 / G + g;
    store_scale(a.scale, to * a.lds + row0 + r, a.st, s_scale[g][r]);
    if (OFF) store_scale(a.offset, to * a.ldo + row0 + r, a.st, s_offset[g][r]);
  }
}

struct D4Args {
  const uint8_t* Q;
  const char* scale;
  const char* offset;
  char* Y;
  int64_t rows, cols, ldq, lds, ldo, ldy;
  int32_t st, log_group;
  uint32_t across;
};

// The same tile; s q rounded to fp32, the offset added in a rounding of its
// own, then rounded to Y's type.
template <bool OFF, bool YF32, int STEPS>
__global__ __launch_bounds__(256) void dequantize4_kernel(D4Args a) {
#pragma clang fp contract(off)
  constexpr int kRows = 4 * STEPS;
  __shared__ float s_scale[kTileCols / 32][kRows + 1], s_offset[OFF ? kTileCols / 32 : 1][kRows + 1];
  const int64_t row0 = int64_t(blockIdx.x / a.across) * kRows, col0 = int64_t(blockIdx.x % a.across) * kTileCols;
  const int lane = int(threadIdx.x) % kWave, wave = int(threadIdx.x) / kWave;
  const int64_t i = col0 + 8 * lane;
  uint32_t words[STEPS];
#pragma unroll
  for (int u = 0; u < STEPS; ++u) {
    const int64_t row = std::min<int64_t>(row0 + 4 * u + wave, a.rows - 1);
    words[u] = *reinterpret_cast<const uint32_t*>(a.Q + row * a.ldq + std::min<int64_t>(i, a.cols - 1) / 8 * 4);
  }
  const int64_t groups = ((a.cols - 1) >> a.log_group) + 1, first = col0 >> a.log_group;
  for (int at = int(threadIdx.x); at < (kTileCols >> a.log_group) * kRows; at += 256) {
    const int g = at / kRows, r = at % kRows;
    const int64_t from = std::min(first + g, groups - 1), row = std::min<int64_t>(row0 + r, a.rows - 1);
    s_scale[g][r] = load_scale(a.scale, from * a.lds + row, a.st);
    if (OFF) s_offset[g][r] = load_scale(a.offset, from * a.ldo + row, a.st);
  }
  __syncthreads();
  if (i >= a.cols) return;
  const int g = (8 * lane) >> a.log_group;
#pragma unroll
  for (int u = 0; u < STEPS; ++u) {
    const int r = 4 * u + wave;
    if (row0 + r >= a.rows) break;
    const uint32_t w = words[u] ^ 0x88888888u;
    const float s = s_scale[g][r], m = OFF ? s_offset[g][r] : 0.f;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] = float(int32_t(w << (28 - 4 * e)) >> 28) * s;
      if (OFF) f[e] = f[e] + m;
    }
    if (YF32) {
      float* y = reinterpret_cast<float*>(a.Y) + (row0 + r) * a.ldy + i;
      if (i + 8 <= a.cols) {
        __builtin_memcpy(y, f, 32);
      } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
          if (i + e < a.cols) y[e] = f[e];
      }
      continue;
    }
    uint16_t* y = reinterpret_cast<uint16_t*>(a.Y) + (row0 + r) * a.ldy + i;
    const uint32_t v[4] = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
    if (i + 8 <= a.cols) {
      __builtin_memcpy(y, v, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (i + e < a.cols) y[e] = uint16_t(v[e / 2] >> (16 * (e & 1)));
    }
  }
}

// Rows that a launch takes where `across` tiles cover a row: it holds fewer
// than 2^32 threads.  0: not even one tile high.
int64_t band_rows(int64_t across, int steps) { return ((int64_t(1) << 24) - 1) / across * (4 * steps); }
int64_t tiles_across(int64_t cols) { return (cols + kTileCols - 1) / kTileCols; }
unsigned tiles_of(int64_t rows, int64_t across, int steps) {
  return unsigned((rows + 4 * steps - 1) / (4 * steps) * across);
}

// Tiles of 16 rows where they fill the compute units four times over, else of 8
// (37 x 1001 takes 3.5 us then, with 32 10.5).
bool tall_tiles(int64_t rows, int64_t cols) { return (rows + 15) / 16 >= (4 * kCus + tiles_across(cols) - 1) / tiles_across(cols); }

template <bool F32, int G, bool OFF, int STEPS>
int run_quantize_steps(const Q4Args& a, hipStream_t s) {
  const int64_t across = tiles_across(a.cols), band = band_rows(across, STEPS);
  if (band == 0) return fail(UW_ERR_UNSUPPORTED, "uw_i4_quantize: a row wider than a launch holds");
  for (int64_t row0 = 0; row0 < a.rows; row0 += band) {
    Q4Args b = a;
    const int64_t es = a.st == UW_F32 ? 4 : 2;
    b.rows = std::min(band, a.rows - row0);
    b.across = uint32_t(across);
    b.X += row0 * a.ldx * (F32 ? 4 : 2);
    b.Q += row0 * a.ldq;
    b.scale += row0 * es;
    if (OFF) b.offset += row0 * es;
    hipLaunchKernelGGL((quantize4_kernel<F32, G, OFF, STEPS>), dim3(tiles_of(b.rows, across, STEPS)), dim3(256), 0, s, b);
    if (int rc = hip_check(hipGetLastError(), "quantize4_kernel launch")) return rc;
  }
  return UW_OK;
}

template <bool F32, int G, bool OFF>
int run_quantize(const Q4Args& a, hipStream_t s) {
  return tall_tiles(a.rows, a.cols) ? run_quantize_steps<F32, G, OFF, 4>(a, s) : run_quantize_steps<F32, G, OFF, 2>(a, s);
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

// 32-bit offsets inside a tile of 256 rows, and over the scales.  (Where there is
// one row the stride says nothing of its length.)
bool offsets_ok(const I4Args& a, int group) {
  if (a.cols >= int64_t(1) << 21) return false;
  const int64_t span = (a.cols + group - 1) / group * (a.st == UW_F32 ? 4 : 2), most = int64_t(1) << 31;
  return a.ldx < (int64_t(1) << 21) && a.ldw < (int64_t(1) << 22) && span * a.lds < most && span * a.ldo < most &&
         a.rows * 4 < most;
}
// 16-byte chunks of the activations.
bool aligned_ok(const I4Args& a) { return reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && a.ldx % 8 == 0; }

// Shapes: weight and batch rows of a workgroup's tile (at groups of 128), the
// kernel (uw_i4_gemm.h) and the threads of a workgroup (of kDirect at most).
// per_cu, start, alone, shared, lead and loose are for expected_us below.
enum Kind { kDirect, kToken, kStream, kSlice, kDeep, kStage, kLoose };
struct I4Shape {
  int bw, bb;
  Kind kind;
  int threads;
  int per_cu;
  float start, alone, shared, lead, loose;
};
constexpr I4Shape kShapeList[] = {
    {0, 0, kDirect, 0, 1, 0, 0, 0, 0, 0},  // 0: the choice below
    {16, 16, kDirect, 512, 1, 0, 0, 0, 0, 0},
    {32, 4, kToken, 512, 1, 1.07f, 0.0718f, 0.0008f, 0.0062f, 0.0079f},
    {16, 4, kToken, 512, 2, 1.18f, 0.0291f, 0.0456f, 0.0112f, 0.0125f},
    {16, 16, kStream, 512, 4, 2.89f, 0.0192f, 0.0353f, 0.0066f, 0.0095f},
    {64, 16, kSlice, 512, 1, 1.84f, 0.1460f, 0.0006f, 0.0047f, 0.0109f},
    {16, 16, kSlice, 1024, 1, 1.78f, 0.0539f, 0, 0.0040f, 0.0068f},
    {32, 16, kSlice, 1024, 1, 1.65f, 0.0865f, 0.0508f, 0.0035f, 0.0092f},
    {16, 16, kDeep, 512, 1, 1.63f, 0.0711f, 0.0607f, 0.0007f, 0},
    {32, 16, kDeep, 512, 1, 1.73f, 0.0952f, 0.0571f, 0.0010f, 0},
    {64, 16, kStage, 1024, 1, 2.21f, 0.2259f, 0.0001f, 0.0007f, 0},  // 4 groups of waves
    {64, 32, kStage, 1024, 1, 2.76f, 0.2677f, 0.2120f, 0.0009f, 0},  // 4
    {64, 64, kStage, 1024, 1, 3.65f, 0.3461f, 0.2914f, 0.0013f, 0},  // 4
    {128, 64, kStage, 768, 1, 3.87f, 0.5498f, 0.4785f, 0.0014f, 0},  // 3
    {128, 128, kStage, 512, 1, 5.22f, 0.8902f, 0.6110f, 0.0022f, 0},  // 2
    {256, 256, kStage, 512, 1, 6.47f, 2.7515f, 2.7968f, 0.0013f, 0},
    {64, 32, kLoose, 1024, 1, 2.23f, 0.3020f, 0.2638f, 0.0004f, 0.0024f},  // 4
    {64, 64, kLoose, 1024, 1, 3.33f, 0.4104f, 0.2865f, 0.0007f, 0.0036f},  // 4
    {128, 128, kLoose, 512, 1, 5.50f, 1.0149f, 0.3523f, 0.0015f, 0.0049f},  // 2
    {256, 128, kLoose, 512, 1, 4.43f, 1.6052f, 1.4308f, 0.0029f, 0.0065f},
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

// Rows and tokens of a shape's tile.
int64_t tile_rows(const I4Shape& s, int group) { return s.kind == kSlice && s.bw == 64 && group == 32 ? 32 : s.bw; }
int64_t tile_tokens(const I4Shape& s, const I4Args& a, int group) { return s.bb == 256 && (a.offset || group == 32) ? 192 : s.bb; }

// Whether a launch holds the shape's workgroups, as their launchers check it
// (check_launch; the stream's workgroups take many tiles each).  What is past it,
// from 2^27 rows on, is left to shapes of larger or fewer tiles, and to the direct
// kernel.
bool launch_holds(const I4Shape& s, const I4Args& a, int group) {
  if (s.kind == kStream) return true;
  const double nw = double((a.rows + tile_rows(s, group) - 1) / tile_rows(s, group) + kXcds);
  const double nb = double((a.batch + tile_tokens(s, a, group) - 1) / tile_tokens(s, a, group));
  return (nw * nb + kXcds) * s.threads < 4294967296.0;
}

// What a product takes on a shape, in us: 1.6 for the launch, then rounds of
// workgroups.  Each round costs `start` (first loads, epilogue), `lead` (or
// `loose`, where the rows of X are off 16-byte boundaries) per token and block
// of 128 columns that a workgroup reads, and `alone` per block where it waits on
// its own loads; a compute unit needs `shared` per block and workgroup it holds;
// and the operands' bytes come at 5.4 TB/s.  The three limits of the loop add as
// fourth powers (the largest rules, a near second counts).
// The constants were fitted to the shapes' times on 3000 sizes over 1..4096 x
// 64..28672 x 64..14336 (three of ten with the rows and columns of eight usual
// matrices, the others drawn), all groups, forms and types of scales, half of them
// with rows of X off 16 bytes, each on 3 to 8 rotated operand sets.  Only their
// order counts: the times themselves are up to a quarter off.  On 2590 other sizes,
// all drawn, the choice takes 1.03 of the best shape's time in the mean, 95 of 100
// under 1.21, the worst 2.3 (on those of the fit 1.03, 1.17 and 2.8); without any
// one of the shapes the best would be up to 2.7 percent slower in the mean, and 1.1
// to 2.6 times in single sizes.  The stream's workgroups stay and take tile after
// tile, which `rounds` says badly: 4 tokens of 14336 x 4096 go to it (10.3 us, the
// token kernel 8.9), 16 of 28672 x 4096 not (slices 26.5, the stream 22.4).
float expected_us(const I4Shape& s, const I4Args& a, int group, bool aligned) {
  const float blocks = float((a.cols + 127) / 128);
  const int64_t bw = tile_rows(s, group), bb = tile_tokens(s, a, group);
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
    if (!shape_ok(a, group, i) || !launch_holds(kShapeList[i], a, group)) continue;
    // one shape for up to 4 tokens is always among the first two kinds, and the others' times are fitted to more tokens
    // (with all of them 1.05 of the best in the mean there, the worst 2.6; so 1.03 and 1.4)
    if (a.batch <= 4 && kShapeList[i].kind != kToken && kShapeList[i].kind != kStream) continue;
    // a slice for each 16 tokens reads the weights as often: not past a few of them.  (Where rows are few and off 16 bytes
    // this loses: 81 to 256 such tokens take 1.12 of the best shape's time in the mean, up to 2.3; of all sizes 95 of 100
    // would be under 1.18 without it, the worst 2.1)
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

template <bool OFF, bool YF32, int STEPS>
int run_dequantize(const D4Args& a, hipStream_t s) {
  const int64_t across = tiles_across(a.cols), band = band_rows(across, STEPS), es = a.st == UW_F32 ? 4 : 2;
  if (band == 0) return fail(UW_ERR_UNSUPPORTED, "uw_i4_dequantize: a row wider than a launch holds");
  for (int64_t row0 = 0; row0 < a.rows; row0 += band) {
    D4Args b = a;
    b.rows = std::min(band, a.rows - row0);
    b.across = uint32_t(across);
    b.Q += row0 * a.ldq;
    b.scale += row0 * es;
    if (OFF) b.offset += row0 * es;
    b.Y += row0 * a.ldy * (YF32 ? 4 : 2);
    hipLaunchKernelGGL((dequantize4_kernel<OFF, YF32, STEPS>), dim3(tiles_of(b.rows, across, STEPS)), dim3(256), 0, s, b);
    if (int rc = hip_check(hipGetLastError(), "dequantize4_kernel launch")) return rc;
  }
  return UW_OK;
}
template <bool OFF, bool YF32>
int run_dequantize_tiles(const D4Args& a, hipStream_t s) {
  return tall_tiles(a.rows, a.cols) ? run_dequantize<OFF, YF32, 4>(a, s) : run_dequantize<OFF, YF32, 2>(a, s);
}

int launch_i4_dequantize(const uint8_t* Q, int64_t rows, int64_t cols, int64_t ldq, int group, const void* scale, int64_t lds,
                         const void* offset, int64_t ldo, int st, void* Y, int64_t ldy, int yt, void* stream) {
  const D4Args a{Q, static_cast<const char*>(scale), static_cast<const char*>(offset), static_cast<char*>(Y), rows, cols, ldq,
                 lds, ldo, ldy, st, group == 32 ? 5 : group == 64 ? 6 : 7, 0};
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (offset) return yt == UW_F32 ? run_dequantize_tiles<true, true>(a, s) : run_dequantize_tiles<true, false>(a, s);
  return yt == UW_F32 ? run_dequantize_tiles<false, true>(a, s) : run_dequantize_tiles<false, false>(a, s);
}

}  // namespace uw
