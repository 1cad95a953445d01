// The product with weights in 4-bit integers (uw_i4.hip says how they lie): the
// kernels, and their launcher for a group of G columns, which the uw_i4_g*.hip
// files instantiate.
//
//   Y[b, n] = sum_g s[g, n] (sum_k q[n, k] X[b, k]) + m[g, n] (sum_k X[b, k]) (+ bias[n])
//
// A weight's integer becomes bf16 exactly, its product with a bf16 activation is
// exact too, and the matrix cores add a group's products in fp32; the sum is
// scaled and added in fp32.  Nothing is rounded to fewer bits before Y.
// The decoding decides how far the products are from the matrix cores' rate, or
// the weights from memory's.  Two ways:
//   decode_u8  u = q + 8 as an 8-bit float code (e4m3: the codes 0 .. 15 stand for
//     0 .. 15 times 2^-9), converted two at a time: 9 operations per 8 weights;
//     the sum starts from -8 times the group's sum of activations, a product more
//     per 16 tokens, and ends as sum q x.  All kernels but i4_stage_kernel.
//   decode_q8  q / 16 from v_cvt_off_f32_i4 and a packing: 15 operations, and no
//     sum of activations but where there are offsets.  i4_stage_kernel, whose
//     waves would each form the sums of up to 256 tokens.
// Sums are kept in 2^-11 of their value with the first (so that -8 x and u x of
// 128 finite activations stay in the fp32 range: 15 * 128 * 2^-11 < 1), in 1 / 16
// with the second (a group's |x| may add up to 2^129), and take it back at the
// end; powers of two, so no result is rounded otherwise down to 2^-115, where its
// sum reaches fp32's denormals.
// With A = 16 activation rows and B = 16 weight rows, lane (r = lane % 16, q =
// lane / 16) holds 8 consecutive k of row r, and of the result weight row r for
// activation rows 4 q .. 4 q + 3: one scale per lane and tile.
#pragma once

#include <algorithm>

#include "uw_i4.h"

namespace uw {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x4 load16_any(const void* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// q / 16 of eight nibbles q + 8, in bf16, in order: 15 operations.  The odd
// nibbles' word is kept apart, so that the conversions take their bytes from
// the two words by themselves instead of shifting each (19 operations).
__device__ __forceinline__ bf16x8 decode_q8(uint32_t w) {
  w ^= 0x88888888u;  // two's complement
  uint32_t h = w >> 4;
  asm("" : "+v"(h));
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = pack_bf16(__builtin_amdgcn_cvt_off_f32_i4(int(w >> (8 * i) & 255u)), __builtin_amdgcn_cvt_off_f32_i4(int(h >> (8 * i) & 255u)));
  return __builtin_bit_cast(bf16x8, v);
}

// u 2^-11 of eight nibbles u, in bf16, in order: 9 operations.
__device__ __forceinline__ bf16x8 decode_u8(uint32_t w) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = w >> 4 & 0x0F0F0F0Fu;
  const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400u), hi = __builtin_amdgcn_perm(odd, even, 0x07030602u);
  const bf16x2_t v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 0.25f, false), v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 0.25f, true);
  const bf16x2_t v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 0.25f, false), v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 0.25f, true);
  return bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// Values [k, k + 8) of a row of n bf16 values; those past the end read as zero
// and are not touched.
__device__ __forceinline__ u32x4 load_x8(const uint16_t* row, int64_t k, int64_t n) {
  if (k + 8 <= n) return load16_any(row + k);
  uint32_t e[7];
#pragma unroll
  for (int i = 0; i < 7; ++i) e[i] = k + i < n ? row[k + i] : 0u;
  return u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6]};
}

__device__ __forceinline__ f32x4 mfma_bf16(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// The 4 x 4 transposition of 32-bit words over the wave's four rows of 16
// lanes: word i of lane (r, q) becomes word q of lane (r, i).
__device__ __forceinline__ void transpose4(u32x4& v) {
  // rows 1 and 3 of the first against rows 0 and 2 of the second, then the halves
  auto a = __builtin_amdgcn_permlane16_swap(v.x, v.y, false, false);
  auto b = __builtin_amdgcn_permlane16_swap(v.z, v.w, false, false);
  auto c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
  v = u32x4{c[0], d[0], c[1], d[1]};
}

__device__ __forceinline__ void store_y(const I4Args& a, int64_t b, int64_t n, float v) {
  if (b >= a.batch || n >= a.rows) return;
  if (a.yt == UW_F32) reinterpret_cast<float*>(a.Y)[b * a.ldy + n] = v;
  else reinterpret_cast<__bf16*>(a.Y)[b * a.ldy + n] = static_cast<__bf16>(v);
}

// Eight times -8 in 2^-11, whose product with the activations is what the sums start from.
__device__ __forceinline__ bf16x8 minus_eights() {
  constexpr uint32_t k = 0xBB80BB80u;
  return __builtin_bit_cast(bf16x8, u32x4{k, k, k, k});
}

// An offset against -8 sum x.
__device__ __forceinline__ float against_eights(float m) { return m * -0.125f; }

// A result from its sum in 1 / UNIT, the bias added in a rounding of its own.
constexpr int kFewUnit = 2048, kStageUnit = 16;
template <int UNIT>
__device__ __forceinline__ float finish(float acc, bool biased, float bias) {
#pragma clang fp contract(off)
  const float v = acc * float(UNIT);
  return biased ? v + bias : v;
}
// The same for four tokens of weight row n.  The bias is loaded and used under
// one branch: a value that outlives it would be waited for, and the loads in flight
// with it, where there is no bias too (i4_stream_kernel, 4 tokens of 14336 x 4096:
// 11.4 us against 10.5).
__device__ __forceinline__ void finish4(const I4Args& a, int64_t n, f32x4& v) {
#pragma clang fp contract(off)
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] *= float(kFewUnit);
  if (a.bias) {
    const float bias = a.bias[n];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += bias;
  }
}

// A workgroup holds 16 weight rows and 16 activation rows; its KS waves split
// k: wave w takes the blocks of 128 columns w, w + KS, ... and the partial
// tiles are summed in LDS, wave by wave.  Everything is read straight from
// global memory; activation rows may start at any element.  With 64-bit offsets:
// what the other kernels do not reach comes here (one token of 14336 x 4096: 18.5
// us, 16 24.7, 4096 4312: the loads' latency, block after block).
template <int G, bool OFF>
__global__ __launch_bounds__(512) void i4_direct_kernel(I4Args a, int n_groups, int ny, int KS) {
  const int L = int(blockIdx.x);
  const int grp = (L / (kXcds * ny)) * kXcds + L % kXcds;
  const int y = (L / kXcds) % ny;
  if (grp >= n_groups) return;  // whole workgroups
  const int lane = int(threadIdx.x) % kWave, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int r = lane % 16, q = lane / 16;
  const int64_t n = int64_t(grp) * 16 + r, n_in = std::min<int64_t>(n, a.rows - 1);
  const int64_t b0 = int64_t(y) * 16;
  const uint8_t* wr = a.W + n_in * a.ldw;
  const uint16_t* xr = a.X + std::min<int64_t>(b0 + r, a.batch - 1) * a.ldx;
  const int64_t last = (a.cols - 1) / 32;  // the rows' last 16-byte word
  const int64_t n_blocks = (a.cols + 127) / 128;
  const bf16x8 eights = minus_eights();
  const f32x4 zero{0.f, 0.f, 0.f, 0.f};
  f32x4 acc = zero;
  for (int64_t kb = wave; kb < n_blocks; kb += KS) {
    const int64_t k0 = kb * 128;
    u32x4 w = load16_any(wr + 16 * std::min<int64_t>(4 * kb + q, last));
    transpose4(w);  // word s: columns k0 + 32 s + 8 q and on
#pragma unroll
    for (int g = 0; g < 128 / G; ++g) {
      if (k0 + g * G >= a.cols) break;
      bf16x8 x[G / 32];
      f32x4 sum = zero;
#pragma unroll
      for (int s = 0; s < G / 32; ++s) {
        x[s] = __builtin_bit_cast(bf16x8, load_x8(xr, k0 + g * G + 32 * s + 8 * q, a.cols));
        sum = mfma_bf16(x[s], eights, sum);
      }
      f32x4 part = sum;
#pragma unroll
      for (int s = 0; s < G / 32; ++s) part = mfma_bf16(x[s], decode_u8(w[g * (G / 32) + s]), part);
      const int64_t at = k0 / G + g;
      const float sc = load_scale(a.scale, at * a.lds + n_in, a.st);
      const float m = OFF ? against_eights(load_scale(a.offset, at * a.ldo + n_in, a.st)) : 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[e] = fmaf(sc, part[e], acc[e]);
        if (OFF) acc[e] = fmaf(m, sum[e], acc[e]);
      }
    }
  }
  st128(uint32_t(wave * 1024 + 16 * lane), __builtin_bit_cast(uint4, acc));
  __syncthreads();
  if (wave) return;
  for (int w = 1; w < KS; ++w) {
    const f32x4 other = __builtin_bit_cast(f32x4, ld128(uint32_t(w * 1024 + 16 * lane)));
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += other[e];
  }
  const float bias = a.bias ? a.bias[n_in] : 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) store_y(a, b0 + 4 * q + e, n, finish<kFewUnit>(acc[e], a.bias, bias));
}

// A buffer over an operand: addresses in it are 32-bit offsets, of which the
// part that a wave shares stays in a scalar register; nothing past `bytes` is
// read (it reads as zero).  The values are the same in every lane;
// readfirstlane keeps them in scalar registers.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_over(const void* p, int64_t bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(v)), hi = __builtin_amdgcn_readfirstlane(uint32_t(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uint64_t(hi) << 32 | lo), int16_t(0),
                                           __builtin_amdgcn_readfirstlane(int(bytes)), 0x00020000);
}

__device__ __forceinline__ u32x4 buffer_load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, int(voff), int(soff), 0);
}

// Scales and offsets of the rows from row0 on (S32: fp32, else bf16), loaded as
// they lie in memory: apart from their value, so that a load is not waited for
// before it is used.
template <bool S32>
struct GroupRows {
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t step;  // bytes between groups
  static constexpr int kShift = S32 ? 2 : 1;

  __device__ __forceinline__ GroupRows(const char* p, int64_t ld, int64_t groups, int64_t rows, int64_t row0) {
    step = __builtin_amdgcn_readfirstlane(uint32_t(ld << kShift));
    rsrc = buffer_over(p + (row0 << kShift), ((groups - 1) * ld + rows - row0) << kShift);
  }
  // group g (of the wave), row `row` (of the lane) + base (of the wave)
  __device__ __forceinline__ uint32_t load(uint32_t g, uint32_t row, uint32_t base = 0) const {
    const int voff = int(row << kShift), soff = int(__builtin_amdgcn_readfirstlane(g * step + (base << kShift)));
    if (S32) return uint32_t(__builtin_amdgcn_raw_buffer_load_b32(rsrc, voff, soff, 0));
    return uint16_t(__builtin_amdgcn_raw_buffer_load_b16(rsrc, voff, soff, 0));
  }
  __device__ __forceinline__ static float value(uint32_t raw) { return bits_f32(S32 ? raw : raw << 16); }
};

// Few tokens: bound by the weights' read.  A workgroup holds 16 WI weight rows
// and 16 BJ activation rows, and its KW waves split k: wave w takes the blocks
// of 128 columns w, w + KW, ...  A wave keeps D blocks in flight in registers
// (weights, activations and scales), each refilled as soon as it is used, and
// meets the others only to add the partial tiles at the end.
// Loads of blocks that are not there are made all the same, from one address:
// where a load hangs on a branch, the wait for an older one becomes a wait for
// all.  A last block that is not whole comes at the end, by itself.
// 16 tokens of 14336 x 4096 take 12.4 us with 64 weight rows, 77 of 1000 x 4100
// 8.3 with 32: the first loads' latency, then the decoding.
template <int G, bool OFF, bool S32, int WI, int BJ, int KW, int D>
__global__ __launch_bounds__(64 * KW) void i4_slice_kernel(I4Args a, int nw_tiles, int nb_tiles) {
  constexpr int GB = 128 / G;  // groups of a block
  // the batch tiles of one weight tile run back to back on one XCD
  const int id = int(blockIdx.x);
  const int wt = (id / (kXcds * nb_tiles)) * kXcds + id % kXcds, y = (id / kXcds) % nb_tiles;
  if (wt >= nw_tiles) return;  // whole workgroups
  const int64_t row0 = int64_t(wt) * 16 * WI, b0 = int64_t(y) * 16 * BJ;
  const int lane = int(threadIdx.x) % kWave, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int r = lane % 16, q = lane / 16;
  const uint32_t wlast = uint32_t(std::min<int64_t>(16 * WI, a.rows - row0)) - 1;  // rows past the last are that row again
  const auto wbuf = buffer_over(a.W + row0 * a.ldw, int64_t(wlast) * a.ldw + (a.cols + 31) / 32 * 16);
  const uint32_t groups = uint32_t((a.cols + G - 1) / G);
  const GroupRows<S32> scale(a.scale, a.lds, groups, a.rows, row0), offset(OFF ? a.offset : a.scale, OFF ? a.ldo : a.lds, groups, a.rows, row0);
  uint32_t wr[WI], wvo[WI];
#pragma unroll
  for (int i = 0; i < WI; ++i) {
    wr[i] = min(uint32_t(16 * i + r), wlast);
    wvo[i] = wr[i] * uint32_t(a.ldw) + 16 * q;
  }
  // G = 128: lane (r, q) holds columns 32 q and on; else, transposed, 8 q and on of each 32
  constexpr int kStep = G == 128 ? 8 : 32;
  const char* xt = reinterpret_cast<const char*>(a.X + b0 * a.ldx);
  uint32_t xvo[BJ];
#pragma unroll
  for (int j = 0; j < BJ; ++j)  // tokens past the last are that token again, into results that are not written
    xvo[j] = 2 * (uint32_t(std::min<int64_t>(16 * j + r, a.batch - b0 - 1)) * uint32_t(a.ldx) + uint32_t(G == 128 ? 32 * q : 8 * q));
  const int nfull = int(a.cols / 128), n = (nfull - wave + KW - 1) / KW;  // this wave's whole blocks
  struct Block {
    u32x4 w[WI], x[BJ][4];
    uint32_t s[WI][GB], m[WI][GB];
  };
  Block ring[D];
  auto load_weights = [&](Block& b, int kb) {
#pragma unroll
    for (int t = 0; t < WI; ++t) b.w[t] = buffer_load16(wbuf, wvo[t], uint32_t(kb) * 64);
#pragma unroll
    for (int g = 0; g < GB; ++g) {
      const uint32_t gi = min(uint32_t(kb * GB + g), groups - 1);
#pragma unroll
      for (int t = 0; t < WI; ++t) {
        b.s[t][g] = scale.load(gi, wr[t]);
        if (OFF) b.m[t][g] = offset.load(gi, wr[t]);
      }
    }
  };
  auto load = [&](Block& b, int i) {
    const int kb = i < n ? wave + KW * i : 0;
    const char* at = xt + int64_t(kb) * 256;
#pragma unroll
    for (int j = 0; j < BJ; ++j)
#pragma unroll
      for (int s = 0; s < 4; ++s) b.x[j][s] = load16_any(at + (xvo[j] + 2 * kStep * s));
    load_weights(b, kb);
  };
  const bf16x8 eights = minus_eights();
  const f32x4 zero{0.f, 0.f, 0.f, 0.f};
  f32x4 acc[WI][BJ];
#pragma unroll
  for (int i = 0; i < WI; ++i)
#pragma unroll
    for (int j = 0; j < BJ; ++j) acc[i][j] = zero;
  auto multiply = [&](Block& b) {
    if (G != 128) {
#pragma unroll
      for (int i = 0; i < WI; ++i) transpose4(b.w[i]);
    }
#pragma unroll
    for (int g = 0; g < GB; ++g) {
      f32x4 part[WI][BJ], sum[BJ];
#pragma unroll
      for (int s = 0; s < 4 / GB; ++s)
#pragma unroll
        for (int j = 0; j < BJ; ++j) sum[j] = mfma_bf16(__builtin_bit_cast(bf16x8, b.x[j][g * (4 / GB) + s]), eights, s ? sum[j] : zero);
#pragma unroll
      for (int s = 0; s < 4 / GB; ++s) {
        const int at = g * (4 / GB) + s;
#pragma unroll
        for (int i = 0; i < WI; ++i) {
          const bf16x8 w = decode_u8(b.w[i][at]);
#pragma unroll
          for (int j = 0; j < BJ; ++j) part[i][j] = mfma_bf16(__builtin_bit_cast(bf16x8, b.x[j][at]), w, s ? part[i][j] : sum[j]);
        }
      }
#pragma unroll
      for (int i = 0; i < WI; ++i) {
        const float sc = scale.value(b.s[i][g]), m = OFF ? against_eights(offset.value(b.m[i][g])) : 0.f;
#pragma unroll
        for (int j = 0; j < BJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[i][j][e] = fmaf(sc, part[i][j][e], acc[i][j][e]);
            if (OFF) acc[i][j][e] = fmaf(m, sum[j][e], acc[i][j][e]);
          }
      }
    }
  };
  if (n > 0) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      load(ring[d], d);
      __builtin_amdgcn_sched_barrier(0);  // in this order, which the waits count on
    }
    int i = 0;
#pragma unroll 1
    for (; i + 2 * D <= n; i += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        multiply(ring[d]);
        load(ring[d], i + d + D);
      }
    }
    // the last blocks, up to 2 D - 1
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (i + d < n) multiply(ring[d]);
      if (i + d + D < n) load(ring[d], i + d + D);
    }
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
      if (i + d + D < n) multiply(ring[d]);
  }
  if (nfull * 128 < a.cols && nfull % KW == wave) {
    Block b;
    load_weights(b, nfull);
#pragma unroll
    for (int j = 0; j < BJ; ++j) {
      const uint16_t* row = a.X + std::min<int64_t>(b0 + 16 * j + r, a.batch - 1) * a.ldx;
#pragma unroll
      for (int s = 0; s < 4; ++s) b.x[j][s] = load_x8(row, int64_t(nfull) * 128 + (G == 128 ? 32 * q : 8 * q) + kStep * s, a.cols);
    }
    multiply(b);
  }
  // partial tile (i, j) of wave w at (w WI BJ + i BJ + j) KB
#pragma unroll
  for (int i = 0; i < WI; ++i)
#pragma unroll
    for (int j = 0; j < BJ; ++j)
      if (b0 + 16 * j + 4 * q < a.batch)
        st128(uint32_t(((wave * WI + i) * BJ + j) * 1024 + 16 * lane), __builtin_bit_cast(uint4, acc[i][j]));
  __syncthreads();
  for (int t = wave; t < WI * BJ; t += KW) {
    const int64_t b = b0 + 16 * (t % BJ) + 4 * q, nn = row0 + 16 * (t / BJ) + r;
    if (b >= a.batch || nn >= a.rows) continue;
    f32x4 total = zero;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const f32x4 v = __builtin_bit_cast(f32x4, ld128(uint32_t((w * WI * BJ + t) * 1024 + 16 * lane)));
#pragma unroll
      for (int e = 0; e < 4; ++e) total[e] += v[e];
    }
    finish4(a, nn, total);
#pragma unroll
    for (int e = 0; e < 4; ++e) store_y(a, b + e, nn, total[e]);
  }
}

// Up to NB = 1 or 4 tokens.  As the slices, with WI tiles of 16 weight rows per
// workgroup, but a block's activations are 256 bytes per token: one 4-byte load
// of the wave (in the operand's layout it would be four of 16 bytes, most of
// them for tokens that are not there), put in order by the wave's own corner of
// LDS.  One token of 14336 x 4096 takes 8.0 us with 32 weight rows, 3.8 TB/s of
// weights and scales (a plain read of them 5.6 to 6.6 us with its launch), of
// 4096 x 14336 7.6 with 16: bound by the one round of loads that a workgroup
// makes, and the launch.
template <int G, bool OFF, bool S32, int WI, int NB, int KW, int D>
__global__ __launch_bounds__(64 * KW) void i4_token_kernel(I4Args a, int nw_tiles) {
  constexpr int GB = 128 / G;       // groups of a block
  constexpr uint32_t kRow = 272;    // a token's 256 bytes, 16 further into the banks than the one before
  // workgroups are dealt to the XCDs round-robin: each XCD takes a run of tiles, since the scales of 16 rows are 32 bytes
  // of a group and neighbours on other XCDs would fetch the rest of the line again (one token of 14336 x 4096: 8.4 -> 8.1
  // us, of 4096 x 14336 8.1 -> 7.6; no gain for the slices, whose time has more to it)
  const int xcd = int(blockIdx.x) % kXcds;
  const int wt = xcd * (nw_tiles / kXcds) + min(xcd, nw_tiles % kXcds) + int(blockIdx.x) / kXcds;
  const int64_t row0 = int64_t(wt) * 16 * WI;
  const int lane = int(threadIdx.x) % kWave, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int r = lane % 16, q = lane / 16, batch = int(a.batch);
  const uint32_t wlast = uint32_t(std::min<int64_t>(16 * WI, a.rows - row0)) - 1;  // rows past the last are that row again
  const auto wbuf = buffer_over(a.W + row0 * a.ldw, int64_t(wlast) * a.ldw + (a.cols + 31) / 32 * 16);
  const uint32_t groups = uint32_t((a.cols + G - 1) / G);
  const GroupRows<S32> scale(a.scale, a.lds, groups, a.rows, row0), offset(OFF ? a.offset : a.scale, OFF ? a.ldo : a.lds, groups, a.rows, row0);
  uint32_t wr[WI], wvo[WI];
#pragma unroll
  for (int i = 0; i < WI; ++i) {
    wr[i] = min(uint32_t(16 * i + r), wlast);
    wvo[i] = wr[i] * uint32_t(a.ldw) + 16 * q;
  }
  const int nfull = int(a.cols / 128), n = (nfull - wave + KW - 1) / KW;  // this wave's whole blocks
  struct Block {
    u32x4 w[WI];
    uint32_t x[NB], s[WI][GB], m[WI][GB];
  };
  Block ring[D];
  auto load_weights = [&](Block& b, int kb) {
#pragma unroll
    for (int t = 0; t < WI; ++t) b.w[t] = buffer_load16(wbuf, wvo[t], uint32_t(kb) * 64);
#pragma unroll
    for (int g = 0; g < GB; ++g) {
      const uint32_t gi = min(uint32_t(kb * GB + g), groups - 1);
#pragma unroll
      for (int t = 0; t < WI; ++t) {
        b.s[t][g] = scale.load(gi, wr[t]);
        if (OFF) b.m[t][g] = offset.load(gi, wr[t]);
      }
    }
  };
  auto load = [&](Block& b, int i) {
    const int kb = i < n ? wave + KW * i : 0;
#pragma unroll
    for (int t = 0; t < NB; ++t) {
      const char* at = reinterpret_cast<const char*>(a.X + int64_t(min(t, batch - 1)) * a.ldx) + int64_t(kb) * 256;
      __builtin_memcpy(&b.x[t], at + 4 * lane, 4);
    }
    load_weights(b, kb);
  };
  const uint32_t corner = uint32_t(wave) * (NB * kRow);
  const uint32_t xat = corner + uint32_t(min(r, NB - 1)) * kRow + (G == 128 ? 64 * q : 16 * q);
  constexpr uint32_t kStep = G == 128 ? 16 : 64;  // lane (r, q) holds columns 32 q and on; else, transposed, 8 q and on of each 32
  const bf16x8 eights = minus_eights();
  const f32x4 zero{0.f, 0.f, 0.f, 0.f};
  f32x4 acc[WI];
#pragma unroll
  for (int i = 0; i < WI; ++i) acc[i] = zero;
  auto multiply = [&](Block& b) {
    bf16x8 x[4];
#pragma unroll
    for (int t = 0; t < NB; ++t) st32(corner + uint32_t(t) * kRow + 4 * lane, b.x[t]);
    wave_lds_fence();
#pragma unroll
    for (int s = 0; s < 4; ++s) x[s] = __builtin_bit_cast(bf16x8, ld128(xat + kStep * s));
    wave_lds_fence();
    if (G != 128) {
#pragma unroll
      for (int i = 0; i < WI; ++i) transpose4(b.w[i]);
    }
#pragma unroll
    for (int g = 0; g < GB; ++g) {
      f32x4 part[WI], sum = zero;
#pragma unroll
      for (int s = 0; s < 4 / GB; ++s) sum = mfma_bf16(x[g * (4 / GB) + s], eights, sum);
#pragma unroll
      for (int s = 0; s < 4 / GB; ++s)
#pragma unroll
        for (int i = 0; i < WI; ++i) part[i] = mfma_bf16(x[g * (4 / GB) + s], decode_u8(b.w[i][g * (4 / GB) + s]), s ? part[i] : sum);
#pragma unroll
      for (int i = 0; i < WI; ++i) {
        const float sc = scale.value(b.s[i][g]), m = OFF ? against_eights(offset.value(b.m[i][g])) : 0.f;
#pragma unroll
        for (int e = 0; e < NB; ++e) {  // of the lanes q = 0, the others' tokens are not there
          acc[i][e] = fmaf(sc, part[i][e], acc[i][e]);
          if (OFF) acc[i][e] = fmaf(m, sum[e], acc[i][e]);
        }
      }
    }
  };
  if (n > 0) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      load(ring[d], d);
      __builtin_amdgcn_sched_barrier(0);  // in this order, which the waits count on
    }
    int i = 0;
#pragma unroll 1
    for (; i + 2 * D <= n; i += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        multiply(ring[d]);
        load(ring[d], i + d + D);
      }
    }
    // the last blocks, up to 2 D - 1
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (i + d < n) multiply(ring[d]);
      if (i + d + D < n) load(ring[d], i + d + D);
    }
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
      if (i + d + D < n) multiply(ring[d]);
  }
  if (nfull * 128 < a.cols && nfull % KW == wave) {
    Block b;
    load_weights(b, nfull);
    const int64_t k = int64_t(nfull) * 128 + 2 * lane;
#pragma unroll
    for (int t = 0; t < NB; ++t) {
      const uint16_t* row = a.X + int64_t(min(t, batch - 1)) * a.ldx;
      b.x[t] = k < a.cols ? row[k] : 0u;
      if (k + 1 < a.cols) b.x[t] |= uint32_t(row[k + 1]) << 16;
    }
    multiply(b);
  }
  // of tile i, wave w's sums at (w WI + i) 256 bytes
  __syncthreads();  // the corners are done with
#pragma unroll
  for (int i = 0; i < WI; ++i)
    if (q == 0) st128(uint32_t((wave * WI + i) * 256 + 16 * r), __builtin_bit_cast(uint4, acc[i]));
  __syncthreads();
  for (int t = wave; t < WI; t += KW) {
    const int64_t nn = row0 + 16 * t + r;
    if (q || nn >= a.rows) continue;
    f32x4 total = zero;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const f32x4 v = __builtin_bit_cast(f32x4, ld128(uint32_t((w * WI + t) * 256 + 16 * r)));
#pragma unroll
      for (int e = 0; e < NB; ++e) total[e] += v[e];
    }
    finish4(a, nn, total);
#pragma unroll
    for (int e = 0; e < NB; ++e) store_y(a, e, nn, total[e]);
  }
}

// The fewest tokens (at most 16, whose activations fit in LDS): bound by the
// weights' read, which has to run on without a pause.  A workgroup stays on its
// compute unit and takes the tiles of 16 weight rows blockIdx, blockIdx + grid,
// ...  It puts the activations into LDS once.  Of every tile, wave w takes the
// blocks of 128 columns w, w + KW, ..., with D of them in flight in registers,
// those of the next tiles among them (and, as above, loads that are made
// whether there is a block or not); at a tile's end the waves put their sums
// into LDS, and one of them adds them up while the others go on.
// An activation row starts 16 bytes further into the banks than the one before
// it; lanes of tokens that are not there read the last one's again, into
// results that are not written.
// 28672 x 4096 with 16 tokens, groups of 64 with offsets: 22.4 us, the slices 26.5;
// 14336 x 4096 with 4 tokens: 10.3 (the token kernel 8.9).
// LDS: activations; the waves' sums of two tiles, of the tokens that are there.
template <int G, bool OFF, bool S32, int KW, int D, int U>
__global__ __launch_bounds__(64 * KW) void i4_stream_kernel(I4Args a, int n_tiles, uint32_t pitch) {
  constexpr int GB = 128 / G;  // groups of a block
  const int lane = int(threadIdx.x) % kWave, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int r = lane % 16, q = lane / 16, batch = int(a.batch);
  const int nkb = int((a.cols + 127) / 128), n = (nkb - wave + KW - 1) / KW;  // this wave's blocks of a tile
  const int grid = int(gridDim.x), tiles = (n_tiles - int(blockIdx.x) + grid - 1) / grid;
  const uint32_t groups = uint32_t((a.cols + G - 1) / G);
  const uint32_t parts = uint32_t(batch) * pitch;
  const uint32_t part_bytes = uint32_t((batch + 3) / 4) * 256;  // of a wave
  // the activations' whole chunks of 8 columns, U steps of the workgroup's threads at a time: step (row b, part c) by step
  constexpr int T = 64 * KW;
  const int full = int(a.cols / 8), per = (full + T - 1) / T;
  int xb = 0, xc = 0, sb = 0, sc = 0;
  u32x4 xv[U];
  auto load_x = [&]() {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      xv[u] = load16_any(reinterpret_cast<const char*>(a.X + int64_t(xb) * a.ldx) + uint32_t(16 * min(xc * T + int(threadIdx.x), full - 1)));
      const bool row = xc + 1 == per;
      xc = row ? 0 : xc + 1;
      xb = min(xb + (row ? 1 : 0), batch - 1);
    }
  };
  auto store_x = [&]() {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = sc * T + int(threadIdx.x);
      if (sb < batch && c < full) st128(uint32_t(sb) * pitch + uint32_t(c) * 16, __builtin_bit_cast(uint4, xv[u]));
      const bool row = sc + 1 == per;
      sc = row ? 0 : sc + 1;
      sb += row ? 1 : 0;
    }
  };
  if (full) load_x();
  // rows past the last are that row again
  const auto wbuf = buffer_over(a.W, (a.rows - 1) * a.ldw + (a.cols + 31) / 32 * 16);
  const GroupRows<S32> scale(a.scale, a.lds, groups, a.rows, 0), offset(OFF ? a.offset : a.scale, OFF ? a.ldo : a.lds, groups, a.rows, 0);
  struct Block {
    u32x4 w;
    uint32_t s[GB], m[GB];
  };
  Block ring[D];
  int lt = int(blockIdx.x), lb = 0, left = tiles * n;  // the next block to load: its tile and place; how many are left
  const int last_row = int(a.rows) - 1;
  auto load = [&](Block& b) {
    const bool there = left > 0;
    const uint32_t kb = there ? uint32_t(wave + KW * lb) : 0u, tile = there ? uint32_t(lt) : 0u;
    const uint32_t row = there ? uint32_t(min(r, last_row - int(tile) * 16)) : 0u;
    b.w = buffer_load16(wbuf, row * uint32_t(a.ldw) + (there ? 16 * q : 0), tile * 16 * uint32_t(a.ldw) + kb * 64);
#pragma unroll
    for (int g = 0; g < GB; ++g) {
      const uint32_t gi = min(kb * GB + g, groups - 1);
      b.s[g] = scale.load(gi, row, tile * 16);
      if (OFF) b.m[g] = offset.load(gi, row, tile * 16);
    }
    --left;
    if (++lb == n) {
      lb = 0;
      lt += grid;
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) {
    load(ring[d]);
    __builtin_amdgcn_sched_barrier(0);  // in this order, which the waits count on
  }
  if (full) {
    store_x();
    while (sb < batch) {
      load_x();
      store_x();
    }
  }
  // behind a row's last whole chunk: its last columns, then zeros
  for (int b = wave; b < batch; b += KW) {
    for (int c = full + lane; c < 16 * nkb; c += kWave)
      st128(uint32_t(b) * pitch + uint32_t(c) * 16,
            __builtin_bit_cast(uint4, 8 * int64_t(c) < a.cols ? load_x8(a.X + int64_t(b) * a.ldx, 8 * int64_t(c), a.cols) : u32x4{0u, 0u, 0u, 0u}));
  }
  lds_barrier();
  const uint32_t xat = uint32_t(min(r, batch - 1)) * pitch;
  // G = 128: lane (r, q) holds columns 32 q and on; else, transposed, 8 q and on of each 32
  auto read_x = [&](int kb, int s) {
    return __builtin_bit_cast(bf16x8, ld128(xat + uint32_t(kb) * 256 + uint32_t(G == 128 ? 4 * q + s : 4 * s + q) * 16));
  };
  const bf16x8 eights = minus_eights();
  const f32x4 zero{0.f, 0.f, 0.f, 0.f};
  f32x4 acc = zero;
  auto multiply = [&](Block& b, int kb) {
    bf16x8 x[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) x[s] = read_x(kb, s);
    if (G != 128) transpose4(b.w);
#pragma unroll
    for (int g = 0; g < GB; ++g) {
      f32x4 sum = zero;
#pragma unroll
      for (int s = 0; s < 4 / GB; ++s) sum = mfma_bf16(x[g * (4 / GB) + s], eights, sum);
      f32x4 part = sum;
#pragma unroll
      for (int s = 0; s < 4 / GB; ++s) part = mfma_bf16(x[g * (4 / GB) + s], decode_u8(b.w[g * (4 / GB) + s]), part);
      const float sc = scale.value(b.s[g]), m = OFF ? against_eights(offset.value(b.m[g])) : 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[e] = fmaf(sc, part[e], acc[e]);
        if (OFF) acc[e] = fmaf(m, sum[e], acc[e]);
      }
    }
  };
  // the end of a tile: every wave's sums, added by one of them
  auto finish_tile = [&](int t) {
    const uint32_t at = parts + uint32_t(t & 1) * (KW * part_bytes);
    if (4 * q < batch) st128(at + uint32_t(wave) * part_bytes + 16 * lane, __builtin_bit_cast(uint4, acc));
    acc = zero;
    lds_barrier();
    const int64_t nn = (int64_t(blockIdx.x) + int64_t(t) * grid) * 16 + r;
    if (wave != t % KW || 4 * q >= batch || nn >= a.rows) return;
    f32x4 total = zero;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const f32x4 v = __builtin_bit_cast(f32x4, ld128(at + uint32_t(w) * part_bytes + 16 * lane));
#pragma unroll
      for (int e = 0; e < 4; ++e) total[e] += v[e];
    }
    finish4(a, nn, total);
#pragma unroll
    for (int e = 0; e < 4; ++e) store_y(a, 4 * q + e, nn, total[e]);
  };
  if (n == 0) {
    for (int t = 0; t < tiles; ++t) finish_tile(t);
    return;
  }
  int t = 0, at = 0;  // the tile and the place of the block at hand
  while (t < tiles) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (t < tiles) {
        multiply(ring[d], wave + KW * at);
        if (++at == n) {
          finish_tile(t);
          at = 0;
          ++t;
        }
      }
      load(ring[d]);
    }
  }
}

// 16 bytes of row b of Y from column n on: 16 / SIZE values.
template <int SIZE>
__device__ __forceinline__ void store_row16(const I4Args& a, int64_t b, int64_t n, const uint4& v) {
  if (b >= a.batch || n >= a.rows) return;
  char* y = a.Y + (b * a.ldy + n) * SIZE;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const int m = int(std::min<int64_t>(16 / SIZE, a.rows - n));
  if (m == 16 / SIZE) {
    __builtin_memcpy(y, w, 16);
    return;
  }
#pragma unroll
  for (int e = 0; e < 16 / SIZE - 1; ++e) {
    if (e >= m) continue;
    if (SIZE == 4) {
      __builtin_memcpy(y + 4 * e, &w[e], 4);
    } else {
      const uint16_t h = uint16_t(w[e / 2] >> (16 * (e & 1)));
      __builtin_memcpy(y + 2 * e, &h, 2);
    }
  }
}

template <int WI>
constexpr int epilogue_bytes = 16 * (16 * WI * 4 + 16);

// Epilogue of a wave's WI x BJ tiles at (n0, b0), through LDS: 16 activation
// rows at a time as the wave's 16 WI columns, so that rows go out in runs of
// 32 WI bytes (bf16) or twice that.  out: the wave's place in LDS,
// epilogue_bytes<WI> that nothing else uses any more.
template <int WI, int BJ, bool YBF16>
__device__ __forceinline__ void store_through_lds(const I4Args& a, int64_t n0, int64_t b0, uint32_t out, int lane,
                                                  const f32x4 (&acc)[WI][BJ]) {
  constexpr int kCols = 16 * WI, kSize = YBF16 ? 2 : 4, kPitch = kCols * kSize + 16;
  const int r = lane % 16, q = lane / 16;
  float bias[WI];
#pragma unroll
  for (int i = 0; i < WI; ++i) bias[i] = a.bias ? a.bias[std::min<int64_t>(n0 + 16 * i + r, a.rows - 1)] : 0.f;
#pragma unroll
  for (int j = 0; j < BJ; ++j) {
#pragma unroll
    for (int i = 0; i < WI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = finish<kStageUnit>(acc[i][j][e], a.bias, bias[i]);
        const uint32_t dst = out + uint32_t(4 * q + e) * kPitch + uint32_t(16 * i + r) * kSize;
        if (YBF16) st16(dst, pack_bf16(v, 0.f));
        else st32(dst, f32_bits(v));
      }
    wave_lds_fence();
    constexpr int kPer = 16 / kSize, kLanes = kCols / kPer;  // values a lane stores; lanes of a row
    constexpr int kChunks = 16 * kLanes;                     // of the 16 rows
#pragma unroll
    for (int c0 = 0; c0 < kChunks; c0 += kWave) {
      const int at = c0 + lane, br = at / kLanes, c = at % kLanes * kPer;
      if (kChunks % kWave == 0 || at < kChunks)
        store_row16<kSize>(a, b0 + 16 * j + br, n0 + c, ld128(out + uint32_t(br) * kPitch + uint32_t(c) * kSize));
    }
    wave_lds_fence();
  }
}

// A tile of an operand as a buffer: `rows` rows of `bytes` bytes (the end of
// the last one rounded up to 4), ld bytes apart; rows past the last are that
// row again.
struct Staged4 {
  __amdgpu_buffer_rsrc_t rsrc;
  int last;

  __device__ __forceinline__ Staged4(const void* tile, int64_t rows, int64_t bytes, int64_t ld, int tile_rows)
      : last(__builtin_amdgcn_readfirstlane(int(std::min<int64_t>(tile_rows, rows)) - 1)) {
    rsrc = buffer_over(tile, int64_t(last) * ld + (bytes + 3) / 4 * 4);
  }
};

// Mask of 8 bf16 values of which the first `left` lie inside their row.
__device__ __forceinline__ u32x4 tail_mask8(int left) {
  u32x4 m;
#pragma unroll
  for (int d = 0; d < 4; ++d) m[d] = left >= 2 * d + 2 ? ~0u : left == 2 * d + 1 ? 0xFFFFu : 0u;
  return m;
}

// Scales (or offsets) of 16 WI rows on their way into LDS: for each of a
// block's groups 16 WI words of 4 bytes, from the word that holds the first
// row's value on (bf16 values need not start at a word).
template <int G, bool S32, int WI>
struct StagedGroups {
  static constexpr int GB = 128 / G, kLanes = 16 * WI, kLoads = (GB * kLanes + 63) / 64;
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t start, step;  // bytes to row0's value of group 0, and between groups
  uint32_t groups, rows;

  __device__ __forceinline__ StagedGroups(const char* p, int64_t ld, uint32_t n, int64_t all_rows, int64_t row0)
      : groups(n), rows(uint32_t(std::min<int64_t>(16 * WI, all_rows - row0))) {
    constexpr int kShift = S32 ? 2 : 1;
    const char* at = p + (row0 << kShift);
    const int64_t in = int64_t(reinterpret_cast<uint64_t>(at) & 3);
    start = __builtin_amdgcn_readfirstlane(uint32_t(in));
    step = __builtin_amdgcn_readfirstlane(uint32_t(ld << kShift));
    rsrc = buffer_over(at - in, (in + (((int64_t(n) - 1) * ld + rows) << kShift) + 3) / 4 * 4);
  }
  __device__ __forceinline__ void issue(int kb, int lane, uint32_t to) const {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int at = u * 64 + lane, g = at / kLanes, d = at % kLanes;
      const uint32_t byte = start + min(uint32_t(kb * GB + g), groups - 1) * step;
      const uint32_t most = ((byte & 3) + (rows << (S32 ? 2 : 1)) - 1) / 4;  // the word of the last row's value
      stage_load4(rsrc, (byte & ~3u) + 4 * min(uint32_t(d), most), 0u, to + u * 256);
    }
  }
  // the value of row `row` in group g of block kb
  __device__ __forceinline__ float value(int kb, int g, uint32_t row, uint32_t from) const {
    const uint32_t at = from + uint32_t(g) * (kLanes * 4);
    row = min(row, rows - 1);
    if (S32) return bits_f32(ld32(at + 4 * row));
    const uint32_t byte = start + min(uint32_t(kb * GB + g), groups - 1) * step;
    return bits_f32(ld16(at + (byte & 3) + 2 * row) << 16);
  }
};

// Where the 16-byte chunks of a staged block lie in LDS.  A 16-byte read serves
// 16 lanes at a time in 64 banks: lanes 0 .. 3, 12 .. 15, 20 .. 27 first, then
// the other 16 of the half.  The products' lane (r, q) reads activation chunk
// 4 q + s (groups of 128) or 4 s + q of row r, weight chunk q of row r: with
// activations' chunks in the order of 4 s + q, against the row's low bits, and
// weights' against minus the row's quarter, every 16 lanes fall on all 64 banks
// (plain c ^ (r % 16) and c ^ (r / 4): two on each, twice the time).
template <int G>
__device__ __forceinline__ int x_order(int c) { return G == 128 ? c % 4 * 4 + c / 4 : c; }  // its own inverse
template <int G>
__device__ __forceinline__ int x_slot(int chunk, int row) { return x_order<G>(chunk) ^ (row % 16); }
template <int G>
__device__ __forceinline__ int x_chunk(int slot, int row) { return x_order<G>(slot ^ (row % 16)); }
__device__ __forceinline__ int w_slot(int chunk, int row) { return chunk ^ (-(row / 4) & 3); }  // its own inverse

// Few tokens, long rows: as the slices, with everything staged by direct loads
// into the wave's own ring of D blocks in LDS, so that many blocks are in
// flight without registers and nothing but the wave's own loads is waited for.
// A block's weights and activations lie in LDS where w_slot and x_slot say.
// 16 tokens of 4096 x 14336, groups of 64 with offsets: 15.5 us (the slices take
// 20.3), 33 MB of weights at 2.1 TB/s.  Each of the 256 workgroups of 16 weight rows
// takes all tokens' whole rows into LDS, 117 MB through the L2s together, four bytes of X
// for one of W; that, and the waves' rounds of load, wait and decode.
template <int G, bool OFF, bool S32, int WI, int BJ, int KW, int D>
__global__ __launch_bounds__(64 * KW) void i4_deep_kernel(I4Args a, int nw_tiles, int nb_tiles) {
  using Groups = StagedGroups<G, S32, WI>;
  constexpr int GB = 128 / G;  // groups of a block
  constexpr int L = 4 * BJ + WI + Groups::kLoads * (OFF ? 2 : 1);
  constexpr uint32_t kX = 4096 * BJ, kW = 1024 * WI, kS = Groups::kLoads * 256, kSlot = kX + kW + kS * (OFF ? 2 : 1);
  static_assert((D - 1) * L < 64, "vmcnt");
  // the batch tiles of one weight tile run back to back on one XCD
  const int id = int(blockIdx.x);
  const int wt = (id / (kXcds * nb_tiles)) * kXcds + id % kXcds, y = (id / kXcds) % nb_tiles;
  if (wt >= nw_tiles) return;  // whole workgroups
  const int64_t row0 = int64_t(wt) * 16 * WI, b0 = int64_t(y) * 16 * BJ;
  const int lane = int(threadIdx.x) % kWave, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int r = lane % 16, q = lane / 16;
  const Staged4 tw(a.W + row0 * a.ldw, a.rows - row0, (a.cols + 31) / 32 * 16, a.ldw, 16 * WI);
  const Staged4 tx(a.X + b0 * a.ldx, a.batch - b0, 2 * a.cols, 2 * a.ldx, 16 * BJ);
  const uint32_t groups = uint32_t((a.cols + G - 1) / G);
  const Groups scale(a.scale, a.lds, groups, a.rows, row0), offset(OFF ? a.offset : a.scale, OFF ? a.ldo : a.lds, groups, a.rows, row0);
  const int nkb = int((a.cols + 127) / 128), n = (nkb - wave + KW - 1) / KW;  // this wave's blocks
  const int wlast = int((a.cols - 1) / 32) % 4, xlast = int((a.cols - 1) / 8) % 16;  // the last block's last chunks
  const int wchunk = w_slot(lane % 4, lane / 4);
  uint32_t wvo[WI], xvo[4 * BJ];
#pragma unroll
  for (int u = 0; u < WI; ++u) wvo[u] = uint32_t(min(16 * u + lane / 4, tw.last)) * uint32_t(a.ldw);
#pragma unroll
  for (int u = 0; u < 4 * BJ; ++u) xvo[u] = uint32_t(min(4 * u + q, tx.last)) * uint32_t(2 * a.ldx);
  const uint32_t ring = uint32_t(wave) * (D * kSlot);
  auto issue = [&](int i, int slot) {
    const int kb = wave + KW * i;
    const uint32_t base = ring + uint32_t(slot) * kSlot;
    const int wmost = kb == nkb - 1 ? wlast : 3, xmost = kb == nkb - 1 ? xlast : 15;
#pragma unroll
    for (int u = 0; u < 4 * BJ; ++u)
      stage_load<false>(tx.rsrc, xvo[u] + 16 * min(x_chunk<G>(r, 4 * (u % 4) + q), xmost), uint32_t(kb) * 256, base + u * 1024);
#pragma unroll
    for (int u = 0; u < WI; ++u) stage_load<false>(tw.rsrc, wvo[u] + 16 * min(wchunk, wmost), uint32_t(kb) * 64, base + kX + u * 1024);
    scale.issue(kb, lane, base + kX + kW);
    if (OFF) offset.issue(kb, lane, base + kX + kW + kS);
  };
  const bf16x8 eights = minus_eights();
  const f32x4 zero{0.f, 0.f, 0.f, 0.f};
  f32x4 acc[WI][BJ];
#pragma unroll
  for (int i = 0; i < WI; ++i)
#pragma unroll
    for (int j = 0; j < BJ; ++j) acc[i][j] = zero;
#pragma unroll
  for (int i = 0; i < D; ++i)
    if (i < n) issue(i, i);
  int slot = 0;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    wait_ring<L, D - 1>(n - 1 - i);  // block i has landed
    const int kb = wave + KW * i;
    const uint32_t base = ring + uint32_t(slot) * kSlot;
    u32x4 w[WI], x[BJ][4];
    float sc[WI][GB], mc[WI][GB];
#pragma unroll
    for (int t = 0; t < WI; ++t) w[t] = __builtin_bit_cast(u32x4, ld128(base + kX + uint32_t(16 * t + r) * 64 + uint32_t(w_slot(q, r)) * 16));
#pragma unroll
    for (int j = 0; j < BJ; ++j)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        x[j][s] = __builtin_bit_cast(u32x4, ld128(base + uint32_t(16 * j + r) * 256 + uint32_t((4 * s + q) ^ r) * 16));
#pragma unroll
    for (int t = 0; t < WI; ++t)
#pragma unroll
      for (int g = 0; g < GB; ++g) {
        sc[t][g] = scale.value(kb, g, 16 * t + r, base + kX + kW);
        mc[t][g] = OFF ? against_eights(offset.value(kb, g, 16 * t + r, base + kX + kW + kS)) : 0.f;
      }
    if (i + D < n) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot's operands are in registers
      issue(i + D, slot);
    }
    if (kb == nkb - 1 && a.cols % 128) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const u32x4 m = tail_mask8(int(a.cols - int64_t(kb) * 128) - 8 * (G == 128 ? 4 * q + s : 4 * s + q));
#pragma unroll
        for (int j = 0; j < BJ; ++j) x[j][s] &= m;
      }
    }
    if (G != 128) {
#pragma unroll
      for (int t = 0; t < WI; ++t) transpose4(w[t]);
    }
#pragma unroll
    for (int g = 0; g < GB; ++g) {
      f32x4 part[WI][BJ], sum[BJ];
#pragma unroll
      for (int s = 0; s < 4 / GB; ++s)
#pragma unroll
        for (int j = 0; j < BJ; ++j) sum[j] = mfma_bf16(__builtin_bit_cast(bf16x8, x[j][g * (4 / GB) + s]), eights, s ? sum[j] : zero);
#pragma unroll
      for (int s = 0; s < 4 / GB; ++s) {
        const int at = g * (4 / GB) + s;
#pragma unroll
        for (int t = 0; t < WI; ++t) {
          const bf16x8 v = decode_u8(w[t][at]);
#pragma unroll
          for (int j = 0; j < BJ; ++j) part[t][j] = mfma_bf16(__builtin_bit_cast(bf16x8, x[j][at]), v, s ? part[t][j] : sum[j]);
        }
      }
#pragma unroll
      for (int t = 0; t < WI; ++t)
#pragma unroll
        for (int j = 0; j < BJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[t][j][e] = fmaf(sc[t][g], part[t][j][e], acc[t][j][e]);
            if (OFF) acc[t][j][e] = fmaf(mc[t][g], sum[j][e], acc[t][j][e]);
          }
    }
    slot = slot + 1 == D ? 0 : slot + 1;
  }
  __syncthreads();  // every wave is done with its ring
  // partial tile (i, j) of wave w at (w WI BJ + i BJ + j) KB
#pragma unroll
  for (int i = 0; i < WI; ++i)
#pragma unroll
    for (int j = 0; j < BJ; ++j)
      if (b0 + 16 * j + 4 * q < a.batch)
        st128(uint32_t(((wave * WI + i) * BJ + j) * 1024 + 16 * lane), __builtin_bit_cast(uint4, acc[i][j]));
  __syncthreads();
  for (int t = wave; t < WI * BJ; t += KW) {
    const int64_t b = b0 + 16 * (t % BJ) + 4 * q, nn = row0 + 16 * (t / BJ) + r;
    if (b >= a.batch || nn >= a.rows) continue;
    f32x4 total = zero;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const f32x4 v = __builtin_bit_cast(f32x4, ld128(uint32_t((w * WI * BJ + t) * 1024 + 16 * lane)));
#pragma unroll
      for (int e = 0; e < 4; ++e) total[e] += v[e];
    }
    finish4(a, nn, total);
#pragma unroll
    for (int e = 0; e < 4; ++e) store_y(a, b + e, nn, total[e]);
  }
}

// Many tokens.  The activations of a block of 128 columns are staged in LDS for
// the whole workgroup, one block ahead of the products: NW waves hold BB = 16 BJ
// activation rows (256 bytes each) by 16 WI weight rows each, as WI x BJ tiles
// of 16 x 16.  A wave decodes its WI x 128 weights of a block into registers
// once and runs them against one tile of tokens after another, so that a group's
// sums live for one tile only.  KG groups of such waves, each with its own two
// stages, take every KG-th block and add their sums in LDS at the end.
//
// A compute unit's matrix cores take 16 cycles a product and let 8 cycles of
// the vector ALU's through beside it, about 4.3 an operation: two operations a
// product go unseen, the third does not.  Decoding takes 15 per 8 weights, which
// BJ tiles share, scaling one per product, so a tall tile of 256 tokens has
// about two; and the decoding is kept beside other waves' products: with up to
// 3 groups a wave reads its packed rows straight into registers, and half of
// the waves decode the next block behind their products, under the barrier that
// the others decode after (14336 x 4096, 4096 tokens: 438 us, 1.10 PF/s; on a
// faster card 422, where all of them after it took 437, every wave at one priority
// 468).  Four groups are four
// waves to a SIMD, which cover each other without that, and their packed rows
// come faster through LDS, by direct loads (64 x 64 tiles: 867 us against 987).
//
// In the last block, lanes past the last chunk of their row read that chunk
// again; what lies past `cols` is then cleared in the activations.
// The smallest tile, with groups of 128 without offsets, fits twice into a compute unit's
// registers (64 rows of 14336 x 4096 x 16 tokens: 11.5 us against 12.5).
// LOOSE: activation rows that start at any element go through registers into
// LDS, loaded before a block's products and stored behind them.
constexpr bool stage_own(int groups) { return groups < 4; }
template <int G, bool OFF, bool S32, int NW, int WI, int BJ, int KG, bool LOOSE>
__global__ __launch_bounds__(64 * NW * KG, G == 128 && !OFF && KG == 4 && BJ == 1 ? 8 : 1) void i4_stage_kernel(I4Args a, int nw_tiles, int nb_tiles, int per_xcd) {
  constexpr int GB = 128 / G;
  constexpr int BW = 16 * WI * NW, BB = 16 * BJ;
  constexpr int LB = BB / 4;  // 1 KB loads of a stage's activations
  constexpr int LW = BW / 16;
  constexpr bool kOwn = stage_own(KG);
  constexpr uint32_t kX = BB * 256, kStage = kX + (kOwn ? 0 : BW * 64);
  constexpr int kPartial = NW * WI * BJ * 1024;  // a group's sums
  // workgroups are dealt to the XCDs round-robin: each XCD takes a run of
  // tiles, 4 activation tiles deep, so that its L2 serves the rereads
  const int id = int(blockIdx.x % kXcds) * per_xcd + int(blockIdx.x / kXcds);
  if (id >= nw_tiles * nb_tiles) return;  // whole workgroups
  constexpr int kDeep = 4;
  const int strip = id / (kDeep * nw_tiles);
  const int deep = min(kDeep, nb_tiles - strip * kDeep);
  const int in = id - strip * kDeep * nw_tiles;
  const int64_t row0 = int64_t(in / deep) * BW, b0 = (int64_t(strip) * kDeep + in % deep) * BB;
  const int lane = int(threadIdx.x) % kWave, w_all = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int group = w_all / NW, wave = w_all % NW;
  const int r = lane % 16, q = lane / 16;
  const Staged4 tw(a.W + row0 * a.ldw, a.rows - row0, (a.cols + 31) / 32 * 16, a.ldw, BW);
  const Staged4 tx(a.X + b0 * a.ldx, a.batch - b0, 2 * a.cols, 2 * a.ldx, BB);
  const int nkb = int((a.cols + 127) / 128), n = (nkb - group + KG - 1) / KG;
  const uint32_t ring = uint32_t(group) * (2 * kStage);
  // a lane's rows and chunks of each load; chunks are the same for all of them
  static_assert(NW % 4 == 0, "rows of a load");
  constexpr int LBN = (LB + NW - 1) / NW;
  const int xchunk = x_chunk<G>(r, 4 * (wave % 4) + q);
  // own weights: rows r of the wave's tiles and chunk q; else the rows and chunks of its 1 KB loads
  constexpr int LWN = kOwn ? WI : (LW + NW - 1) / NW;
  const int wchunk = kOwn ? q : w_slot(lane % 4, lane / 4);
  uint32_t wvo[LWN], xvo[LBN];
#pragma unroll
  for (int u = 0; u < LWN; ++u) {
    const int row = kOwn ? 16 * (wave * WI + u) + r : 16 * (u * NW + wave) + lane / 4;
    wvo[u] = uint32_t(min(row, tw.last)) * uint32_t(a.ldw) + 16 * wchunk;
  }
#pragma unroll
  for (int u = 0; u < LBN; ++u) xvo[u] = uint32_t(min(4 * (u * NW + wave) + q, tx.last)) * uint32_t(2 * a.ldx) + 16 * xchunk;
  // in the last block, how far a lane's chunk lies past the row's last one
  const int wlast = int((a.cols - 1) / 32) % 4, xlast = int((a.cols - 1) / 8) % 16;
  const uint32_t wover = 16 * max(0, wchunk - wlast), xover = 16 * max(0, xchunk - xlast);
  // block i of the group; LOOSE begins with the last one, so that only its
  // start has to do with a block that is not whole
  auto block = [&](int i) {
    const int t = i * KG + group;
    return !LOOSE ? t : t == 0 ? nkb - 1 : t - 1;
  };
  // LOOSE: the activations' way through registers
  u32x4 xr[LOOSE ? LBN : 1];
  auto load_tokens = [&](int i) {
    const char* at = reinterpret_cast<const char*>(a.X + b0 * a.ldx) + int64_t(block(i)) * 256;
#pragma unroll
    for (int u = 0; u < LBN; ++u) xr[u] = load16_any(at + xvo[u]);
  };
  auto load_first = [&]() {
#pragma unroll
    for (int u = 0; u < LBN; ++u) {
      const int64_t row = b0 + min(4 * (u * NW + wave) + q, tx.last);
      const int64_t k = int64_t(block(0)) * 128 + 8 * xchunk;
      xr[u] = u32x4{0u, 0u, 0u, 0u};
      if (k < a.cols) xr[u] = load_x8(a.X + row * a.ldx, k, a.cols);
    }
  };
  auto store_tokens = [&](int i) {
    const uint32_t base = ring + uint32_t(i & 1) * kStage + 16 * lane;
#pragma unroll
    for (int u = 0; u < LBN; ++u)
      if (LB % NW == 0 || u * NW + wave < LB) st128(base + uint32_t(u * NW + wave) * 1024, __builtin_bit_cast(uint4, xr[u]));
  };
  auto issue = [&](int i) {
    const int kb = block(i);
    const uint32_t base = ring + uint32_t(i & 1) * kStage;
    const bool end = kb == nkb - 1;
    if (LOOSE && i > 0) load_tokens(i);
#pragma unroll
    for (int u = 0; u < LBN; ++u)
      if (!LOOSE && (LB % NW == 0 || u * NW + wave < LB))
        stage_load<false>(tx.rsrc, xvo[u] - (end ? xover : 0u), uint32_t(kb) * 256, base + uint32_t(u * NW + wave) * 1024);
  };
  // what the last block holds past `cols` is cleared by the group's threads
  auto clear_tail = [&](int i) {
    const int left = int(a.cols - int64_t(nkb - 1) * 128);
    for (int at = wave * kWave + lane; at < BB * 16; at += NW * kWave) {
      const int row = at / 16, chunk = at % 16;
      if (8 * chunk + 8 <= left) continue;
      const uint32_t p = ring + uint32_t(i & 1) * kStage + uint32_t(row) * 256 + uint32_t(x_slot<G>(chunk, row)) * 16;
      st128(p, __builtin_bit_cast(uint4, __builtin_bit_cast(u32x4, ld128(p)) & tail_mask8(left - 8 * chunk)));
    }
  };
  const int64_t groups = (a.cols + G - 1) / G;
  const GroupRows<S32> scale(a.scale, a.lds, groups, a.rows, row0), offset(OFF ? a.offset : a.scale, OFF ? a.ldo : a.lds, groups, a.rows, row0);
  uint32_t sn[WI][GB], mn[WI][GB];  // the next block's scales and offsets
  auto scales = [&](int i) {
    const uint32_t g0 = uint32_t(block(i)) * GB;
#pragma unroll
    for (int g = 0; g < GB; ++g) {
      const uint32_t gi = min(g0 + g, uint32_t(groups - 1));
#pragma unroll
      for (int t = 0; t < WI; ++t) {
        const uint32_t row = min(uint32_t(16 * (wave * WI + t) + r), uint32_t(tw.last));
        sn[t][g] = scale.load(gi, row);
        if (OFF) mn[t][g] = offset.load(gi, row);
      }
    }
  };
  constexpr uint32_t kSixteenths = 0x3D803D80u;  // two times 1 / 16 in bf16: their products' sums are in the weights' unit
  const bf16x8 sixteenths = __builtin_bit_cast(bf16x8, u32x4{kSixteenths, kSixteenths, kSixteenths, kSixteenths});
  const f32x4 zero{0.f, 0.f, 0.f, 0.f};
  f32x4 acc[WI][BJ];
#pragma unroll
  for (int i = 0; i < WI; ++i)
#pragma unroll
    for (int j = 0; j < BJ; ++j) acc[i][j] = zero;
  // the wave's weights of a block: as they lie in memory, then decoded
  u32x4 raw[WI];
  bf16x8 w[WI][4];
  auto load_weights = [&](int i) {
    const int kb = block(i);
#pragma unroll
    for (int u = 0; u < LWN; ++u) {
      const uint32_t voff = wvo[u] - (kb == nkb - 1 ? wover : 0u);
      if (kOwn) raw[u] = buffer_load16(tw.rsrc, voff, uint32_t(kb) * 64);
      else if (LW % NW == 0 || u * NW + wave < LW)
        stage_load<false>(tw.rsrc, voff, uint32_t(kb) * 64, ring + uint32_t(i & 1) * kStage + kX + uint32_t(u * NW + wave) * 1024);
    }
  };
  auto decode = [&](int i) {
#pragma unroll
    for (int t = 0; t < WI; ++t) {
      if (!kOwn) {
        const uint32_t row = uint32_t((wave * WI + t) * 16 + r);
        raw[t] = __builtin_bit_cast(u32x4, ld128(ring + uint32_t(i & 1) * kStage + kX + row * 64 + uint32_t(w_slot(q, r)) * 16));
      }
      if (G != 128) transpose4(raw[t]);
#pragma unroll
      for (int s = 0; s < 4; ++s) w[t][s] = decode_q8(raw[t][s]);
    }
  };
  const uint32_t xat = uint32_t(r) * 256;
  auto multiply = [&](int i, const float (&sc)[WI][GB], const float (&mc)[WI][GB]) {
    const uint32_t base = ring + uint32_t(i & 1) * kStage;
    // one tile of tokens at a time: the next one's operands are read and the last one's sums are scaled while this one's
    // products run; the barriers keep the compiler from holding more tiles than that in registers
    bf16x8 x[2][4];
    f32x4 part[2][WI], sum[2];
    // kept apart, so that a read's address is one of these and a constant
    uint32_t xs[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      xs[s] = base + xat + uint32_t((4 * s + q) ^ r) * 16;
      asm("" : "+v"(xs[s]));
    }
    auto read = [&](int j, bf16x8 (&to)[4]) {
#pragma unroll
      for (int s = 0; s < 4; ++s) to[s] = __builtin_bit_cast(bf16x8, ld128(xs[s] + uint32_t(j) * 4096));
    };
    auto fold = [&](int j, int g, const f32x4 (&pt)[WI], const f32x4& sm) {
#pragma unroll
      for (int t = 0; t < WI; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[t][j][e] = fmaf(sc[t][g], pt[t][e], acc[t][j][e]);
          if (OFF) acc[t][j][e] = fmaf(mc[t][g], sm[e], acc[t][j][e]);
        }
      }
    };
    read(0, x[0]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < BJ; ++j) {
      if (j + 1 < BJ) read(j + 1, x[(j + 1) & 1]);
#pragma unroll
      for (int g = 0; g < GB; ++g) {
        const int now = (j * GB + g) & 1;
#pragma unroll
        for (int s = 0; s < 4 / GB; ++s) {
          const int at = g * (4 / GB) + s;
#pragma unroll
          for (int t = 0; t < WI; ++t) part[now][t] = mfma_bf16(x[j & 1][at], w[t][at], s ? part[now][t] : zero);
          if (OFF) sum[now] = mfma_bf16(x[j & 1][at], sixteenths, s ? sum[now] : zero);
        }
        if (j * GB + g > 0) fold((j * GB + g - 1) / GB, (j * GB + g - 1) % GB, part[now ^ 1], sum[now ^ 1]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    fold(BJ - 1, GB - 1, part[(BJ * GB - 1) & 1], sum[(BJ * GB - 1) & 1]);
  };
  if (n > 0) {
    if (LOOSE) load_first();
    load_weights(0);
    issue(0);
    scales(0);
    if (LOOSE) store_tokens(0);
  }
  // every wave takes part in the barriers of the first group's blocks
  const int steps = (nkb + KG - 1) / KG;
  const bool late = kOwn && w_all / 4 % 2;
  if (late && n > 0) decode(0);
  if (late) __builtin_amdgcn_s_setprio(2);
  else if (kOwn || w_all >= 4) __builtin_amdgcn_s_setprio(1);
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
    wait_vmcnt<0>();  // this wave's loads of block i (and its scales) have landed
    lds_barrier();    // every wave's have; block i - 1 is no longer read
    if (!LOOSE && i == steps - 1 && a.cols % 128) {
      if (i * KG + group == nkb - 1) clear_tail(i);
      lds_barrier();
    }
    float sc[WI][GB], mc[WI][GB];
#pragma unroll
    for (int t = 0; t < WI; ++t)
#pragma unroll
      for (int g = 0; g < GB; ++g) {
        sc[t][g] = scale.value(sn[t][g]);
        mc[t][g] = OFF ? offset.value(mn[t][g]) : 0.f;
      }
    // ahead of the loads, whose arrival the compiler would wait for together with the weights'
    if (kOwn && !late && i < n) decode(i);
    if (i + 1 < n) {
      load_weights(i + 1);
      issue(i + 1);
      scales(i + 1);
    }
    // a branch even where every group has the block: across it the compiler would hold more in registers than there are
    if (i < n) {
      if (!kOwn) decode(i);
      multiply(i, sc, mc);
    }
    if (LOOSE && i + 1 < n) store_tokens(i + 1);
    if (late && i + 1 < n) {
      __builtin_amdgcn_s_setprio(0);
      decode(i + 1);
      __builtin_amdgcn_s_setprio(2);
    }
  }
  __syncthreads();  // no wave reads the rings any more
  if (KG > 1) {
    const uint32_t mine = uint32_t(wave) * (WI * BJ * 1024) + 16 * lane;
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < WI; ++i)
#pragma unroll
        for (int j = 0; j < BJ; ++j)
          st128(uint32_t((group - 1) * kPartial) + mine + uint32_t(i * BJ + j) * 1024, __builtin_bit_cast(uint4, acc[i][j]));
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 0; g < KG - 1; ++g)
#pragma unroll
      for (int i = 0; i < WI; ++i)
#pragma unroll
        for (int j = 0; j < BJ; ++j) {
          const f32x4 v = __builtin_bit_cast(f32x4, ld128(uint32_t(g * kPartial) + mine + uint32_t(i * BJ + j) * 1024));
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] += v[e];
        }
  }
  const int64_t n0 = row0 + 16 * wave * WI, bw0 = b0;
  const uint32_t out = uint32_t((KG - 1) * kPartial + wave * epilogue_bytes<WI>);
  if (a.yt == UW_F32) store_through_lds<WI, BJ, false>(a, n0, bw0, out, lane, acc);
  else store_through_lds<WI, BJ, true>(a, n0, bw0, out, lane, acc);
}

// A launch holds fewer than 2^32 threads.  In double: sizes below 2^40 make
// products past 64 bits.
int check_launch(int64_t nw, int64_t nb, int threads) {
  if ((double(nw) * double(nb) + kXcds) * threads < 4294967296.0) return UW_OK;
  return fail(UW_ERR_UNSUPPORTED, "uw_i4_gemm: too many tiles for one launch");
}

template <int G, bool OFF>
int run_direct(const I4Args& a, hipStream_t s) {
  const int64_t n_groups = (a.rows + 15) / 16, ny = (a.batch + 15) / 16;
  const int ks = int(std::min<int64_t>(8, (a.cols + 127) / 128));
  if (int rc = check_launch((n_groups + kXcds - 1) / kXcds * kXcds, ny, ks * kWave)) return rc;
  const int64_t grid = (n_groups + kXcds - 1) / kXcds * kXcds * ny;
  hipLaunchKernelGGL((i4_direct_kernel<G, OFF>), dim3(unsigned(grid)), dim3(ks * kWave), size_t(ks) * 1024, s, a,
                     int(n_groups), int(ny), ks);
  return hip_check(hipGetLastError(), "i4_direct_kernel launch");
}

template <int G, bool OFF, bool S32, int KW, int D>
int run_stream(const I4Args& a, hipStream_t s) {
  const int64_t tiles = (a.rows + 15) / 16, lds = stream_lds(a, KW);
  const int64_t grid = std::min<int64_t>(tiles, kCus * std::max<int64_t>(1, std::min<int64_t>(16 / KW, kLdsLimit / lds)));
  const bool small = a.batch * ((a.cols / 8 + 64 * KW - 1) / (64 * KW)) <= 2;  // steps of the activations' way into LDS
  auto kern = small ? i4_stream_kernel<G, OFF, S32, KW, D, 2> : i4_stream_kernel<G, OFF, S32, KW, D, 8>;
  allow_full_lds(kern);
  hipLaunchKernelGGL(kern, dim3(unsigned(grid)), dim3(KW * kWave), size_t(lds), s, a, int(tiles), stream_pitch(a.cols));
  return hip_check(hipGetLastError(), "i4_stream_kernel launch");
}

template <int G, bool OFF, bool S32, int WI, int KW, int D>
int run_token(const I4Args& a, hipStream_t s) {
  const int64_t nw = (a.rows + 16 * WI - 1) / (16 * WI);
  if (int rc = check_launch(nw, 1, KW * kWave)) return rc;
  auto kern = a.batch == 1 ? i4_token_kernel<G, OFF, S32, WI, 1, KW, D> : i4_token_kernel<G, OFF, S32, WI, 4, KW, D>;
  const size_t lds = size_t(KW) * std::max(256 * WI, 272 * (a.batch == 1 ? 1 : 4));
  hipLaunchKernelGGL(kern, dim3(unsigned(nw)), dim3(KW * kWave), lds, s, a, int(nw));
  return hip_check(hipGetLastError(), "i4_token_kernel launch");
}

template <int G, bool OFF, bool S32, int WI, int BJ, int KW, int D>
int run_slice(const I4Args& a, hipStream_t s) {
  const int64_t nw = (a.rows + 16 * WI - 1) / (16 * WI), nb = (a.batch + 16 * BJ - 1) / (16 * BJ);
  if (int rc = check_launch((nw + kXcds - 1) / kXcds * kXcds, nb, KW * kWave)) return rc;
  const int64_t grid = (nw + kXcds - 1) / kXcds * kXcds * nb;
  auto kern = i4_slice_kernel<G, OFF, S32, WI, BJ, KW, D>;
  constexpr size_t kLds = size_t(KW) * WI * BJ * 1024;
  static_assert(kLds <= kLdsLimit, "LDS");
  allow_full_lds(kern);
  hipLaunchKernelGGL(kern, dim3(unsigned(grid)), dim3(KW * kWave), kLds, s, a, int(nw), int(nb));
  return hip_check(hipGetLastError(), "i4_slice_kernel launch");
}

template <int G, bool OFF, bool S32, int WI, int BJ, int KW, int D>
int run_deep(const I4Args& a, hipStream_t s) {
  const int64_t nw = (a.rows + 16 * WI - 1) / (16 * WI), nb = (a.batch + 16 * BJ - 1) / (16 * BJ);
  if (int rc = check_launch((nw + kXcds - 1) / kXcds * kXcds, nb, KW * kWave)) return rc;
  const int64_t grid = (nw + kXcds - 1) / kXcds * kXcds * nb;
  auto kern = i4_deep_kernel<G, OFF, S32, WI, BJ, KW, D>;
  constexpr size_t kRing = size_t(KW) * D * (4096 * BJ + 1024 * WI + StagedGroups<G, S32, WI>::kLoads * 256 * (OFF ? 2 : 1));
  constexpr size_t kLds = std::max(kRing, size_t(KW) * WI * BJ * 1024);
  static_assert(kLds <= kLdsLimit, "LDS");
  allow_full_lds(kern);
  hipLaunchKernelGGL(kern, dim3(unsigned(grid)), dim3(KW * kWave), kLds, s, a, int(nw), int(nb));
  return hip_check(hipGetLastError(), "i4_deep_kernel launch");
}

template <int G, bool OFF, bool S32, int NW, int WI, int BJ, int KG, bool LOOSE = false>
int run_stage(const I4Args& a, hipStream_t s) {
  constexpr int BW = 16 * WI * NW, BB = 16 * BJ, kThreads = 64 * NW * KG;
  const int64_t nw = (a.rows + BW - 1) / BW, nb = (a.batch + BB - 1) / BB;
  if (int rc = check_launch(nw, nb, kThreads)) return rc;
  const int64_t per_xcd = (nw * nb + kXcds - 1) / kXcds;
  auto kern = i4_stage_kernel<G, OFF, S32, NW, WI, BJ, KG, LOOSE>;
  constexpr size_t kLds = std::max(size_t(KG) * 2 * (BB * 256 + (stage_own(KG) ? 0 : BW * 64)), size_t(KG - 1) * NW * WI * BJ * 1024 + NW * epilogue_bytes<WI>);
  static_assert(kLds <= kLdsLimit, "LDS");
  allow_full_lds(kern);
  hipLaunchKernelGGL(kern, dim3(unsigned(per_xcd * kXcds)), dim3(kThreads), kLds, s, a, int(nw), int(nb), int(per_xcd));
  return hip_check(hipGetLastError(), "i4_stage_kernel launch");
}

template <int G, bool OFF, bool S32>
int run_gemm(const I4Args& a, int shape, hipStream_t s) {
  switch (shape) {
    case 1: return run_direct<G, OFF>(a, s);
    case 2: return run_token<G, OFF, S32, 2, 8, 2>(a, s);
    case 3: return run_token<G, OFF, S32, 1, 8, 4>(a, s);
    case 4: return run_stream<G, OFF, S32, 8, 4>(a, s);
    case 5: return run_slice<G, OFF, S32, G == 32 ? 2 : 4, 1, 8, 2>(a, s);
    case 6: return run_slice<G, OFF, S32, 1, 1, 16, 2>(a, s);
    case 7: return run_slice<G, OFF, S32, 2, 1, 16, 1>(a, s);
    case 8: return run_deep<G, OFF, S32, 1, 1, 8, 3>(a, s);
    case 9: return run_deep<G, OFF, S32, 2, 1, 8, 2>(a, s);
    case 10: return run_stage<G, OFF, S32, 4, 1, 1, 4>(a, s);   // 64 x 16, 4 groups
    case 11: return run_stage<G, OFF, S32, 4, 1, 2, 4>(a, s);   // 64 x 32, 4 groups
    case 12: return run_stage<G, OFF, S32, 4, 1, 4, 4>(a, s);   // 64 x 64, 4 groups
    case 13: return run_stage<G, OFF, S32, 4, 2, 4, 3>(a, s);   // 128 x 64, 3 groups
    case 14: return run_stage<G, OFF, S32, 4, 2, 8, 2>(a, s);   // 128 x 128, 2 groups
    case 15: return run_stage<G, OFF, S32, 8, 2, (OFF || G == 32 ? 12 : 16), 1>(a, s);  // 256 x 256, or 192 where registers hold no more
    case 16: return run_stage<G, OFF, S32, 4, 1, 2, 4, true>(a, s);   // 64 x 32, 4 groups
    case 17: return run_stage<G, OFF, S32, 4, 1, 4, 4, true>(a, s);   // 64 x 64, 4 groups
    case 18: return run_stage<G, OFF, S32, 4, 2, 8, 2, true>(a, s);   // 128 x 128, 2 groups
    default: return run_stage<G, OFF, S32, 8, 2, 8, 1, true>(a, s);   // 256 x 128
  }
}

template <int G>
int run_form(const I4Args& a, int shape, hipStream_t s) {
  if (a.st == UW_F32) return a.offset ? run_gemm<G, true, true>(a, shape, s) : run_gemm<G, false, true>(a, shape, s);
  return a.offset ? run_gemm<G, true, false>(a, shape, s) : run_gemm<G, false, false>(a, shape, s);
}

}  // namespace
}  // namespace uw
