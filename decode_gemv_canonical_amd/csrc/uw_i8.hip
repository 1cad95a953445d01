// Product of 8-bit integer matrices with a scale per token and per channel,
// on the gfx950 matrix cores:
//
//   Y[b, n] = x_scale[b] * w_scale[n] * sum_k X[b, k] W[n, k] (+ bias[n])
//
// The sum is exact: v_mfma_i32_16x16x64_i8 adds into 32-bit integers, and
// cols <= 131071 keeps |sum| <= 131071 * 128 * 128 < 2^31.  So the result does
// not depend on tiles, waves or splits of k; it is rounded to fp32, scaled
// in fp32 and rounded once more where Y is bf16.
//
// W [rows, cols] and X [batch, cols] are both k-contiguous.  A = 16 weight
// rows, B = 16 activation rows: lane (r = lane % 16, q = lane / 16) holds 16
// consecutive bytes of row r, at the same k for both operands; lane (r, q) of
// the result holds weight rows 4 q .. 4 q + 3 for activation row r, four
// consecutive values of a row of Y.
#include <algorithm>
#include <cmath>

#include "uw_device.h"

namespace uw {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kXcds = 8;

struct I8Args {
  const int8_t* W;
  const float* sw;
  const int8_t* X;
  const float* sx;
  const float* bias;  // may be null
  char* Y;
  int64_t rows, cols, ldw, batch, ldx, ldy;
};

__device__ __forceinline__ i32x4 mfma_i8(const u32x4& a, const u32x4& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

__device__ __forceinline__ u32x4 load16_any(const int8_t* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// 16 bytes of a row at p, of which `left` lie inside it (may be <= 0); the
// others read as zero and are not touched.
__device__ __forceinline__ u32x4 load16_tail(const int8_t* p, int64_t left) {
  if (left >= 16) return load16_any(p);
  uint32_t b[15];  // all loads before the first use
#pragma unroll
  for (int e = 0; e < 15; ++e) b[e] = 0u;
#pragma unroll
  for (int e = 0; e < 15; ++e)
    if (e < left) b[e] = uint8_t(p[e]);
  u32x4 v{0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 15; ++e) v[e / 4] |= b[e] << (8 * (e & 3));
  return v;
}

// A sum as it goes out: rounded to fp32, scaled, the bias added, three
// roundings in every kernel (left to itself the compiler makes the last two one
// in some of them, and a result would hang on the shape that runs).
__device__ __forceinline__ float scaled(int sum, float scale, bool biased, float bias) {
#pragma clang fp contract(off)
  const float v = float(sum) * scale;
  return biased ? v + bias : v;
}

// Four consecutive values of row b of Y, weight rows n .. n + 3 (n < rows).
template <bool YBF16>
__device__ __forceinline__ void store_row4(const I8Args& a, int64_t b, int64_t n, const float (&v)[4]) {
  const int m = int(std::min<int64_t>(4, a.rows - n));
  if (YBF16) {
    uint16_t* y = reinterpret_cast<uint16_t*>(a.Y) + b * a.ldy + n;
    const uint32_t w[2] = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    if (m == 4) {
      __builtin_memcpy(y, w, 8);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < m) y[e] = uint16_t(w[e / 2] >> (16 * (e & 1)));
    }
  } else {
    float* y = reinterpret_cast<float*>(a.Y) + b * a.ldy + n;
    if (m == 4) {
      __builtin_memcpy(y, v, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < m) y[e] = v[e];
    }
  }
}

// Values n .. n + 3 of a vector of `rows`; past the end, its last one.
__device__ __forceinline__ void load_row4(const float* p, int64_t n, int64_t rows, float (&v)[4]) {
  if (n + 4 <= rows) {
    __builtin_memcpy(v, p + n, 16);
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = p[std::min<int64_t>(n + e, rows - 1)];
}

// 16 bytes of row b of Y from column n on: 16 / SIZE values.  NT: whole lines
// are written, past the caches.
template <int SIZE, bool NT>
__device__ __forceinline__ void store_row16(const I8Args& a, int64_t b, int64_t n, const uint4& v) {
  if (b >= a.batch || n >= a.rows) return;
  char* y = a.Y + (b * a.ldy + n) * SIZE;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const int m = int(std::min<int64_t>(16 / SIZE, a.rows - n));
  if (m == 16 / SIZE) {
    if (NT) __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4*>(y));
    else __builtin_memcpy(y, w, 16);
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

// The same from the integer sums of one 16 x 16 tile.
template <bool YBF16>
__device__ __forceinline__ void store_y4(const I8Args& a, int64_t b, int64_t n, const i32x4& acc) {
  if (b >= a.batch || n >= a.rows) return;
  const float sx = a.sx[b];
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t at = std::min<int64_t>(n + e, a.rows - 1);
    v[e] = scaled(acc[e], sx * a.sw[at], a.bias, a.bias ? a.bias[at] : 0.f);
  }
  store_row4<YBF16>(a, b, n, v);
}

template <int WI, bool YBF16>
constexpr int epilogue_bytes = 16 * (16 * WI * (YBF16 ? 2 : 4) + 16);

// Epilogue of a wave's WI x BJ tiles at (n0, bw0), through LDS: 16 activation
// rows at a time as the wave's 16 WI columns, so that rows go out in runs of
// 32 WI bytes (bf16) or twice that (without it, 4096 x 4096 x 64 took 19.1 us,
// with it 13.4); 16 bytes of padding a row spread the writes over the banks.
// The scales are read before anything is stored.  out: the wave's place in
// LDS, epilogue_bytes<WI, YBF16> that nothing else uses any more.
// NT: Y's rows start at whole lines, which are then stored non-temporally and
// leave the caches to the operands (4096 x 14336 x 4096: 237 -> 215 us, 2048 x
// 4096 x 14336: 124 -> 117; a silu that reads the result next loses nothing).
template <int WI, int BJ, bool YBF16, bool NT>
__device__ __forceinline__ void store_through_lds(const I8Args& a, int64_t n0, int64_t bw0, uint32_t out, int lane,
                                                  const i32x4 (&acc)[WI][BJ]) {
  constexpr int kCols = 16 * WI, kSize = YBF16 ? 2 : 4, kPitch = kCols * kSize + 16;
  const int r = lane % 16, q = lane / 16;
  float sx[BJ], sw[WI][4], bias[WI][4] = {};
#pragma unroll
  for (int j = 0; j < BJ; ++j) sx[j] = a.sx[std::min<int64_t>(bw0 + 16 * j + r, a.batch - 1)];
#pragma unroll
  for (int i = 0; i < WI; ++i) {
    load_row4(a.sw, n0 + 16 * i + 4 * q, a.rows, sw[i]);
    if (a.bias) load_row4(a.bias, n0 + 16 * i + 4 * q, a.rows, bias[i]);
  }
#pragma unroll
  for (int j = 0; j < BJ; ++j) {
#pragma unroll
    for (int i = 0; i < WI; ++i) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = scaled(acc[i][j][e], sx[j] * sw[i][e], a.bias, bias[i][e]);
      const uint32_t dst = out + uint32_t(r) * kPitch + uint32_t(16 * i + 4 * q) * kSize;
      if (YBF16) st64(dst, pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
      else st128(dst, uint4{f32_bits(v[0]), f32_bits(v[1]), f32_bits(v[2]), f32_bits(v[3])});
    }
    wave_lds_fence();
    constexpr int kPer = 16 / kSize, kLanes = kCols / kPer;  // values a lane stores; lanes of a row
    constexpr int kChunks = 16 * kLanes;                     // of the 16 rows
#pragma unroll
    for (int c0 = 0; c0 < kChunks; c0 += kWave) {
      const int at = c0 + lane, br = at / kLanes, c = at % kLanes * kPer;
      if (kChunks % kWave == 0 || at < kChunks)
        store_row16<kSize, NT>(a, bw0 + 16 * j + br, n0 + c, ld128(out + uint32_t(br) * kPitch + uint32_t(c) * kSize));
    }
    wave_lds_fence();
  }
}

// Operands of any alignment, few rows: straight from global memory into
// registers.  A workgroup holds 16 weight rows and 16 activation rows; its KS
// waves split k: wave w takes the 256-byte groups w, w + KS, ... and the
// partial tiles are summed in LDS.  The next group's loads are issued before
// this group's products.  Rows may start at any byte; nothing outside a row is
// read.  1 x 4096 x 4099: 12.4 us, against 17.0 for i8_loose_kernel.
template <bool YBF16>
__global__ __launch_bounds__(512) void i8_direct_kernel(I8Args a, int n_groups, int ny, int KS) {
  const int L = int(blockIdx.x);
  const int grp = (L / (kXcds * ny)) * kXcds + L % kXcds;
  const int y = (L / kXcds) % ny;
  if (grp >= n_groups) return;  // whole workgroups
  const int lane = int(threadIdx.x) % kWave, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int r = lane % 16, q = lane / 16;
  const int64_t row0 = int64_t(grp) * 16, b0 = int64_t(y) * 16;
  const int8_t* wr = a.W + std::min<int64_t>(row0 + r, a.rows - 1) * a.ldw + 16 * q;
  const int8_t* xr = a.X + std::min<int64_t>(b0 + r, a.batch - 1) * a.ldx + 16 * q;
  i32x4 acc{0, 0, 0, 0};
  const int nfull = int(a.cols / 256);
  u32x4 wc[4], xc[4], wn[4], xn[4];
  auto load = [&](int g, u32x4 (&w)[4], u32x4 (&x)[4]) {
    const int64_t k = int64_t(g) * 256;
#pragma unroll
    for (int s = 0; s < 4; ++s) w[s] = load16_any(wr + k + 64 * s);
#pragma unroll
    for (int s = 0; s < 4; ++s) x[s] = load16_any(xr + k + 64 * s);
  };
  auto mul = [&](const u32x4 (&w)[4], const u32x4 (&x)[4]) {
#pragma unroll
    for (int s = 0; s < 4; ++s) acc = mfma_i8(w[s], x[s], acc);
  };
  int g = wave;
  if (g < nfull) load(g, wc, xc);
  while (g < nfull) {
    const int next = g + KS;
    if (next < nfull) load(next, wn, xn);
    mul(wc, xc);
    g = next;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      wc[s] = wn[s];
      xc[s] = xn[s];
    }
  }
  if (a.cols % 256 && nfull % KS == wave) {
    const int64_t k = int64_t(nfull) * 256, left = a.cols - k - 16 * q;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      wc[s] = load16_tail(wr + k + 64 * s, left - 64 * s);
      xc[s] = load16_tail(xr + k + 64 * s, left - 64 * s);
    }
    mul(wc, xc);
  }
  st128(uint32_t(wave * 1024 + 16 * lane), __builtin_bit_cast(uint4, acc));
  __syncthreads();
  if (wave) return;
  for (int w = 1; w < KS; ++w) acc += __builtin_bit_cast(i32x4, ld128(uint32_t(w * 1024 + 16 * lane)));
  store_y4<YBF16>(a, b0 + r, row0 + 4 * q, acc);
}

// Staging of an operand's tile: rows of 128 bytes of k in LDS, the 16-byte
// chunk c of row r at chunk c ^ (r % 8), so that the 8 rows an operand read
// touches at a time lie in 8 different bank groups.  One load moves 8 rows:
// lane l puts row l / 8's chunk (l % 8) ^ (l / 8) at 16 l.  Needs a 16-byte
// aligned operand whose stride is a multiple of 16.
//
// The block that holds the end of the rows is loaded like the others, but
// lanes past the last chunk of their row read that chunk again: no address
// lies outside the 16-byte chunks that hold the operand (and the buffer ends
// at the last row's last 4-byte word).  What lies past `cols` is masked out
// of the activation operand when it is read back (whole numbers: any value
// times zero is zero).
struct Staged {
  __amdgpu_buffer_rsrc_t rsrc;
  int last;  // the tile's last row; the rows past it are that row again

  __device__ __forceinline__ Staged(const int8_t* tile, int64_t rows, int64_t cols, int64_t ld, int tile_rows)
      : last(__builtin_amdgcn_readfirstlane(int(std::min<int64_t>(tile_rows, rows)) - 1)) {
    // the same in every lane; readfirstlane keeps it in scalar registers
    const uint64_t p = reinterpret_cast<uint64_t>(tile);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(p)), hi = __builtin_amdgcn_readfirstlane(uint32_t(p >> 32));
    const int bytes = __builtin_amdgcn_readfirstlane(int(int64_t(last) * ld + (cols + 3) / 4 * 4));
    rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uint64_t(hi) << 32 | lo), int16_t(0), bytes, 0x00020000);
  }
  // byte offset of staged row `row` (of the lane) at k = 0
  __device__ __forceinline__ uint32_t row_offset(int row, int64_t ld) const {
    return uint32_t(min(row, last)) * uint32_t(ld);
  }
};

// Mask of 16 bytes of which the first `left` lie inside their row.
__device__ __forceinline__ u32x4 tail_mask(int left) {
  u32x4 m;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int n = left - 4 * d;
    m[d] = n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
  }
  return m;
}

// Small batches: a workgroup holds BW weight rows and BB activation rows, and
// its KW waves split k: wave w takes the 128-byte blocks w, w + KW, ... for the
// whole tile.  A wave stages its blocks into its own ring of ST slots in LDS
// by direct loads and reads them back as operands, so nothing but its own
// loads is ever waited for: no barrier until the partial tiles are summed at
// the end.  A slot is refilled as soon as its operands are in registers, so
// ST blocks are in flight.  NT: the weights are loaded non-temporally.
template <int BW, int BB, int KW, int ST, bool NT, bool YBF16>
__global__ __launch_bounds__(64 * KW) void i8_slice_kernel(I8Args a, int nw_tiles, int nb_tiles) {
  constexpr int WI = BW / 16, BJ = BB / 16;
  constexpr int LW = BW / 8, LB = BB / 8, L = LW + LB;  // 1 KB loads per block
  constexpr uint32_t kWBytes = BW * 128, kSlot = (BW + BB) * 128;
  static_assert(ST * L < 64, "vmcnt");
  // the batch tiles of one weight tile run back to back on one XCD
  const int id = int(blockIdx.x);
  const int wt = (id / (kXcds * nb_tiles)) * kXcds + id % kXcds, y = (id / kXcds) % nb_tiles;
  if (wt >= nw_tiles) return;  // whole workgroups
  const int64_t row0 = int64_t(wt) * BW, b0 = int64_t(y) * BB;
  const int lane = int(threadIdx.x) % kWave, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int lrow = lane / 8, lchunk = (lane % 8) ^ lrow;
  const Staged tw(a.W + row0 * a.ldw, a.rows - row0, a.cols, a.ldw, BW);
  const Staged tx(a.X + b0 * a.ldx, a.batch - b0, a.cols, a.ldx, BB);
  uint32_t wvo[LW], xvo[LB];
#pragma unroll
  for (int u = 0; u < LW; ++u) wvo[u] = tw.row_offset(8 * u + lrow, a.ldw) + 16 * lchunk;
#pragma unroll
  for (int u = 0; u < LB; ++u) xvo[u] = tx.row_offset(8 * u + lrow, a.ldx) + 16 * lchunk;
  const uint32_t ring = uint32_t(wave) * (ST * kSlot);
  const int nkb = int((a.cols + 127) / 128), n = (nkb - wave + KW - 1) / KW;  // this wave's blocks
  // Rows whose stride is a multiple of 4 KB have the same k on the same memory
  // channels: the workgroups of an XCD then start at k's spread over the row
  // (1 x 8192 x 8192: 13.4 -> 12.2 us, 16 x 28672 x 4096: 22.3 -> 20.5, 32 x
  // 8192 x 8192: 17.3 -> 15.2; at a stride of 14336 it costs 2 %).
  const int rot = a.ldw % 4096 == 0 ? __builtin_amdgcn_readfirstlane(int(int64_t(wt / kXcds % 32) * nkb / 32)) : 0;
  auto block = [&](int i) {
    const int p = wave + KW * i + rot;
    return p >= nkb ? p - nkb : p;
  };
  // in the last block, how far a lane's chunk lies past the row's last one
  const int over = max(0, 16 * (lchunk - (int(a.cols - 1) % 128) / 16));
  auto issue = [&](int i, int st) {
    const int kb = block(i);
    const uint32_t base = ring + uint32_t(st) * kSlot, k = uint32_t(kb) * 128, back = kb == nkb - 1 ? over : 0;
#pragma unroll
    for (int u = 0; u < LW; ++u) stage_load<NT>(tw.rsrc, wvo[u] - back, k, base + u * 1024);
#pragma unroll
    for (int u = 0; u < LB; ++u) stage_load<false>(tx.rsrc, xvo[u] - back, k, base + kWBytes + u * 1024);
  };
  const int r = lane % 16, q = lane / 16;
  i32x4 acc[WI][BJ];
#pragma unroll
  for (int i = 0; i < WI; ++i)
#pragma unroll
    for (int j = 0; j < BJ; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < ST; ++i)
    if (i < n) issue(i, i);
  int st = 0;
  for (int i = 0; i < n; ++i) {
    wait_ring<L, ST - 1>(n - 1 - i);  // block i has landed
    const uint32_t base = ring + uint32_t(st) * kSlot;
    u32x4 w[WI][2], x[BJ][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t at = base + uint32_t(r) * 128 + uint32_t(((4 * s + q) ^ (r & 7)) * 16);
#pragma unroll
      for (int e = 0; e < WI; ++e) w[e][s] = __builtin_bit_cast(u32x4, ld128(at + uint32_t(e) * 2048));
#pragma unroll
      for (int j = 0; j < BJ; ++j) x[j][s] = __builtin_bit_cast(u32x4, ld128(at + kWBytes + uint32_t(j) * 2048));
    }
    if (i + ST < n) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot's operands are in registers
      issue(i + ST, st);
    }
    const int kb = block(i);
    if (kb == nkb - 1 && a.cols % 128) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const u32x4 m = tail_mask(int(a.cols - int64_t(kb) * 128) - 16 * (4 * s + q));
#pragma unroll
        for (int j = 0; j < BJ; ++j) x[j][s] &= m;
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int e = 0; e < WI; ++e)
#pragma unroll
        for (int j = 0; j < BJ; ++j) acc[e][j] = mfma_i8(w[e][s], x[j][s], acc[e][j]);
    st = st + 1 == ST ? 0 : st + 1;
  }
  // partial tile idx = i BJ + j of wave w at (w WI BJ + idx) KB
  __syncthreads();  // every wave is done with its ring
#pragma unroll
  for (int i = 0; i < WI; ++i)
#pragma unroll
    for (int j = 0; j < BJ; ++j)
      st128(uint32_t(((wave * WI + i) * BJ + j) * 1024 + 16 * lane), __builtin_bit_cast(uint4, acc[i][j]));
  __syncthreads();
  for (int idx = wave; idx < WI * BJ; idx += KW) {
    i32x4 sum{0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < KW; ++v)
      sum += __builtin_bit_cast(i32x4, ld128(uint32_t((v * WI * BJ + idx) * 1024 + 16 * lane)));
    store_y4<YBF16>(a, b0 + 16 * (idx % BJ) + r, row0 + 16 * (idx / BJ) + 4 * q, sum);
  }
}

// Large batches: both operands of a 128-byte block of k are staged for the
// whole workgroup, in a ring of ST stages: BW weight rows and BB activation
// rows, whose WGW x WGB waves each hold a BW / WGW by BB / WGB tile.  KG groups
// of such waves, each with its own ring, take every KG-th block and add their
// sums in LDS at the end: where the tiles are few and k is long, a compute
// unit then works on as many blocks at a time as with KG workgroups.
template <int BW, int BB, int WGW, int WGB, int ST, int KG, bool YBF16, bool NT>
__global__ __launch_bounds__(64 * WGW * WGB * KG) void i8_stage_kernel(I8Args a, int nw_tiles, int nb_tiles, int per_xcd) {
  constexpr int NW = WGW * WGB;
  constexpr int WI = BW / WGW / 16, BJ = BB / WGB / 16;
  constexpr int LW = BW / 8 / NW, LB = BB / 8 / NW;  // 1 KB loads (8 rows) per wave and stage
  constexpr uint32_t kWBytes = BW * 128, kStage = (BW + BB) * 128;
  constexpr int kPartial = NW * WI * BJ * 1024;  // a group's sums
  static_assert(BW % (8 * NW) == 0 && BB % (8 * NW) == 0, "whole loads");
  static_assert((KG - 1) * kPartial + NW * epilogue_bytes<WI, YBF16> <= KG * ST * int(kStage), "LDS");
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
  const int lrow = lane / 8, lchunk = (lane % 8) ^ lrow;
  const Staged tw(a.W + row0 * a.ldw, a.rows - row0, a.cols, a.ldw, BW);
  const Staged tx(a.X + b0 * a.ldx, a.batch - b0, a.cols, a.ldx, BB);
  uint32_t wvo[LW], xvo[LB];
#pragma unroll
  for (int u = 0; u < LW; ++u) wvo[u] = tw.row_offset(8 * (u * NW + wave) + lrow, a.ldw) + 16 * lchunk;
#pragma unroll
  for (int u = 0; u < LB; ++u) xvo[u] = tx.row_offset(8 * (u * NW + wave) + lrow, a.ldx) + 16 * lchunk;
  const int nkb = int((a.cols + 127) / 128);
  const int n = (nkb - group + KG - 1) / KG;  // this group's blocks; the first group has the most
  const int over = max(0, 16 * (lchunk - (int(a.cols - 1) % 128) / 16));
  const uint32_t ring = uint32_t(group) * (ST * kStage);
  auto issue = [&](int i, int st) {
    const int kb = i * KG + group;
    const uint32_t base = ring + uint32_t(st) * kStage, k = uint32_t(kb) * 128, back = kb == nkb - 1 ? over : 0;
#pragma unroll
    for (int u = 0; u < LW; ++u) stage_load<false>(tw.rsrc, wvo[u] - back, k, base + uint32_t(u * NW + wave) * 1024);
#pragma unroll
    for (int u = 0; u < LB; ++u)
      stage_load<false>(tx.rsrc, xvo[u] - back, k, base + kWBytes + uint32_t(u * NW + wave) * 1024);
  };
  const int r = lane % 16, q = lane / 16;
  const int ww = wave / WGB, wb = wave % WGB;
  const uint32_t arow = uint32_t(ww * WI * 16 + r) * 128, xrow = kWBytes + uint32_t(wb * BJ * 16 + r) * 128;
  i32x4 acc[WI][BJ];
#pragma unroll
  for (int i = 0; i < WI; ++i)
#pragma unroll
    for (int j = 0; j < BJ; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  auto multiply = [&](uint32_t base, bool tail) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t ch = uint32_t(((4 * s + q) ^ (r & 7)) * 16);
      u32x4 x[BJ];
#pragma unroll
      for (int j = 0; j < BJ; ++j) x[j] = __builtin_bit_cast(u32x4, ld128(base + xrow + uint32_t(j) * 2048 + ch));
      if (tail) {
        const u32x4 m = tail_mask(int(a.cols - int64_t(nkb - 1) * 128) - 16 * (4 * s + q));
#pragma unroll
        for (int j = 0; j < BJ; ++j) x[j] &= m;
      }
#pragma unroll
      for (int i = 0; i < WI; ++i) {
        const u32x4 w = __builtin_bit_cast(u32x4, ld128(base + arow + uint32_t(i) * 2048 + ch));
#pragma unroll
        for (int j = 0; j < BJ; ++j) acc[i][j] = mfma_i8(w, x[j], acc[i][j]);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < ST - 1; ++i)
    if (i < n) issue(i, i);
  int st = 0;
  // every wave takes part in the barriers of the first group's n blocks
  const int steps = (nkb + KG - 1) / KG;
  auto step = [&](int i, bool last) {
    if (i < n) wait_ring<LW + LB, ST - 2>(n - 1 - i);  // this wave's loads of block i have landed
    lds_barrier();                                     // every wave's have; block i - 1 is no longer read
    if (i + ST - 1 < n) issue(i + ST - 1, st == 0 ? ST - 1 : st - 1);
    if (!last || i < n) multiply(ring + uint32_t(st) * kStage, last && a.cols % 128 != 0 && i * KG + group == nkb - 1);
    st = st + 1 == ST ? 0 : st + 1;
  };
  for (int i = 0; i < steps - 1; ++i) step(i, false);  // every group has these
  step(steps - 1, true);
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
        for (int j = 0; j < BJ; ++j)
          acc[i][j] += __builtin_bit_cast(i32x4, ld128(uint32_t(g * kPartial) + mine + uint32_t(i * BJ + j) * 1024));
  }
  store_through_lds<WI, BJ, YBF16, NT>(a, row0 + ww * 16 * WI, b0 + wb * BJ * 16,
                                       uint32_t((KG - 1) * kPartial + wave * epilogue_bytes<WI, YBF16>), lane, acc);
}

// Operands of any alignment, many rows: as i8_stage_kernel, but a block's
// 16-byte pieces go through registers (gfx950 loads them from any byte) and
// into the other of two LDS buffers, one block ahead of the products.  Rows
// may start at any byte; nothing outside a row is read.
// Bound by the loads: off a 16-byte boundary they take a lane per cycle, 0.5 us
// per 16 KB and compute unit (4096 x 14336 x 4099: 427 us, against 5865 for 32
// x 32 tiles in i8_direct_kernel; at a stride of 4112, staged: 293).  Eight
// waves beat four (64 x 14336 x 4099, operands partly in the last-level cache:
// 19.9 us against 23.2; all from memory 27.1); two to four blocks ahead
// changed nothing, nor did words loaded on a 4-byte boundary and shifted.
template <int BW, int BB, int WGW, int WGB, bool YBF16>
__global__ __launch_bounds__(64 * WGW * WGB) void i8_loose_kernel(I8Args a, int nw_tiles, int nb_tiles, int per_xcd) {
  constexpr int NW = WGW * WGB;
  constexpr int WI = BW / WGW / 16, BJ = BB / WGB / 16;
  constexpr int LW = BW / 8 / NW, LB = BB / 8 / NW, L = LW + LB;
  constexpr uint32_t kWBytes = BW * 128, kStage = (BW + BB) * 128;
  static_assert(BW % (8 * NW) == 0 && BB % (8 * NW) == 0, "whole loads");
  static_assert(NW * epilogue_bytes<WI, YBF16> <= 2 * int(kStage), "LDS");
  const int id = int(blockIdx.x % kXcds) * per_xcd + int(blockIdx.x / kXcds);
  if (id >= nw_tiles * nb_tiles) return;  // whole workgroups
  constexpr int kDeep = 4;
  const int strip = id / (kDeep * nw_tiles);
  const int deep = min(kDeep, nb_tiles - strip * kDeep);
  const int in = id - strip * kDeep * nw_tiles;
  const int64_t row0 = int64_t(in / deep) * BW, b0 = (int64_t(strip) * kDeep + in % deep) * BB;
  const int lane = int(threadIdx.x) % kWave, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int lrow = lane / 8, lchunk = (lane % 8) ^ lrow;
  const int8_t* from[L];  // rows past the last are the last one again
  uint32_t to[L];
#pragma unroll
  for (int u = 0; u < L; ++u) {
    const bool w = u < LW;
    const int at = (w ? u : u - LW) * NW + wave;
    const int64_t row = std::min<int64_t>((w ? row0 : b0) + 8 * at + lrow, (w ? a.rows : a.batch) - 1);
    from[u] = (w ? a.W : a.X) + row * (w ? a.ldw : a.ldx) + 16 * lchunk;
    to[u] = (w ? 0u : kWBytes) + uint32_t(at) * 1024 + 16 * lane;
  }
  const int r = lane % 16, q = lane / 16;
  const int ww = wave / WGB, wb = wave % WGB;
  const uint32_t arow = uint32_t(ww * WI * 16 + r) * 128, xrow = kWBytes + uint32_t(wb * BJ * 16 + r) * 128;
  i32x4 acc[WI][BJ];
#pragma unroll
  for (int i = 0; i < WI; ++i)
#pragma unroll
    for (int j = 0; j < BJ; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  const int nkb = int((a.cols + 127) / 128), nfull = int(a.cols / 128);
  u32x4 v[L];
  auto load = [&](int kb) {
    const int64_t k = int64_t(kb) * 128;
    if (kb < nfull) {
#pragma unroll
      for (int u = 0; u < L; ++u) v[u] = load16_any(from[u] + k);
    } else if (kb < nkb) {
#pragma unroll
      for (int u = 0; u < L; ++u) v[u] = load16_tail(from[u] + k, a.cols - k - 16 * lchunk);
    }
  };
  auto store = [&](uint32_t base) {
#pragma unroll
    for (int u = 0; u < L; ++u) st128(base + to[u], __builtin_bit_cast(uint4, v[u]));
  };
  load(0);
  store(0);
  load(1);
  for (int kb = 0; kb < nkb; ++kb) {
    const uint32_t base = uint32_t(kb & 1) * kStage;
    lds_barrier();  // block kb is in LDS; block kb - 1 is no longer read
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t ch = uint32_t(((4 * s + q) ^ (r & 7)) * 16);
      u32x4 x[BJ];
#pragma unroll
      for (int j = 0; j < BJ; ++j) x[j] = __builtin_bit_cast(u32x4, ld128(base + xrow + uint32_t(j) * 2048 + ch));
#pragma unroll
      for (int i = 0; i < WI; ++i) {
        const u32x4 w = __builtin_bit_cast(u32x4, ld128(base + arow + uint32_t(i) * 2048 + ch));
#pragma unroll
        for (int j = 0; j < BJ; ++j) acc[i][j] = mfma_i8(w, x[j], acc[i][j]);
      }
    }
    if (kb + 1 < nkb) {
      store(kStage - base);
      load(kb + 2);
    }
  }
  __syncthreads();  // no wave reads the buffers any more
  store_through_lds<WI, BJ, YBF16, false>(a, row0 + ww * 16 * WI, b0 + wb * BJ * 16,
                                          uint32_t(wave) * epilogue_bytes<WI, YBF16>, lane, acc);
}

// The largest batches.  As above with the operands of the next step read
// between this step's products: WGW x WGB waves (two per SIMD: one alone
// issues the 16 x 16 products at 0.85 of the rate), steps of 64 bytes of k, one
// barrier per step; the slot a step's operands came from is refilled while
// its products run, so ST steps are in flight.
// Bound by power: with operands of zeros 4096 x 4096 x 16384 runs in 153 us
// (3.6 POP/s, 4.0 inside the loop), with random ones in 202 to 227 us (2.7 to
// 2.4 POP/s from run to run), the clock falling from 2.3 to about 1.8 GHz;
// products alone, operands held in registers, reach 3.4 POP/s on random
// values.  Where this took 202 us, 32 x 32 products (twice the accumulator
// traffic per operation) took 265, four waves with the 16 x 16 form 241, the
// kernel above at 256 x 256 219.
template <int BW, int BB, int WGW, int WGB, int ST, bool YBF16, bool NT>
__global__ __launch_bounds__(64 * WGW * WGB) void i8_wide_kernel(I8Args a, int nw_tiles, int nb_tiles, int per_xcd) {
  constexpr int NW = WGW * WGB;
  constexpr int WI = BW / WGW / 16, BJ = BB / WGB / 16;  // 16 x 16 tiles of a wave
  constexpr int LW = BW / 16 / NW, LB = BB / 16 / NW, L = LW + LB;  // 1 KB loads (16 rows) per wave and step
  constexpr int G = WI + BJ, M = WI * BJ;                // operand reads and products per step
  constexpr uint32_t kWBytes = BW * 64, kStep = (BW + BB) * 64;
  static_assert(BW % (16 * NW) == 0 && BB % (16 * NW) == 0, "whole loads");
  static_assert(ST * kStep <= kLdsLimit && ST >= 3 && M >= 2 * G && M >= 4 * L, "ring");
  const int id = int(blockIdx.x % kXcds) * per_xcd + int(blockIdx.x / kXcds);
  if (id >= nw_tiles * nb_tiles) return;  // whole workgroups
  constexpr int kDeep = 4;
  const int strip = id / (kDeep * nw_tiles);
  const int deep = min(kDeep, nb_tiles - strip * kDeep);
  const int in = id - strip * kDeep * nw_tiles;
  const int64_t row0 = int64_t(in / deep) * BW, b0 = (int64_t(strip) * kDeep + in % deep) * BB;
  const int lane = int(threadIdx.x) % kWave, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int lrow = lane / 4, lchunk = (lane % 4) ^ ((lrow >> 1) & 3);
  const Staged tw(a.W + row0 * a.ldw, a.rows - row0, a.cols, a.ldw, BW);
  const Staged tx(a.X + b0 * a.ldx, a.batch - b0, a.cols, a.ldx, BB);
  uint32_t vo[L];
#pragma unroll
  for (int u = 0; u < LW; ++u) vo[u] = tw.row_offset(16 * (u * NW + wave) + lrow, a.ldw) + 16 * lchunk;
#pragma unroll
  for (int u = 0; u < LB; ++u) vo[LW + u] = tx.row_offset(16 * (u * NW + wave) + lrow, a.ldx) + 16 * lchunk;
  const int n = int((a.cols + 63) / 64);
  const int over = max(0, 16 * (lchunk - (int(a.cols - 1) % 64) / 16));
  auto issue = [&](int u, int t, int slot, bool last) {
    const uint32_t dst = uint32_t(slot) * kStep + (u < LW ? uint32_t(u * NW + wave) * 1024 : kWBytes + uint32_t((u - LW) * NW + wave) * 1024);
    stage_load<false>(u < LW ? tw.rsrc : tx.rsrc, vo[u] - (last ? over : 0), uint32_t(t) * 64, dst);
  };
  const int r = lane % 16, q = lane / 16;
  const int ww = wave / WGB, wb = wave % WGB;
  const uint32_t chunk = uint32_t((q ^ ((r >> 1) & 3)) * 16);
  const uint32_t arow = uint32_t(ww * WI * 16 + r) * 64 + chunk, xrow = kWBytes + uint32_t(wb * BJ * 16 + r) * 64 + chunk;
  i32x4 acc[WI][BJ];
#pragma unroll
  for (int i = 0; i < WI; ++i)
#pragma unroll
    for (int j = 0; j < BJ; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  u32x4 f0[G], f1[G];  // a step's operands: BJ of the activations, WI of the weights
  auto read = [&](int g, int slot, u32x4 (&f)[G]) {
    const uint32_t base = uint32_t(slot) * kStep;
    f[g] = __builtin_bit_cast(u32x4, ld128(g < BJ ? base + xrow + uint32_t(g) * 1024 : base + arow + uint32_t(g - BJ) * 1024));
  };
#pragma unroll
  for (int t = 0; t < ST; ++t)
    if (t < n) {
#pragma unroll
      for (int u = 0; u < L; ++u) issue(u, t, t, t == n - 1);
    }
  wait_ring<L, ST - 1>(n - 1);
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int g = 0; g < G; ++g) read(g, 0, f0);
  int slot = 0;
  auto step = [&](int t, const u32x4 (&fc)[G], u32x4 (&fn)[G], bool steady) {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): fc is in registers
    const bool more = steady || t + 1 < n, refill = steady || t + ST < n;
    if (more) {
      wait_ring<L, ST - 2>(steady ? ST - 2 : n - 2 - t);  // this wave's loads of step t + 1 have landed
      asm volatile("s_barrier" ::: "memory");             // every wave's have, and every wave holds step t
    }
    const int next = slot + 1 == ST ? 0 : slot + 1;
#pragma unroll
    for (int g = 0; g < M; ++g) {
      if (more && g % 2 == 0 && g / 2 < G) read(g / 2, next, fn);
      if (refill && g % 4 == 1 && g / 4 < L) issue(g / 4, t + ST, slot, !steady && t + ST == n - 1);
      const int i = g / BJ, j = g % BJ;
      acc[i][j] = mfma_i8(fc[BJ + i], fc[j], acc[i][j]);
      if (g % 2 == 1) __builtin_amdgcn_sched_barrier(0);
    }
    slot = next;
  };
  int t = 0;
  for (; t + ST + 2 < n; t += 2) {
    step(t, f0, f1, true);
    step(t + 1, f1, f0, true);
  }
  auto mask = [&](int t, u32x4 (&f)[G]) {
    if (t != n - 1 || a.cols % 64 == 0) return;
    const u32x4 m = tail_mask(int(a.cols - int64_t(t) * 64) - 16 * q);
#pragma unroll
    for (int j = 0; j < BJ; ++j) f[j] &= m;
  };
  for (; t < n; t += 2) {
    mask(t, f0);
    step(t, f0, f1, false);
    if (t + 1 >= n) break;
    mask(t + 1, f1);
    step(t + 1, f1, f0, false);
  }
  static_assert(NW * epilogue_bytes<WI, YBF16> <= ST * int(kStep), "LDS");
  __syncthreads();  // no wave reads the ring any more
  store_through_lds<WI, BJ, YBF16, NT>(a, row0 + ww * 16 * WI, b0 + wb * BJ * 16,
                                       uint32_t(wave) * epilogue_bytes<WI, YBF16>, lane, acc);
}

// A launch holds fewer than 2^32 threads: nw x nb tiles, rounded up to a
// multiple of kXcds.  In double: sizes below 2^40 make products past 64 bits.
int check_launch(int64_t nw, int64_t nb, int threads) {
  if ((double(nw) * double(nb) + kXcds) * threads < 4294967296.0) return UW_OK;
  return fail(UW_ERR_UNSUPPORTED, "uw_i8_gemm: too many tiles for one launch");
}

int run_direct(const I8Args& a, int yt, int ks, hipStream_t s) {
  const int64_t n_groups = (a.rows + 15) / 16, ny = (a.batch + 15) / 16;
  if (int rc = check_launch((n_groups + kXcds - 1) / kXcds * kXcds, ny, ks * kWave)) return rc;
  const int64_t grid = (n_groups + kXcds - 1) / kXcds * kXcds * ny;
  auto kern = yt == UW_BF16 ? i8_direct_kernel<true> : i8_direct_kernel<false>;
  hipLaunchKernelGGL(kern, dim3(unsigned(grid)), dim3(ks * kWave), size_t(ks) * 1024, s, a, int(n_groups), int(ny), ks);
  return hip_check(hipGetLastError(), "i8_direct_kernel launch");
}

// Whether every row of Y starts at a 128-byte line.
bool whole_lines(const I8Args& a, int yt) {
  return reinterpret_cast<uintptr_t>(a.Y) % 128 == 0 && a.ldy * int64_t(elem_size(yt)) % 128 == 0;
}

template <int BW, int BB, int WGW, int WGB, int ST, int KG = 1>
int run_stage(const I8Args& a, int yt, hipStream_t s) {
  const int64_t nw = (a.rows + BW - 1) / BW, nb = (a.batch + BB - 1) / BB;
  constexpr int kThreads = 64 * WGW * WGB * KG;
  if (int rc = check_launch(nw, nb, kThreads)) return rc;
  const int64_t per_xcd = (nw * nb + kXcds - 1) / kXcds;
  auto kern = whole_lines(a, yt)
                  ? (yt == UW_BF16 ? i8_stage_kernel<BW, BB, WGW, WGB, ST, KG, true, true> : i8_stage_kernel<BW, BB, WGW, WGB, ST, KG, false, true>)
                  : (yt == UW_BF16 ? i8_stage_kernel<BW, BB, WGW, WGB, ST, KG, true, false> : i8_stage_kernel<BW, BB, WGW, WGB, ST, KG, false, false>);
  allow_full_lds(kern);
  hipLaunchKernelGGL(kern, dim3(unsigned(per_xcd * kXcds)), dim3(kThreads), size_t(KG) * ST * (BW + BB) * 128, s, a, int(nw),
                     int(nb), int(per_xcd));
  return hip_check(hipGetLastError(), "i8_stage_kernel launch");
}

template <int BW, int BB, int KW, int ST>
int run_slice(const I8Args& a, int yt, hipStream_t s) {
  const int64_t nw = (a.rows + BW - 1) / BW, nb = (a.batch + BB - 1) / BB;
  if (int rc = check_launch((nw + kXcds - 1) / kXcds * kXcds, nb, KW * kWave)) return rc;
  const int64_t grid = (nw + kXcds - 1) / kXcds * kXcds * nb;
  // weights that one workgroup reads once pass the caches by
  auto kern = nb == 1 ? (yt == UW_BF16 ? i8_slice_kernel<BW, BB, KW, ST, true, true> : i8_slice_kernel<BW, BB, KW, ST, true, false>)
                      : (yt == UW_BF16 ? i8_slice_kernel<BW, BB, KW, ST, false, true> : i8_slice_kernel<BW, BB, KW, ST, false, false>);
  allow_full_lds(kern);
  constexpr size_t kLds = std::max(size_t(KW) * ST * (BW + BB) * 128, size_t(KW) * BW * BB * 4);
  static_assert(kLds <= kLdsLimit, "LDS");
  hipLaunchKernelGGL(kern, dim3(unsigned(grid)), dim3(KW * kWave), kLds, s, a, int(nw), int(nb));
  return hip_check(hipGetLastError(), "i8_slice_kernel launch");
}

template <int BW, int BB, int WGW, int WGB>
int run_loose(const I8Args& a, int yt, hipStream_t s) {
  const int64_t nw = (a.rows + BW - 1) / BW, nb = (a.batch + BB - 1) / BB;
  constexpr int kThreads = 64 * WGW * WGB;
  if (int rc = check_launch(nw, nb, kThreads)) return rc;
  const int64_t per_xcd = (nw * nb + kXcds - 1) / kXcds;
  auto kern = yt == UW_BF16 ? i8_loose_kernel<BW, BB, WGW, WGB, true> : i8_loose_kernel<BW, BB, WGW, WGB, false>;
  allow_full_lds(kern);
  hipLaunchKernelGGL(kern, dim3(unsigned(per_xcd * kXcds)), dim3(kThreads), size_t(2) * (BW + BB) * 128, s, a, int(nw),
                     int(nb), int(per_xcd));
  return hip_check(hipGetLastError(), "i8_loose_kernel launch");
}

template <int BW, int BB, int WGW, int WGB, int ST>
int run_wide(const I8Args& a, int yt, hipStream_t s) {
  const int64_t nw = (a.rows + BW - 1) / BW, nb = (a.batch + BB - 1) / BB;
  constexpr int kThreads = 64 * WGW * WGB;
  if (int rc = check_launch(nw, nb, kThreads)) return rc;
  const int64_t per_xcd = (nw * nb + kXcds - 1) / kXcds;
  auto kern = whole_lines(a, yt)
                  ? (yt == UW_BF16 ? i8_wide_kernel<BW, BB, WGW, WGB, ST, true, true> : i8_wide_kernel<BW, BB, WGW, WGB, ST, false, true>)
                  : (yt == UW_BF16 ? i8_wide_kernel<BW, BB, WGW, WGB, ST, true, false> : i8_wide_kernel<BW, BB, WGW, WGB, ST, false, false>);
  allow_full_lds(kern);
  hipLaunchKernelGGL(kern, dim3(unsigned(per_xcd * kXcds)), dim3(kThreads), size_t(ST) * (BW + BB) * 64, s, a, int(nw),
                     int(nb), int(per_xcd));
  return hip_check(hipGetLastError(), "i8_wide_kernel launch");
}

// Shapes: weight and batch rows of a workgroup's tile, and how its operands
// reach the matrix cores: straight from global memory or through registers and
// LDS (both for any alignment), in slices that each wave stages for itself, or
// staged for all waves.  per_cu workgroups fit a compute unit (by their LDS);
// start, alone and shared are us, for expected_us below.
enum Kind { kDirect, kLoose, kSlice, kStage };
struct I8Shape {
  int bw, bb;
  Kind kind;
  int per_cu;
  float start, alone, shared;
};
constexpr I8Shape kShapeList[] = {
    {0, 0, kDirect, 1, 0, 0, 0},  // 0: the choice below
    {16, 16, kDirect, 1, 0, 0, 0},
    {64, 64, kLoose, 1, 0, 0, 0},
    {128, 128, kLoose, 1, 0, 0, 0},
    {16, 16, kSlice, 2, 1.55f, 0.052f, 0.056f},
    {64, 16, kSlice, 2, 1.75f, 0.157f, 0.145f},
    {16, 32, kSlice, 1, 1.58f, 0.083f, 0.068f},
    {32, 32, kSlice, 2, 1.79f, 0.119f, 0.118f},
    {64, 32, kSlice, 1, 2.54f, 0.198f, 0.107f},
    {32, 32, kStage, 5, 1.53f, 0.219f, 0.138f},
    {32, 64, kStage, 3, 1.70f, 0.252f, 0.191f},
    {64, 64, kStage, 4, 1.65f, 0.490f, 0.295f},
    {64, 64, kStage, 1, 2.32f, 0.228f, 0.236f},    // 3 groups of waves
    {64, 128, kStage, 1, 2.86f, 0.347f, 0.379f},   // 2 groups
    {128, 128, kStage, 2, 3.86f, 0.756f, 0.597f},  // 2 slots
    {128, 128, kStage, 1, 3.80f, 0.623f, 0.517f},  // 3 slots
    {128, 128, kStage, 1, 4.05f, 0.560f, 0.560f},  // 2 groups
    {256, 128, kStage, 1, 4.48f, 1.040f, 0.941f},
    {256, 256, kStage, 1, 8.17f, 1.313f, 1.729f},
};
constexpr int kShapes = int(sizeof(kShapeList) / sizeof(kShapeList[0]));
constexpr int kFirstStaged = 4;
constexpr int kCus = 256;

bool stage_ok(const I8Args& a) {
  // 16-byte chunks, and 32-bit offsets inside a tile of 256 rows
  return reinterpret_cast<uintptr_t>(a.W) % 16 == 0 && reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && a.ldw % 16 == 0 &&
         a.ldx % 16 == 0 && a.ldw < (int64_t(1) << 22) && a.ldx < (int64_t(1) << 22);
}

// What a product takes on a shape, in us: 1.6 for the launch, then rounds of
// workgroups.  Each round costs `start` (first loads, epilogue) and `alone` per
// 128-byte block of k where a workgroup waits on its own loads; a compute unit
// needs `shared` per block and workgroup it holds; and the operands' bytes come
// at 5.4 TB/s.  The three limits of the loop add as fourth powers (the largest
// rules, a near second counts).
// The constants were fitted to the shapes' times on sizes drawn over 1..4096 x
// 64..28672 x 64..14336 (and the MLP's), each on 3 to 8 rotated operand sets.
// Only their order counts: the times themselves are up to a quarter off.  On
// 2373 other sizes of that range the choice takes 1.026 of the best shape's
// time in the mean (95 of 100 under 1.15, the worst 2.2: 2618 x 141 x 8032),
// against 1.47 for the best single shape.
float expected_us(const I8Shape& s, int64_t rows, int64_t cols, int64_t batch) {
  const float blocks = float((cols + 127) / 128);
  const float n = float((rows + s.bw - 1) / s.bw) * float((batch + s.bb - 1) / s.bb) / kCus;
  const float rounds = std::ceil(n / float(s.per_cu));
  const float held = n < 1.f ? n : 0.5f * (n + std::ceil(n));
  const auto p4 = [](float v) { return v * v * v * v; };
  const float loop = p4(blocks * s.alone * rounds) + p4(blocks * s.shared * held) +
                     p4(float(rows + batch) * blocks * (128.f / 5.4e6f));
  return 1.6f + s.start * rounds + std::sqrt(std::sqrt(loop));
}

// Operands that can be staged run the shape expected to be fastest.  Of the
// others, the smallest tile of which a compute unit gets at most two, or the
// largest: 1.035 of the best shape's time in the mean of 4034 sizes drawn as
// above at odd strides (95 of 100 under 1.23, the worst 2.6: 1655 x 64 x 14289;
// always 64 x 64: 1.16, always 128 x 128: 1.69).
int pick_shape(int64_t rows, int64_t cols, int64_t batch, bool staged) {
  if (!staged) {
    for (int i = 1; i < kFirstStaged - 1; ++i) {
      const I8Shape& s = kShapeList[i];
      if ((rows + s.bw - 1) / s.bw * ((batch + s.bb - 1) / s.bb) <= 2 * kCus) return i;
    }
    return kFirstStaged - 1;
  }
  int shape = kFirstStaged;
  float best = expected_us(kShapeList[shape], rows, cols, batch);
  for (int i = shape + 1; i < kShapes; ++i) {
    const float us = expected_us(kShapeList[i], rows, cols, batch);
    if (us < best) {
      best = us;
      shape = i;
    }
  }
  return shape;
}

}  // namespace

int i8_gemm_shape_count() { return kShapes; }

bool i8_gemm_shape_ok(const int8_t* W, int64_t rows, int64_t ldw, const int8_t* X, int64_t batch, int64_t ldx, int shape) {
  I8Args a{};
  a.W = W;
  a.X = X;
  a.ldw = rows > 1 ? ldw : 0;
  a.ldx = batch > 1 ? ldx : 0;
  return shape < kFirstStaged || stage_ok(a);
}

int launch_i8_gemm(const int8_t* W, int64_t rows, int64_t cols, int64_t ldw, const float* sw, const int8_t* X,
                   int64_t batch, int64_t ldx, const float* sx, const float* bias, void* Y, int64_t ldy, int yt,
                   int shape, int ks, void* stream) {
  // a single row has no stride
  const I8Args a{W, sw, X, sx, bias, static_cast<char*>(Y), rows, cols, rows > 1 ? ldw : 0, batch, batch > 1 ? ldx : 0, ldy};
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (shape <= 0) shape = pick_shape(rows, cols, batch, stage_ok(a));
  if (ks <= 0) ks = int(std::min<int64_t>(8, (cols + 255) / 256));
  switch (shape) {
    case 1: return run_direct(a, yt, ks, s);
    case 2: return run_loose<64, 64, 4, 2>(a, yt, s);
    case 3: return run_loose<128, 128, 4, 2>(a, yt, s);
    case 4: return run_slice<16, 16, 8, 2>(a, yt, s);
    case 5: return run_slice<64, 16, 4, 2>(a, yt, s);
    case 6: return run_slice<16, 32, 4, 4>(a, yt, s);
    case 7: return run_slice<32, 32, 4, 2>(a, yt, s);
    case 8: return run_slice<64, 32, 4, 2>(a, yt, s);
    case 9: return run_stage<32, 32, 2, 2, 4>(a, yt, s);
    case 10: return run_stage<32, 64, 2, 2, 4>(a, yt, s);
    case 11: return run_stage<64, 64, 2, 2, 2>(a, yt, s);
    case 12: return run_stage<64, 64, 2, 2, 3, 3>(a, yt, s);
    case 13: return run_stage<64, 128, 2, 2, 3, 2>(a, yt, s);
    case 14: return run_stage<128, 128, 2, 2, 2>(a, yt, s);
    case 15: return run_stage<128, 128, 2, 2, 3>(a, yt, s);
    case 16: return run_stage<128, 128, 2, 2, 2, 2>(a, yt, s);
    case 17: return run_stage<256, 128, 4, 2, 3>(a, yt, s);
    default: return run_wide<256, 256, 2, 4, 4>(a, yt, s);
  }
}

}  // namespace uw
