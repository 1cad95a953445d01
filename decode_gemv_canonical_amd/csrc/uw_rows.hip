// Row operators around the products: the root-mean-square norm with the
// residual's addition, the gated activation silu(g) * u, and rows in 8-bit
// integers with one scale per row (what uw_i8_gemm multiplies).
//
// Mathematics.  For one row of `cols` values:
//   norm:  h = x + r, rounded to r's type where it is kept (h is what the
//          next layer adds to), rstd = 1 / sqrt(mean(h^2) + eps),
//          p = h * gain, y = p * rstd;
//   silu:  p = g / (1 + exp(-g)) * u, y = p;
//   8 bits of a row p: s = max(max|p| / 127, 2^-126), q = p * (1 / s) rounded
//          to the nearest integer (ties to even), scale = s (times rstd for
//          the norm).  rstd is common to the row, so q does not depend on it:
//          the sum of squares and the maximum come from one reduction, and
//          the payload is the same whatever the order of the sum.  2^-126 (the
//          smallest normal fp32) keeps 1 / s finite for rows of zeros.  A row
//          that holds an infinity or a NaN gets q = 0 and scale = NaN, so that
//          everything multiplied with it is NaN, as in the unquantised form.
//
// A row is held in registers from its one read to its write: chunks of 8
// values, chunk t + j * NT on thread t, NT threads per row and VPT chunks per
// thread, so x (and r, u, gain) are read once and every output written once.
// Every load is issued before the first is used.  Sums of squares are fp32:
// the 8 of a chunk, a lane's chunks (at most 4; any number, in fp64, in the
// form for long rows), lanes and waves, so that no square passes more than 8 +
// 3 + 6 + 15 = 32 roundings.  Loads and stores are 16 bytes (8 for the
// integers) at any element alignment: gfx950 takes them unaligned, and a row's
// last chunk goes element by element.
#include <algorithm>

#include "uw_device.h"

namespace uw {
namespace {

enum RowOp { kNorm = 0, kSilu = 1, kQuantize = 2 };
enum RowType { kF32 = UW_F32, kBf16 = UW_BF16, kNone = -1 };

constexpr float kTiny = 1.17549435e-38f;  // 2^-126

// 8 values as they lie in memory: one 16-byte word in bf16, two in fp32.
struct Raw8 {
  u32x4 a, b;
};

__device__ __forceinline__ u32x4 load16_any(const char* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// Values [i, i + 8) of a row of n; those past the end read as zero and their
// addresses are not touched.
template <int T>
__device__ __forceinline__ Raw8 load8(const char* row, int64_t i, int64_t n) {
  Raw8 v{u32x4{0u, 0u, 0u, 0u}, u32x4{0u, 0u, 0u, 0u}};
  if (T == kNone || i >= n) return v;
  const char* p = row + i * (T == kF32 ? 4 : 2);
  if (i + 8 <= n) {
    v.a = load16_any(p);
    if (T == kF32) v.b = load16_any(p + 16);
    return v;
  }
  const int m = int(n - i);
  uint32_t w[7];  // all loads before the first use
#pragma unroll
  for (int e = 0; e < 7; ++e) w[e] = 0u;
#pragma unroll
  for (int e = 0; e < 7; ++e) {
    if (e < m) {
      if (T == kF32) __builtin_memcpy(&w[e], p + 4 * e, 4);
      else __builtin_memcpy(&w[e], p + 2 * e, 2);
    }
  }
#pragma unroll
  for (int e = 0; e < 7; ++e) {
    if (T != kF32) v.a[e / 2] |= w[e] << (16 * (e & 1));
    else if (e < 4) v.a[e] = w[e];
    else v.b[e - 4] = w[e];
  }
  return v;
}

template <int T>
__device__ __forceinline__ void unpack8(const Raw8& r, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (T == kF32) f[e] = bits_f32(e < 4 ? r.a[e] : r.b[e - 4]);
    else f[e] = bits_f32((e & 1) ? (r.a[e / 2] & 0xFFFF0000u) : (r.a[e / 2] << 16));
  }
}

// 16 bytes at any element alignment; past: non-temporally.
__device__ __forceinline__ void store16_any(void* p, const u32x4& v, bool past) {
  typedef uint32_t any4 __attribute__((ext_vector_type(4), aligned(2)));
  const any4 w{v.x, v.y, v.z, v.w};
  if (past) __builtin_nontemporal_store(w, static_cast<any4*>(p));
  else *static_cast<any4*>(p) = w;
}

// Values [i, i + 8) of a row of n, written as bf16 or fp32.
__device__ __forceinline__ void store8(char* row, int type, int64_t i, int64_t n, const float (&f)[8], bool past = false) {
  if (i >= n) return;
  if (type == UW_F32) {
    float* p = reinterpret_cast<float*>(row) + i;
    if (i + 8 <= n) {
      store16_any(p, u32x4{f32_bits(f[0]), f32_bits(f[1]), f32_bits(f[2]), f32_bits(f[3])}, past);
      store16_any(p + 4, u32x4{f32_bits(f[4]), f32_bits(f[5]), f32_bits(f[6]), f32_bits(f[7])}, past);
      return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (i + e < n) p[e] = f[e];
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
  uint16_t* p = reinterpret_cast<uint16_t*>(row) + i;
  if (i + 8 <= n) {
    store16_any(p, u32x4{w[0], w[1], w[2], w[3]}, past);
    return;
  }
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (i + e < n) p[e] = uint16_t(w[e / 2] >> (16 * (e & 1)));
}

// q = rint(p * inv) of 8 values, |p * inv| <= 127: adding 1.5 * 2^23 rounds to
// the nearest integer, ties to even, and leaves it in the low byte.
__device__ __forceinline__ void store_q8(int8_t* row, int64_t i, int64_t n, const float (&p)[8], float inv, bool fine) {
#pragma clang fp contract(off)  // the product is rounded before the sum: an fma would round once
  if (i >= n) return;
  uint32_t b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) b[e] = f32_bits(p[e] * inv + 12582912.f);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x0C0C0400u);
    w[h] = fine ? (lo | (hi << 16)) : 0u;
  }
  if (i + 8 <= n) {
    __builtin_memcpy(row + i, w, 8);
    return;
  }
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (i + e < n) row[i + e] = int8_t(w[e / 4] >> (8 * (e & 3)));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 0xF, 0xF, false)));
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x4E, 0xF, 0xF, false)));
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x141, 0xF, 0xF, false)));
  v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x140, 0xF, 0xF, false)));
  const uint32_t a = __builtin_amdgcn_readlane(int(v), 0), b = __builtin_amdgcn_readlane(int(v), 16);
  const uint32_t c = __builtin_amdgcn_readlane(int(v), 32), d = __builtin_amdgcn_readlane(int(v), 48);
  return max(max(a, b), max(c, d));
}

// Sum and maximum over the NT threads of a row; every thread gets both.
template <int NT>
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& top) {
  sum = wave_sum(sum);
  top = wave_max(top);
  if (NT == kWave) return;
  __shared__ float s_sum[16];
  __shared__ uint32_t s_top[16];
  const int wave = int(threadIdx.x) / kWave;
  if (threadIdx.x % kWave == 0) {
    s_sum[wave] = sum;
    s_top[wave] = top;
  }
  lds_barrier();  // h's stores stay in flight (1111 x 8192, fp32 stream: 24.7 -> 24.3 us)
  sum = s_sum[0];
  top = s_top[0];
#pragma unroll
  for (int i = 1; i < NT / kWave; ++i) {
    sum += s_sum[i];
    top = max(top, s_top[i]);
  }
}

// 112 bytes: with 120 every launch took 0.4 us longer.
struct RowArgs {
  const char* x;
  const char* r;  // the residual (norm) or u (silu)
  const char* gain;
  char* h;  // x + r, in r's type; may be null
  char* y;
  float* scale;  // 8-bit outputs
  int64_t rows, cols, ldx, ldr, ldh, ldy;  // strides in elements
  float eps, inv_cols;
  int8_t gt, yt;
  bool h_past;  // h is stored past the caches
};

// A stream of this many bytes is not read again before other data has taken
// its place in the caches: stored past them, it leaves them to what the norm
// reads and to y, which the next product reads (1111 x 8192, fp32 stream: 24.0
// -> 19.6 us, 25.1 -> 24.1 with cold inputs; 2048 x 4096, bf16: 18.2 -> 17.9
// with the dequantize behind it).  y itself stored so is slower to read next.
constexpr int64_t kStreamPast = int64_t(16) << 20;

// exp(-g) = 2^t, t = -g log2(e): 2^t from the transcendental unit (1 ulp),
// times 2^d for what the rounding of t lost, d = (-g log2(e)) - t with log2(e)
// in two parts, to first order (|d| < 2^-16 for |t| < 126).  Past |t| = 126
// the correction would be lost in 1 + exp(-g), or meet an infinity.
__device__ __forceinline__ float exp_neg(float g) {
  constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f, kLn2 = 0.693147182f;  // log2(e) = kHi + kLo
  const float t = -g * kHi;
  const float d = fmaf(-g, kLo, fmaf(-g, kHi, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fabsf(t) < 126.f ? fmaf(e, d * kLn2, e) : e;
}

// silu(g) * u for g < kSiluFar, where 1 + exp(-g) nears 2^126 and its
// reciprocal would be flushed to zero: there g exp(g) u, the exponential held
// as 2^160 times its value, so that a large u finds all of its bits.
constexpr float kSiluFar = -87.f;
__device__ __forceinline__ float silu_far(float g, float u) {
#pragma clang fp contract(off)  // t is rounded before 160 is added: d is what that rounding lost
  constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f, kLn2 = 0.693147182f;  // as in exp_neg
  const float c = fmaxf(g, -300.f);  // exp(-300) * 2^160 is zero in fp32, and t stays finite
  const float t = c * kHi, d = fmaf(c, kLo, fmaf(c, kHi, -t));
  const float e = __builtin_amdgcn_exp2f(t + 160.f);  // the sum is exact
  return __builtin_amdgcn_ldexpf(g * fmaf(e, d * kLn2, e) * (u * 0x1p-64f), -96);
}

// One chunk's p = h * gain (norm; h is also rounded, kept and squared),
// silu(g) * u, or x.  Inlined twice: held in registers, or computed again.
template <int OP, int XT, int RT>
__device__ __forceinline__ void chunk_p(const RowArgs& a, const Raw8& xr, const Raw8& rr, const Raw8& gr, float (&p)[8],
                                        char* hrow, int64_t i, float& sum) {
  unpack8<XT>(xr, p);
  if (OP == kNorm) {
    if (RT != kNone) {
      float r[8];
      unpack8<RT>(rr, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] += r[e];
      if (RT == kBf16) {
        // the norm reads what the next layer will: h as it is kept
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = static_cast<float>(static_cast<__bf16>(p[e]));
      }
      if (hrow) store8(hrow, RT, i, a.cols, p, a.h_past);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(p[e], p[e], sum);
    if (a.gain) {
      float g[8];
      if (a.gt == UW_F32) unpack8<kF32>(gr, g);
      else unpack8<kBf16>(gr, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] *= g[e];
    }
  } else if (OP == kSilu) {
    float u[8];
    unpack8<XT>(rr, u);
    uint32_t far = 0u;  // as unsigned numbers, only large negative values (and NaN) lie past kSiluFar
#pragma unroll
    for (int e = 0; e < 8; ++e) far = max(far, f32_bits(p[e]));
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = p[e] * __builtin_amdgcn_rcpf(1.f + exp_neg(p[e])) * u[e];
    if (far > f32_bits(kSiluFar)) {
      float g[8];
      unpack8<XT>(xr, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = g[e] < kSiluFar ? silu_far(g[e], u[e]) : p[e];
    }
  }
}

__device__ __forceinline__ Raw8 load_gain(const RowArgs& a, int64_t i) {
  if (a.gt == UW_F32) return load8<kF32>(a.gain, i, a.gain ? a.cols : 0);
  return load8<kBf16>(a.gain, i, a.gain ? a.cols : 0);
}

// s and 1 / s of an 8-bit row from max|p|'s bits; whether the row is finite.
__device__ __forceinline__ bool row_scale(uint32_t top, float& s, float& inv) {
  s = fmaxf(bits_f32(top) / 127.f, kTiny);
  inv = 1.f / s;
  return top < 0x7F800000u;
}

template <int OP, int XT, int RT, bool I8, int NT, int VPT>
__global__ __launch_bounds__(NT == kWave ? 256 : NT) void row_kernel(RowArgs a) {
  constexpr int kRowsPer = NT == kWave ? 4 : 1;
  constexpr int kXs = XT == kF32 ? 4 : 2, kRs = RT == kF32 ? 4 : 2;
  const int t = int(threadIdx.x) % NT;
  const int64_t row = int64_t(blockIdx.x) * kRowsPer + (NT == kWave ? int(threadIdx.x) / kWave : 0);
  if (row >= a.rows) return;  // whole waves, and no barrier follows where a workgroup holds several rows
  const char* x = a.x + row * a.ldx * kXs;
  const char* r = a.r + row * a.ldr * kRs;
  char* h = a.h ? a.h + row * a.ldh * kRs : nullptr;
  Raw8 xr[VPT], rr[VPT] = {}, gr[VPT] = {};
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int64_t i = 8 * (t + int64_t(j) * NT);
    xr[j] = load8<XT>(x, i, a.cols);
    if (RT != kNone) rr[j] = load8<RT>(r, i, a.cols);
    if (OP == kNorm) gr[j] = load_gain(a, i);
  }
  float p[VPT][8];
  float sum = 0.f;
  uint32_t top = 0u;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float part = 0.f;
    chunk_p<OP, XT, RT>(a, xr[j], rr[j], gr[j], p[j], h, 8 * (t + int64_t(j) * NT), part);
    sum += part;
    if (I8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, f32_bits(p[j][e]) & 0x7FFFFFFFu);
    }
  }
  float rstd = 1.f;
  if (OP == kNorm || I8) row_reduce<NT>(sum, top);
  if (OP == kNorm) rstd = 1.f / sqrtf(fmaf(sum, a.inv_cols, a.eps));
  if (I8) {
    float s, inv;
    const bool fine = row_scale(top, s, inv);
    int8_t* q = reinterpret_cast<int8_t*>(a.y) + row * a.ldy;
#pragma unroll
    for (int j = 0; j < VPT; ++j) store_q8(q, 8 * (t + int64_t(j) * NT), a.cols, p[j], inv, fine);
    if (t == 0) a.scale[row] = fine ? s * rstd : bits_f32(0x7FC00000u);
  } else {
    char* y = a.y + row * a.ldy * (a.yt == UW_F32 ? 4 : 2);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[j][e] *= rstd;
      store8(y, a.yt, 8 * (t + int64_t(j) * NT), a.cols, p[j]);
    }
  }
}

// silu(g) * u without scales has nothing to reduce: a row is spread over
// workgroups, one chunk per thread (one row of 14336: 3.5 us held in one
// workgroup, whose compute unit the exponentials keep busy for 1 us, 2.1 here).
template <int XT>
__global__ __launch_bounds__(256) void silu_kernel(RowArgs a, unsigned per_row) {
  constexpr int kXs = XT == kF32 ? 4 : 2;
  const int64_t row = blockIdx.x / per_row, i = 8 * (int64_t(blockIdx.x % per_row) * 256 + threadIdx.x);
  if (i >= a.cols) return;
  const Raw8 xr = load8<XT>(a.x + row * a.ldx * kXs, i, a.cols), ur = load8<XT>(a.r + row * a.ldr * kXs, i, a.cols);
  float p[8], unused = 0.f;
  chunk_p<kSilu, XT, XT>(a, xr, ur, Raw8{}, p, nullptr, i, unused);
  store8(a.y + row * a.ldy * (a.yt == UW_F32 ? 4 : 2), a.yt, i, a.cols, p);
}

// Rows past the register form's 32768 values: two passes over the row, the
// second reading h back where it was kept (r may have been overwritten by
// it) and computing it again where not.
template <int OP, int XT, int RT, bool I8>
__global__ __launch_bounds__(1024) void long_row_kernel(RowArgs a) {
  constexpr int NT = 1024;
  constexpr int kXs = XT == kF32 ? 4 : 2, kRs = RT == kF32 ? 4 : 2;
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x;
  const char* x = a.x + row * a.ldx * kXs;
  const char* r = a.r + row * a.ldr * kRs;
  char* h = a.h ? a.h + row * a.ldh * kRs : nullptr;
  double squares = 0.;  // a lane's chunks: fp32 lost 220 half steps of y over 2^24 equal values
  uint32_t top = 0u;
  for (int64_t i = 8 * t; i < a.cols; i += 8 * NT) {
    Raw8 rr{}, gr{};
    const Raw8 xr = load8<XT>(x, i, a.cols);
    if (RT != kNone) rr = load8<RT>(r, i, a.cols);
    if (OP == kNorm) gr = load_gain(a, i);
    float p[8], part = 0.f;
    chunk_p<OP, XT, RT>(a, xr, rr, gr, p, h, i, part);
    if (OP == kNorm) squares += double(part);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, f32_bits(p[e]) & 0x7FFFFFFFu);
  }
  float sum = float(squares);
  row_reduce<NT>(sum, top);
  const float rstd = OP == kNorm ? 1.f / sqrtf(fmaf(sum, a.inv_cols, a.eps)) : 1.f;
  float s, inv;
  const bool fine = row_scale(top, s, inv);
  for (int64_t i = 8 * t; i < a.cols; i += 8 * NT) {
    Raw8 rr{}, gr{};
    float p[8], unused = 0.f;
    if (OP == kNorm) gr = load_gain(a, i);
    if (OP == kNorm && RT != kNone && h) {
      chunk_p<OP, RT, kNone>(a, load8<RT>(h, i, a.cols), rr, gr, p, nullptr, i, unused);
    } else {
      const Raw8 xr = load8<XT>(x, i, a.cols);
      if (RT != kNone) rr = load8<RT>(r, i, a.cols);
      chunk_p<OP, XT, RT>(a, xr, rr, gr, p, nullptr, i, unused);
    }
    if (I8) {
      store_q8(reinterpret_cast<int8_t*>(a.y) + row * a.ldy, i, a.cols, p, inv, fine);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] *= rstd;
      store8(a.y + row * a.ldy * (a.yt == UW_F32 ? 4 : 2), a.yt, i, a.cols, p);
    }
  }
  if (I8 && t == 0) a.scale[row] = fine ? s * rstd : bits_f32(0x7FC00000u);
}

template <int OP, int XT, int RT, bool I8>
int run_rows(const RowArgs& a, hipStream_t s) {
  const int64_t chunks = (a.cols + 7) / 8;
  // a launch holds fewer than 2^32 threads: bands of 2^21 rows
  constexpr int64_t kBand = int64_t(1) << 21;
  constexpr int kXs = XT == kF32 ? 4 : 2, kRs = RT == kF32 ? 4 : 2;
  auto go = [&](auto kern, int threads, int rows_per) {
    for (int64_t row0 = 0; row0 < a.rows; row0 += kBand) {
      RowArgs b = a;
      b.rows = std::min(kBand, a.rows - row0);
      b.x += row0 * a.ldx * kXs;
      if (b.r) b.r += row0 * a.ldr * kRs;
      if (b.h) b.h += row0 * a.ldh * kRs;
      b.y += row0 * a.ldy * (I8 ? 1 : a.yt == UW_F32 ? 4 : 2);
      if (I8) b.scale += row0;
      hipLaunchKernelGGL(kern, dim3(unsigned((b.rows + rows_per - 1) / rows_per)), dim3(threads), 0, s, b);
      if (int rc = hip_check(hipGetLastError(), "row_kernel launch")) return rc;
    }
    return int(UW_OK);
  };
  // as many threads as there are chunks, to have every load of a row in flight at once: one row of 4096 takes 2.7 us
  // with 512 threads, 3.1 with 256; 1111 rows of 8192 (fp32 stream) 26.5 with 1024, 29.2 to 31.2 with fewer.  Where
  // thousands of rows keep the card full anyway, two chunks a thread: 14336 x 4096 to 8 bits 33.0 against 34.5
  if (chunks <= 64) return go(row_kernel<OP, XT, RT, I8, 64, 1>, 256, 4);
  if (chunks <= 128) return go(row_kernel<OP, XT, RT, I8, 64, 2>, 256, 4);
  if (chunks <= 256) return go(row_kernel<OP, XT, RT, I8, 256, 1>, 256, 1);
  if (chunks <= 512 && a.rows > 1024) return go(row_kernel<OP, XT, RT, I8, 256, 2>, 256, 1);
  if (chunks <= 512) return go(row_kernel<OP, XT, RT, I8, 512, 1>, 512, 1);
  if (chunks <= 1024) return go(row_kernel<OP, XT, RT, I8, 1024, 1>, 1024, 1);
  if (chunks <= 2048) return go(row_kernel<OP, XT, RT, I8, 1024, 2>, 1024, 1);
  if (chunks <= 4096) return go(row_kernel<OP, XT, RT, I8, 1024, 4>, 1024, 1);
  return go(long_row_kernel<OP, XT, RT, I8>, 1024, 1);
}

// Rows a launch takes where each is spread over per_row workgroups of 256: a
// launch holds fewer than 2^32 threads.  0: not even one.
int64_t band_rows(int64_t per_row) { return ((int64_t(1) << 24) - 1) / per_row; }

template <int XT>
int run_silu(const RowArgs& a, hipStream_t s) {
  constexpr int kXs = XT == kF32 ? 4 : 2;
  const int64_t per_row = (a.cols + 2047) / 2048, band = band_rows(per_row);
  if (band == 0) return fail(UW_ERR_UNSUPPORTED, "uw_silu_mul: a row wider than a launch holds");
  for (int64_t row0 = 0; row0 < a.rows; row0 += band) {
    RowArgs b = a;
    b.rows = std::min(band, a.rows - row0);
    b.x += row0 * a.ldx * kXs;
    b.r += row0 * a.ldr * kXs;
    b.y += row0 * a.ldy * int64_t(elem_size(a.yt));
    hipLaunchKernelGGL(silu_kernel<XT>, dim3(unsigned(b.rows * per_row)), dim3(256), 0, s, b, unsigned(per_row));
    if (int rc = hip_check(hipGetLastError(), "silu_kernel launch")) return rc;
  }
  return UW_OK;
}

template <int OP, int XT, int RT>
int run_out(const RowArgs& a, hipStream_t s) {
  return a.yt == UW_I8 ? run_rows<OP, XT, RT, true>(a, s) : run_rows<OP, XT, RT, false>(a, s);
}

// Integers back to values: 16 per thread, v = q * scale[row].
__global__ __launch_bounds__(256) void dequantize_kernel(const int8_t* __restrict__ Q, int64_t cols, int64_t ldq,
                                                         const float* __restrict__ scale, char* __restrict__ Y,
                                                         int64_t ldy, int yt, unsigned per_row) {
  const int64_t row = blockIdx.x / per_row;
  const int64_t i = 16 * (int64_t(blockIdx.x % per_row) * 256 + threadIdx.x);
  if (i >= cols) return;
  const int8_t* q = Q + row * ldq + i;
  const float s = scale[row];
  u32x4 v{0u, 0u, 0u, 0u};
  if (i + 16 <= cols) {
    v = load16_any(reinterpret_cast<const char*>(q));
  } else {
#pragma unroll
    for (int e = 0; e < 15; ++e)
      if (i + e < cols) v[e / 4] |= uint32_t(uint8_t(q[e])) << (8 * (e & 3));
  }
  char* y = Y + row * ldy * (yt == UW_F32 ? 4 : 2);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = float(int32_t(v[2 * h + e / 4] << (24 - 8 * (e & 3))) >> 24) * s;
    store8(y, yt, i + 8 * h, cols, f);
  }
}

}  // namespace

int launch_rmsnorm(const void* X, int64_t batch, int64_t cols, int64_t ldx, int xt, const void* R, int64_t ldr, int rt,
                   void* H, int64_t ldh, const void* gain, int gt, float eps, void* Y, int64_t ldy, int yt,
                   float* scale, void* stream) {
  RowArgs a{static_cast<const char*>(X), static_cast<const char*>(R), static_cast<const char*>(gain),
            static_cast<char*>(H), static_cast<char*>(Y), scale, batch, cols, ldx, ldr, ldh, ldy, eps,
            float(1.0 / double(cols)), int8_t(gt), int8_t(yt), batch * cols * int64_t(elem_size(rt)) >= kStreamPast};
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!R) return xt == UW_F32 ? run_out<kNorm, kF32, kNone>(a, s) : run_out<kNorm, kBf16, kNone>(a, s);
  if (rt == UW_F32) return xt == UW_F32 ? run_out<kNorm, kF32, kF32>(a, s) : run_out<kNorm, kBf16, kF32>(a, s);
  return xt == UW_F32 ? run_out<kNorm, kF32, kBf16>(a, s) : run_out<kNorm, kBf16, kBf16>(a, s);
}

int launch_silu_mul(const void* G, int64_t ldg, const void* U, int64_t ldu, int xt, int64_t batch, int64_t cols,
                    void* Y, int64_t ldy, int yt, float* scale, void* stream) {
  RowArgs a{static_cast<const char*>(G), static_cast<const char*>(U), nullptr, nullptr, static_cast<char*>(Y), scale,
            batch, cols, ldg, ldu, 0, ldy, 0.f, 0.f, 0, int8_t(yt), false};
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (yt != UW_I8) return xt == UW_F32 ? run_silu<kF32>(a, s) : run_silu<kBf16>(a, s);
  return xt == UW_F32 ? run_rows<kSilu, kF32, kF32, true>(a, s) : run_rows<kSilu, kBf16, kBf16, true>(a, s);
}

int launch_i8_quantize(const void* X, int64_t rows, int64_t cols, int64_t ldx, int xt, int8_t* Q, int64_t ldq,
                       float* scale, void* stream) {
  RowArgs a{static_cast<const char*>(X), nullptr, nullptr, nullptr, reinterpret_cast<char*>(Q), scale, rows, cols, ldx,
            0, 0, ldq, 0.f, 0.f, 0, UW_I8, false};
  hipStream_t s = static_cast<hipStream_t>(stream);
  return xt == UW_F32 ? run_rows<kQuantize, kF32, kNone, true>(a, s) : run_rows<kQuantize, kBf16, kNone, true>(a, s);
}

int launch_i8_dequantize(const int8_t* Q, int64_t rows, int64_t cols, int64_t ldq, const float* scale, void* Y,
                         int64_t ldy, int yt, void* stream) {
  const int64_t per_row = (cols + 4095) / 4096, band = band_rows(per_row);
  if (band == 0) return fail(UW_ERR_UNSUPPORTED, "uw_i8_dequantize: a row wider than a launch holds");
  for (int64_t row0 = 0; row0 < rows; row0 += band) {
    const int64_t n = std::min(band, rows - row0);
    hipLaunchKernelGGL(dequantize_kernel, dim3(unsigned(n * per_row)), dim3(256), 0, static_cast<hipStream_t>(stream),
                       Q + row0 * ldq, cols, ldq, scale + row0,
                       static_cast<char*>(Y) + row0 * ldy * int64_t(elem_size(yt)), ldy, yt, unsigned(per_row));
    if (int rc = hip_check(hipGetLastError(), "dequantize_kernel launch")) return rc;
  }
  return UW_OK;
}

}  // namespace uw
