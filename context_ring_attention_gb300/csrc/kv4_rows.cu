// Writing rows into the 4-bit cache and reading them back.
//
// Per group of 32 channels (include/ra.h): low = bf16(min), scale = bf16((max - low) * 1/15),
// code = floor((x - low)/scale + 1/2), value = low + scale * code.  Both kernels are bound
// by HBM: a token and head move 2 * d * sizeof(T) bytes of rows and 2 * d * 5/8 of cache.
//
// One thread holds 8 consecutive channels of a key or value row: the 8 nibbles of one
// 32-bit word of key codes, or two 16-bit words of value codes; four threads share a
// group, and its minimum and maximum take two exchanges among them.  A warp takes a run of
// tokens of one head, all their loads first, and counts its place in the cache on from
// token to token.  What bounds a plain form is not memory but the arithmetic of a code
// (190 instructions a row and thread, 76% of the issue slots, are left), so it is kept to
// about a dozen: rounding by adding 1.5 * 2^23, codes packed by a multiply-add each, pairs
// of values by one instruction, and the exact decision taken only next to a border of two
// codes.
//
// Measured (bf16, d = 128, 32768 tokens of 8 heads): write 55 us for 134 MB of rows and
// 42 MB of cache, 3.2 TB/s; read 27 us for the same bytes, 6.5 TB/s.  float32, 16384 tokens
// (134 MB of rows, 21 MB of cache): write 40 us, read 26.  Pairs by one instruction took the
// write from 62 us to 59.5, a quotient by 15 without a division to 57.5 (the product that the
// format has now was not timed against it alone), and 64 registers, for four CTAs an SM instead
// of three, to 54.  The read loads words
// of two groups and exchanges halves (by 16-bit loads it took 37 us, so 31) and makes floats
// of codes by one byte permutation each and pairs of values by one instruction.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kv4_internal.h"
#include "sm100_ptx.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;

// Rows of sequence b that take part: count[b], or all.  A count out of range is reported
// and takes none.
__device__ __forceinline__ int32_t live_rows(const Kv4RowsParams& p, int b) {
  if (p.count == nullptr) return p.rows;
  const int32_t n = __ldg(p.count + b);
  if (n >= 0 && n <= p.rows) return n;
  atomicOr(p.t.status, kKv4StatusRange);
  return 0;
}

// The 8 values of a thread as they come from memory.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* src) { w = __ldcs(reinterpret_cast<const uint4*>(src)); }
  __device__ __forceinline__ void clear() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(a[i] << 16);
      x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* src) {
    a = __ldcs(reinterpret_cast<const float4*>(src));
    b = __ldcs(reinterpret_cast<const float4*>(src) + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&x)[8]);
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* dst, const float (&x)[8]) {
  __stcs(reinterpret_cast<uint4*>(dst), make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]),
                                                   ptx::pack_bf16x2(x[4], x[5]), ptx::pack_bf16x2(x[6], x[7])));
}
template <>
__device__ __forceinline__ void store8<float>(float* dst, const float (&x)[8]) {
  __stcs(reinterpret_cast<float4*>(dst), make_float4(x[0], x[1], x[2], x[3]));
  __stcs(reinterpret_cast<float4*>(dst) + 1, make_float4(x[4], x[5], x[6], x[7]));
}

__device__ __forceinline__ float bf16_round(float x) { return __uint_as_float(ptx::pack_bf16x2(x, 0.f) << 16); }

// 1.5 * 2^23: a float of magnitude below 2^22 added to it is rounded to an integer, which
// stands in the sum's low bits.
constexpr float kRound = 12582912.f;
constexpr uint32_t kRoundBits = 0x4B400000u;
// The constant's share in the sum over i = 0..7 of bits(r_i) * 16^i, in 32 bits.
constexpr uint32_t kRoundShare = kRoundBits * 0x11111111u;

// Code of x, decided exactly where the quotient lies next to a border of two codes.
// d + e is x - low without error (the two terms of a floating-point sum); the quotient
// d * inv is off by 2^-21 of itself at most, so its floor is right or one off, and
// r = d - c * scale is exact: c * scale has 12 bits, and the difference is a multiple of
// the last place of d and smaller than d.
__device__ __noinline__ uint32_t code_at_border(float x, float low, float scale, float inv) {
  const float d = x - low;
  const float bb = d - x;
  const float e = (x - (d - bb)) + (-low - bb);
  float c = floorf(fmaf(d, inv, 0.5f));
  c = fminf(fmaxf(c, 0.f), 15.f);
  const float r = fmaf(-c, scale, d), half = 0.5f * scale;
  if ((r - half) + e >= 0.f) c += 1.f;
  else if ((r + half) + e < 0.f) c -= 1.f;
  return (uint32_t)fminf(fmaxf(c, 0.f), 15.f);
}

// The 8 codes of a thread, first in the lowest nibble: float32 rows, whose low is a rounded
// minimum, so that a quotient may lie outside 0..15 and d is seldom exact.  Codes off the
// borders are sure from the approximate quotient.
__device__ __forceinline__ uint32_t codes_near(const float (&x)[8], float low, float scale, float inv) {
  uint32_t word = 0, near_any = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float v = fminf(fmaxf((x[i] - low) * inv, 0.f), 15.f);
    const float r = v + kRound;
    const float off = v - (r - kRound);
    near_any |= (fabsf(off) > 0.5f - 0x1p-14f) ? 1u << i : 0u;
    word = word * 16u + __float_as_uint(r);  // (the constant's share is taken off below)
  }
  word -= kRoundShare;
  while (near_any) {
    const int i = __ffs(near_any) - 1;
    near_any &= near_any - 1;
    float xi = x[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) xi = k == i ? x[k] : xi;
    word = (word & ~(15u << (4 * i))) | (code_at_border(xi, low, scale, inv) << (4 * i));
  }
  return word;
}

// Two fp32 operations by one instruction.
__device__ __forceinline__ uint64_t pair_bits(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 pair_of(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)), "l"(pair_bits(c)));
  return pair_of(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return pair_of(r);
}

// bf16 rows: low is the minimum itself, so that no quotient lies below 0, and the scale's
// rounding takes none above 15.03.  The quotient is taken a little low (2^-20 of itself,
// more than its error), which leaves one question, whether x - low reaches the border above
// the code.  It is answered by r = d - c * scale, an exact difference, where d = x - low has
// not been rounded across a border.  d + low == x says so where |low| >= |x| or low <= 0: d is
// x - low itself, or rounded away from low; between the two lies no number of x's 8 bits or of
// a border's 13, except x, which x - low reaches as d does.  A positive low may be lost without
// a trace, d = x, where x itself is a border that x - low does not reach: it is below 2^-24 * x
// then, and x below 16 scales, so that groups of 0 < low < 2^-16 * scale, and values that fail
// the test (exponents more than 16 apart), are left to the path above.  Ties are common among
// bf16 values and cost nothing here.
__device__ __forceinline__ uint32_t codes_bf16(const float (&x)[8], float low, float scale, float inv) {
  const float half = 0.5f * scale, under = inv * (1.f - 0x1p-20f);
  const float2 low2 = {low, low}, under2 = {under, under}, scale2 = {scale, scale}, round2 = {kRound, kRound};
  const float2 minus2 = {-1.f, -1.f};
  uint32_t word = 0;
  bool exact = !(low > 0.f && low < scale * 0x1p-16f);
#pragma unroll
  for (int i = 6; i >= 0; i -= 2) {  // two at a time, by the paired fp32 instructions
    const float2 xi = {x[i], x[i + 1]};
    const float2 d = fma2(low2, minus2, xi), again = add2(d, low2);
    exact = exact && again.x == x[i] && again.y == x[i + 1];
    float2 r = fma2(d, under2, round2);
    const float2 rest = fma2(fma2(r, minus2, round2), scale2, d);
    if (rest.x >= half) r.x += 1.f;
    if (rest.y >= half) r.y += 1.f;
    word = word * 16u + __float_as_uint(r.y);
    word = word * 16u + __float_as_uint(r.x);
  }
  return exact ? word - kRoundShare : codes_near(x, low, scale, inv);
}

template <typename T>
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float low, float scale) {
  if (!(scale > 0.f)) return 0u;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));  // (2^-100 <= scale: no underflow)
  return sizeof(T) == 2 ? codes_bf16(x, low, scale, inv) : codes_near(x, low, scale, inv);
}

__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Minimum and maximum of the 8 values of each of four neighbouring lanes.  The maximum
// passes a NaN on, and an infinity makes the range infinite: either way the scale is not
// finite.
__device__ __forceinline__ void group_bounds(const Raw<float>& raw, float& lo, float& hi) {
  float x[8];
  raw.values(x);
  lo = min3_nan(min3_nan(x[0], x[1], x[2]), min3_nan(x[3], x[4], x[5]), fminf(x[6], x[7]));
  hi = max3_nan(max3_nan(x[0], x[1], x[2]), max3_nan(x[3], x[4], x[5]), max3_nan(x[6], x[7], x[7]));
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    const float h = __shfl_xor_sync(0xffffffffu, hi, o);
    hi = max3_nan(hi, h, h);
  }
}
// bf16 rows: by pairs, the exchanges on the minimum and the maximum's negative together.
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void group_bounds(const Raw<__nv_bfloat16>& raw, float& lo, float& hi) {
  const uint32_t l2 = min2_nan(min2_nan(raw.w.x, raw.w.y), min2_nan(raw.w.z, raw.w.w));
  const uint32_t h2 = max2_nan(max2_nan(raw.w.x, raw.w.y), max2_nan(raw.w.z, raw.w.w)) ^ 0x80008000u;
  uint32_t both = min2_nan(__byte_perm(l2, h2, 0x5410), __byte_perm(l2, h2, 0x7632));
  both = min2_nan(both, __shfl_xor_sync(0xffffffffu, both, 1));
  both = min2_nan(both, __shfl_xor_sync(0xffffffffu, both, 2));
  lo = __uint_as_float(both << 16);
  hi = -__uint_as_float(both & 0xffff0000u);
}

// A group's scale and low: zeros for a scale below 2^-100, NaN for low where the range is not finite.
__device__ __forceinline__ void params_of(float lo, float hi, float& scale, float& low) {
  low = bf16_round(lo);
  constexpr float kFifteenth = 1.f / 15.f;  // (part of the format: the product is rounded, not a quotient)
  scale = bf16_round((hi - low) * kFifteenth);
  if (!(fabsf(scale) <= 3.402823466e38f)) {
    scale = 0.f;
    low = __uint_as_float(0x7fff0000u);  // NaN
  } else if (scale < 7.888609052e-31f) {  // 2^-100
    scale = 0.f;
  }
}

// Thread layout of a row pair (the K and the V row of one token and head): D/8 lanes for
// K, then D/8 for V.
template <typename T, int D>
struct Lanes {
  static constexpr int kRow = D / 8;            // lanes of a row
  static constexpr int kPair = D / 4;           // lanes of a token and head: 32 or 16
  static constexpr int kAtOnce = 32 / kPair;    // tokens of a warp at a time
  static constexpr int kSteps = sizeof(T) == 2 ? 8 : 4;
  static constexpr int kRun = kAtOnce * kSteps;  // tokens of a warp
};

// The run of tokens of one sequence and head that a warp takes, and the lane's place in it.
// The place is counted on from token to token; the page table is asked once a page.
template <typename T, int D>
struct Run {
  using L = Lanes<T, D>;
  static constexpr int kBlockBytes = Kv4Block<D>::kBytes;
  const Kv4Table& tb;
  bool any;          // the warp has a token
  int b, h, t;       // the lane's current token t; the next one is kAtOnce further
  int live;          // tokens of the sequence that take part
  int64_t row;       // row of the first token in [batch, heads, rows]
  uint8_t* base;     // block of the current token (nullptr: out of range)
  int row16;         // its row there
  int blocks;        // blocks from there to the page's end
  int64_t page_at;   // place in the page table (-1: before the first position)

  __device__ __forceinline__ explicit Run(const Kv4RowsParams& P) : tb(P.t) {
    const int lane = threadIdx.x & 31;
    const uint32_t per = (uint32_t)(P.rows + L::kRun - 1) / L::kRun;  // runs of a sequence and head
    const uint32_t id = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const uint32_t bh = id / per;
    any = bh < (uint32_t)P.t.batch * (uint32_t)P.t.heads_kv;
    b = any ? (int)(bh / (uint32_t)P.t.heads_kv) : 0;
    h = (int)(bh - (uint32_t)b * (uint32_t)P.t.heads_kv);
    t = (int)(id - bh * per) * L::kRun + lane / L::kPair;
    live = any ? live_rows(P, b) : 0;
    row = (int64_t)bh * P.rows + t;
    base = nullptr;
    row16 = blocks = 0;
    page_at = -1;
    if (t >= live) return;
    const int32_t f = __ldg(P.first + b);
    int32_t in_page = 0;
    if (f >= 0) {
      const uint32_t pos = (uint32_t)f + (uint32_t)t;  // (below 2^32)
      page_at = pos / (uint32_t)tb.page_rows;
      in_page = (int32_t)(pos - (uint32_t)page_at * (uint32_t)tb.page_rows);
    }
    row16 = in_page % kKvBlockRows;
    turn(in_page / kKvBlockRows);
  }
  // Look the current page up; its current block is number `block`.
  __device__ __forceinline__ void turn(int block) {
    int32_t page = -1;
    if (page_at >= 0 && page_at < tb.width) page = __ldg(tb.page_table + (int64_t)b * tb.width + page_at);
    base = nullptr;
    blocks = tb.blocks_per_page - block;
    if (page < 0 || page >= tb.pages) atomicOr(tb.status, kKv4StatusRange);
    else base = tb.cache + (((int64_t)page * tb.heads_kv + h) * tb.blocks_per_page + block) * kBlockBytes;
    RA_BOUNDS(tb.status, b >= 0 && b < tb.batch && h >= 0 && h < tb.heads_kv && block >= 0 && block < tb.blocks_per_page, 90);
  }
  // The current place, and the row of [batch, heads, rows] that goes with it, exist.
  __device__ __forceinline__ bool sound(int32_t rows) const {
    return in_pool<D>(tb, base) && row16 >= 0 && row16 < kKvBlockRows && t >= 0 && t < rows;
  }
  __device__ __forceinline__ void advance() {
    t += L::kAtOnce;
    row16 += L::kAtOnce;
    if (row16 < kKvBlockRows) return;
    row16 -= kKvBlockRows;
    if (--blocks > 0) {
      if (base != nullptr) base += kBlockBytes;
    } else if (t < live) {
      if (page_at >= 0) ++page_at;
      turn(0);
    }
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 1)
    kv4_write_kernel(const Kv4RowsParams P, const T* __restrict__ k, const T* __restrict__ v) {
  using L = Lanes<T, D>;
  using F = Kv4Block<D>;
  constexpr int G = F::kGroups;
  Run<T, D> run(P);
  if (!run.any) return;  // (whole warps)
  const int at = threadIdx.x % L::kPair;
  const bool is_v = at >= L::kRow;
  const int i8 = at % L::kRow;  // channels 8*i8 .. 8*i8 + 7
  const int g = i8 / 4, c = i8 % 4;
  const T* src = (is_v ? v : k) + run.row * D + i8 * 8;
  Raw<T> raw[L::kSteps];
#pragma unroll
  for (int n = 0; n < L::kSteps; ++n)
    if (run.t + n * L::kAtOnce < run.live) {
      RA_BOUNDS(P.t.status, run.row >= 0 && run.row + n * L::kAtOnce < (int64_t)P.t.batch * P.t.heads_kv * P.rows, 91);
      raw[n].load(src + (int64_t)n * L::kAtOnce * D);
    } else {
      raw[n].clear();
    }
  // Values: a lane holds the 16-bit words of chunks 2c (low half) and 2c + 1 (high half)
  // for group g; with the lane of the neighbouring group (4 lanes on) it makes whole 32-bit
  // words: the even group's lane chunk 2c, the odd group's chunk 2c + 1.
  const uint32_t at_word = is_v ? (2 * c + (g & 1)) * (G / 2) + g / 2 : c * G + g;
#pragma unroll
  for (int n = 0; n < L::kSteps; ++n) {
    if (__all_sync(0xffffffffu, run.t >= run.live)) break;
    float x[8];
    raw[n].values(x);
    float lo, hi, scale, low;
    group_bounds(raw[n], lo, hi);  // (every lane takes part in the exchanges)
    params_of(lo, hi, scale, low);
    uint32_t word = codes_of<T>(x, low, scale);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, word, 4);
    if (run.t < run.live && run.base != nullptr) {
      uint8_t* blk = run.base;
      RA_BOUNDS(P.t.status, run.sound(P.rows) && at_word < F::kCodeBytes / 4 && g < G, 92);
      if (is_v) word = (g & 1) ? (other >> 16) | (word & 0xffff0000u) : (word & 0xffffu) | (other << 16);
      reinterpret_cast<uint32_t*>(blk + (is_v ? F::kOffV : F::kOffK) + run.row16 * F::kCodeBytes)[at_word] = word;
      if (c == 0)
        reinterpret_cast<uint32_t*>(blk + (is_v ? F::kOffVPar : F::kOffKPar) + run.row16 * F::kParBytes)[g] =
            (__float_as_uint(scale) >> 16) | (__float_as_uint(low) & 0xffff0000u);
    }
    run.advance();
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 5 : 1) kv4_read_kernel(const Kv4RowsParams P, T* __restrict__ k, T* __restrict__ v) {
  using L = Lanes<T, D>;
  using F = Kv4Block<D>;
  constexpr int G = F::kGroups;
  Run<T, D> run(P);
  if (!run.any) return;
  const int at = threadIdx.x % L::kPair;
  const bool is_v = at >= L::kRow;
  const int i8 = at % L::kRow, g = i8 / 4, c = i8 % 4;
  T* dst = (is_v ? v : k) + run.row * D + i8 * 8;
  const int t0 = run.t;
  // (the words as the write puts them together: the even group's lane has chunk 2c of both
  // groups, the odd one's chunk 2c + 1)
  const uint32_t at_word = is_v ? (2 * c + (g & 1)) * (G / 2) + g / 2 : c * G + g;
  uint32_t word[L::kSteps], par[L::kSteps];
  uint32_t have = 0;  // steps whose token is read
#pragma unroll
  for (int n = 0; n < L::kSteps; ++n) {
    word[n] = par[n] = 0;
    if (run.t < run.live && run.base != nullptr) {
      have |= 1u << n;
      RA_BOUNDS(P.t.status, run.sound(P.rows) && at_word < F::kCodeBytes / 4 && g < G, 93);
      const uint8_t* codes = run.base + (is_v ? F::kOffV : F::kOffK) + run.row16 * F::kCodeBytes;
      word[n] = reinterpret_cast<const uint32_t*>(codes)[at_word];
      par[n] = reinterpret_cast<const uint32_t*>(run.base + (is_v ? F::kOffVPar : F::kOffKPar) + run.row16 * F::kParBytes)[g];
    }
    run.advance();
  }
#pragma unroll
  for (int n = 0; n < L::kSteps; ++n) {
    const bool in = t0 + n * L::kAtOnce < P.rows;
    if (!__any_sync(0xffffffffu, in)) break;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, word[n], 4);
    if (is_v) word[n] = (g & 1) ? (other >> 16) | (word[n] & 0xffff0000u) : (word[n] & 0xffffu) | (other << 16);
    const float scale = __uint_as_float(par[n] << 16), low = __uint_as_float(par[n] & 0xffff0000u);
    float x[8];
    const uint32_t even = word[n] & 0x0f0f0f0fu, odd = (word[n] >> 4) & 0x0f0f0f0fu;  // codes 2i and 2i + 1 in byte i
    const float2 scale2 = {scale, scale}, low2 = {low, low}, minus = {-8388608.f, -8388608.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // 2^23 + code, without a conversion: the code's byte below 0x4B0000
      const float2 f = {__uint_as_float(__byte_perm(even, 0x4B000000u, 0x7550u + i)),
                        __uint_as_float(__byte_perm(odd, 0x4B000000u, 0x7550u + i))};
      const float2 y = fma2(scale2, add2(f, minus), low2);
      x[2 * i] = y.x;
      x[2 * i + 1] = y.y;
    }
    RA_BOUNDS(P.t.status, !in || (run.row >= 0 && run.row + n * L::kAtOnce < (int64_t)P.t.batch * P.t.heads_kv * P.rows), 94);
    if (in && (((have >> n) & 1u) || P.zero_rest)) store8<T>(dst + (int64_t)n * L::kAtOnce * D, x);
  }
}

template <typename T, int D>
unsigned grid_of(const Kv4RowsParams& prm) {
  const int64_t run = Lanes<T, D>::kRun, warps = kThreads / 32;
  const int64_t runs = (int64_t)prm.t.batch * prm.t.heads_kv * ((prm.rows + run - 1) / run);
  return (unsigned)((runs + warps - 1) / warps);
}

template <typename T, int D>
cudaError_t write_as(const Kv4RowsParams& prm, const void* k, const void* v, cudaStream_t st) {
  kv4_write_kernel<T, D><<<grid_of<T, D>(prm), kThreads, 0, st>>>(prm, static_cast<const T*>(k), static_cast<const T*>(v));
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t read_as(const Kv4RowsParams& prm, void* k, void* v, cudaStream_t st) {
  kv4_read_kernel<T, D><<<grid_of<T, D>(prm), kThreads, 0, st>>>(prm, static_cast<T*>(k), static_cast<T*>(v));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_write(int dtype, int head_dim, const Kv4RowsParams& prm, const void* k, const void* v,
                             cudaStream_t stream) {
  if (dtype == RA_DTYPE_BF16)
    return head_dim == 128 ? write_as<__nv_bfloat16, 128>(prm, k, v, stream)
                           : write_as<__nv_bfloat16, 64>(prm, k, v, stream);
  return head_dim == 128 ? write_as<float, 128>(prm, k, v, stream) : write_as<float, 64>(prm, k, v, stream);
}

cudaError_t launch_kv4_read(int dtype, int head_dim, const Kv4RowsParams& prm, void* k, void* v, cudaStream_t stream) {
  if (dtype == RA_DTYPE_BF16)
    return head_dim == 128 ? read_as<__nv_bfloat16, 128>(prm, k, v, stream)
                           : read_as<__nv_bfloat16, 64>(prm, k, v, stream);
  return head_dim == 128 ? read_as<float, 128>(prm, k, v, stream) : read_as<float, 64>(prm, k, v, stream);
}

}  // namespace ra
