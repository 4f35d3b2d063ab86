// Writing rows into the 4-bit cache and reading them back.
//
// Per group of 32 channels (include/ra.h): low = bf16(min), scale = bf16((max - low)/15),
// code = floor((x - low)/scale + 1/2), value = low + scale * code.  Both kernels are bound
// by HBM: a token and head move 2 * d * sizeof(T) bytes of rows and 2 * d * 5/8 of cache.
//
// One thread holds 8 consecutive channels of a key or value row: the 8 nibbles of one
// 32-bit word of key codes, or two 16-bit words of value codes; four threads share a
// group, and its minimum and maximum take two exchanges among them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kv4_internal.h"
#include "sm100_ptx.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;

// Place of position `pos` of sequence b: the byte offset of its block for head h, or -1
// (out of range, reported through the status word).
__device__ __forceinline__ int64_t block_of(const Kv4Table& t, int b, int h, int64_t pos, int block_bytes) {
  const int64_t page_at = pos / t.page_rows;
  int32_t page = -1;
  if (pos >= 0 && page_at < t.width) page = __ldg(t.page_table + (int64_t)b * t.width + page_at);
  if (page < 0 || page >= t.pages) {
    atomicOr(t.status, kKv4StatusRange);
    return -1;
  }
  const int32_t block = (int32_t)(pos % t.page_rows) / kKvBlockRows;
  return (((int64_t)page * t.heads_kv + h) * t.blocks_per_page + block) * block_bytes;
}

// Rows of sequence b that take part: count[b], or all.  A count out of range is reported
// and takes none.
__device__ __forceinline__ int32_t live_rows(const Kv4RowsParams& p, int b) {
  if (p.count == nullptr) return p.rows;
  const int32_t n = __ldg(p.count + b);
  if (n >= 0 && n <= p.rows) return n;
  atomicOr(p.t.status, kKv4StatusRange);
  return 0;
}

template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* src, float (&x)[8]) {
  const uint4 w = __ldcs(reinterpret_cast<const uint4*>(src));
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(a[i] << 16);
    x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* src, float (&x)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(src));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(src) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
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

// Code of x: the border of two codes is decided exactly.  d + e is x - low without error
// (the two terms of a floating-point sum), the quotient's floor is off by one at most, and
// r = d - c * scale is exact: c * scale has 12 bits, and the difference is a multiple of
// the last place of d and smaller than d's leading bits.
__device__ __forceinline__ uint32_t code_of(float x, float low, float scale, float inv) {
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

// One group's parameters from the 8 values of each of four neighbouring lanes.
__device__ __forceinline__ void group_params(const float (&x)[8], float& scale, float& low) {
  float lo = x[0], hi = x[0];
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    fine = fine && fabsf(x[i]) <= 3.402823466e38f;  // false for a NaN as well
  }
  if (!fine) lo = -INFINITY;  // makes the scale infinite below
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  low = bf16_round(lo);
  scale = bf16_round(__fdiv_rn(hi - low, 15.f));
  if (!(fabsf(scale) <= 3.402823466e38f)) {
    scale = 0.f;
    low = __uint_as_float(0x7fff0000u);  // NaN
  } else if (scale < 7.888609052e-31f) {  // 2^-100
    scale = 0.f;
  }
}

// Thread layout of a row pair (the K and the V row of one token and head): D/8 lanes for
// K, then D/8 for V.
template <int D>
struct Lanes {
  static constexpr int kRow = D / 8;    // lanes of a row
  static constexpr int kPair = D / 4;   // lanes of a token and head: 32 or 16
  static constexpr int kPerBlock = kThreads / kPair;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    kv4_write_kernel(const Kv4RowsParams P, const T* __restrict__ k, const T* __restrict__ v) {
  using L = Lanes<D>;
  using F = Kv4Block<D>;
  constexpr int G = F::kGroups;
  const int64_t pairs = (int64_t)P.t.batch * P.t.heads_kv * P.rows;
  const int64_t pair = (int64_t)blockIdx.x * L::kPerBlock + threadIdx.x / L::kPair;
  const int at = threadIdx.x % L::kPair;
  const bool is_v = at >= L::kRow;
  const int i8 = at % L::kRow;  // channels 8*i8 .. 8*i8 + 7
  const int g = i8 / 4, c = i8 % 4;
  int64_t base = -1;
  int64_t pos = 0;
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = 0.f;
  if (pair < pairs) {
    const int t = (int)(pair % P.rows);
    const int bh = (int)(pair / P.rows), b = bh / P.t.heads_kv, h = bh % P.t.heads_kv;
    if (t < live_rows(P, b)) {
      const int32_t f = __ldg(P.first + b);
      pos = f < 0 ? -1 : (int64_t)f + t;
      base = block_of(P.t, b, h, pos, F::kBytes);
      if (base >= 0) load8<T>((is_v ? v : k) + pair * D + i8 * 8, x);
    }
  }
  // (every lane takes part in the exchanges)
  float scale, low;
  group_params(x, scale, low);
  uint32_t word = 0;
  if (scale > 0.f) {
    const float inv = __frcp_rn(scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) word |= code_of(x[i], low, scale, inv) << (4 * i);
  }
  // Values: this lane holds the 16-bit words of chunks 2c (low half) and 2c + 1 (high
  // half) for group g; with the lane of the neighbouring group (4 lanes on) it makes whole
  // 32-bit words: the even group's lane chunk 2c, the odd group's chunk 2c + 1.
  const uint32_t other = __shfl_xor_sync(0xffffffffu, word, 4);
  if (base < 0) return;
  const int row = (int)(pos % kKvBlockRows);
  uint8_t* blk = P.t.cache + base;
  uint32_t at_word;
  if (is_v) {
    word = (g & 1) ? (other >> 16) | (word & 0xffff0000u) : (word & 0xffffu) | (other << 16);
    at_word = (2 * c + (g & 1)) * (G / 2) + g / 2;
  } else {
    at_word = c * G + g;
  }
  reinterpret_cast<uint32_t*>(blk + (is_v ? F::kOffV : F::kOffK) + row * F::kCodeBytes)[at_word] = word;
  if (c == 0)
    reinterpret_cast<uint32_t*>(blk + (is_v ? F::kOffVPar : F::kOffKPar) + row * F::kParBytes)[g] =
        (__float_as_uint(scale) >> 16) | (__float_as_uint(low) & 0xffff0000u);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4RowsParams P, T* __restrict__ k, T* __restrict__ v) {
  using L = Lanes<D>;
  using F = Kv4Block<D>;
  constexpr int G = F::kGroups;
  const int64_t pairs = (int64_t)P.t.batch * P.t.heads_kv * P.rows;
  const int64_t pair = (int64_t)blockIdx.x * L::kPerBlock + threadIdx.x / L::kPair;
  if (pair >= pairs) return;
  const int at = threadIdx.x % L::kPair;
  const bool is_v = at >= L::kRow;
  const int i8 = at % L::kRow, g = i8 / 4, c = i8 % 4;
  const int t = (int)(pair % P.rows);
  const int bh = (int)(pair / P.rows), b = bh / P.t.heads_kv, h = bh % P.t.heads_kv;
  int64_t base = -1, pos = 0;
  if (t < live_rows(P, b)) {
    const int32_t f = __ldg(P.first + b);
    pos = f < 0 ? -1 : (int64_t)f + t;
    base = block_of(P.t, b, h, pos, F::kBytes);
  }
  T* dst = (is_v ? v : k) + pair * D + i8 * 8;
  float x[8];
  if (base < 0) {
    if (!P.zero_rest) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    store8<T>(dst, x);
    return;
  }
  const int row = (int)(pos % kKvBlockRows);
  const uint8_t* blk = P.t.cache + base;
  const uint8_t* codes = blk + (is_v ? F::kOffV : F::kOffK) + row * F::kCodeBytes;
  uint32_t word;
  if (is_v) {
    const uint16_t* half = reinterpret_cast<const uint16_t*>(codes);
    word = half[(2 * c) * G + g] | ((uint32_t)half[(2 * c + 1) * G + g] << 16);
  } else {
    word = reinterpret_cast<const uint32_t*>(codes)[c * G + g];
  }
  const uint32_t par =
      reinterpret_cast<const uint32_t*>(blk + (is_v ? F::kOffVPar : F::kOffKPar) + row * F::kParBytes)[g];
  const float scale = __uint_as_float(par << 16), low = __uint_as_float(par & 0xffff0000u);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf(scale, (float)((word >> (4 * i)) & 15u), low);
  store8<T>(dst, x);
}

template <int D>
unsigned grid_of(const Kv4RowsParams& prm) {
  const int64_t pairs = (int64_t)prm.t.batch * prm.t.heads_kv * prm.rows;
  return (unsigned)((pairs + Lanes<D>::kPerBlock - 1) / Lanes<D>::kPerBlock);
}

template <typename T, int D>
cudaError_t write_as(const Kv4RowsParams& prm, const void* k, const void* v, cudaStream_t st) {
  kv4_write_kernel<T, D><<<grid_of<D>(prm), kThreads, 0, st>>>(prm, static_cast<const T*>(k), static_cast<const T*>(v));
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t read_as(const Kv4RowsParams& prm, void* k, void* v, cudaStream_t st) {
  kv4_read_kernel<T, D><<<grid_of<D>(prm), kThreads, 0, st>>>(prm, static_cast<T*>(k), static_cast<T*>(v));
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
