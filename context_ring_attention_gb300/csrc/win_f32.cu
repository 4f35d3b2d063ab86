// Windowed attention in float32 on CUDA cores (any d <= 128): forward and gradients,
// for the small float32 problems.  The query at position i sees the keys j <= i with
// j > i - window or j < sinks; everything is kept in fp32 with the accurate
// exponential and logarithm (Module 23, "The Math: One Block at a Time").
//
// One warp owns one query row (forward, dQ) or one key row (dK, dV): each lane scores
// one of 32 keys (or queries), and each lane accumulates d/32 output columns.  Only the
// rows that are seen are read: per key block two runs, the sinks and the window.
#include <cuda_runtime.h>

#include <cstdint>

#include "win_internal.h"

namespace ra {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxD = 128;

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float dot_row(const float* a, const float* b, int d) {
  float acc = 0.f;
  for (int c = 0; c < d; ++c) acc = fmaf(a[c], b[c], acc);
  return acc;
}

__global__ void __launch_bounds__(kWarps * 32)
    win_fwd_f32_kernel(const WinParams P, const float* __restrict__ q, const float* __restrict__ k,
                       const float* __restrict__ v) {
  __shared__ float qs[kWarps][kMaxD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t rows_all = (int64_t)P.batch * P.heads_q * P.seq;
  const int64_t grow = (int64_t)blockIdx.x * kWarps + warp;  // global query row
  if (grow >= rows_all) return;
  const int d = P.head_dim, N = P.k.shards;
  const int64_t bh = grow / P.seq;
  const int srow = (int)(grow % P.seq);
  const int p = srow / P.q.s_n, i = srow % P.q.s_n;
  const int b = (int)(bh / P.heads_q), h = (int)(bh % P.heads_q);
  const int64_t kv_base = ((int64_t)b * P.heads_kv + h / P.group) * P.seq;
  const int my_pos = (int)pos_of(P.q.layout, P.q.shards, P.q.s_n, p, i);

  for (int c = lane; c < d; c += 32) qs[warp][c] = q[grow * d + c];
  __syncwarp();

  const bool partials = P.o_parts != nullptr;
  float m = -INFINITY, l = 0.f;
  float acc[kMaxD / 32];
#pragma unroll
  for (int x = 0; x < kMaxD / 32; ++x) acc[x] = 0.f;

  for (int t = P.step_lo; t < P.step_hi; ++t) {
    const int r = N == 1 ? 0 : (p - t + N) % N;
    const int slot = P.kv_rotated ? p : r;  // where the block of step t sits
    const WinSpan sp = win_span(P.k.layout, N, P.k.s_n, P.window, P.sinks, r, my_pos, my_pos);
    RA_BOUNDS(P.status, sp.first >= 0 && sp.lo >= 0 && sp.hi <= P.k.s_n && slot >= 0 && slot < N, 70);
    const float* kb = k + (kv_base + (int64_t)slot * P.k.s_n) * d;
    const float* vb = v + (kv_base + (int64_t)slot * P.k.s_n) * d;
    for (int run = 0; run < 2; ++run) {  // the sinks, then the window
      const int end = run ? sp.hi : sp.first;
      for (int j0 = run ? sp.lo : 0; j0 < end; j0 += 32) {
        const int j = j0 + lane;
        float s = -INFINITY;
        if (j < end) s = dot_row(qs[warp], kb + (int64_t)j * d, d) * P.scale;
        const float m_new = fmaxf(m, warp_max(s));
        // a row whose scores so far are all -inf keeps p = 0 (and O = 0, LSE = -inf)
        const float mref = m_new == -INFINITY ? 0.f : m_new;
        const float corr = expf(m - mref);
        const float pj = (j < end) ? expf(s - mref) : 0.f;
        l = l * corr + warp_sum(pj);
#pragma unroll
        for (int x = 0; x < kMaxD / 32; ++x) acc[x] *= corr;
        const int nj = (end - j0 < 32) ? end - j0 : 32;
        for (int jj = 0; jj < nj; ++jj) {
          const float pb = __shfl_sync(0xffffffffu, pj, jj);
          const float* vr = vb + (int64_t)(j0 + jj) * d;
#pragma unroll
          for (int x = 0; x < kMaxD / 32; ++x) {
            const int col = lane + 32 * x;
            if (col < d) acc[x] = fmaf(pb, vr[col], acc[x]);
          }
        }
        m = m_new;
      }
    }
    if (partials || t == P.step_hi - 1) {  // this step's block alone, or the whole row
      const int64_t at = partials ? (int64_t)(t - P.step_lo) * rows_all + grow : grow;
      float* dst = (partials ? P.o_parts : static_cast<float*>(P.o)) + at * d;
      float* lse = partials ? P.lse_parts : P.lse;
      const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int x = 0; x < kMaxD / 32; ++x) {
        const int col = lane + 32 * x;
        if (col < d) dst[col] = acc[x] * inv;
        acc[x] = 0.f;
      }
      if (lane == 0 && lse != nullptr) lse[at] = l > 0.f ? m + logf(l) : -INFINITY;
      m = -INFINITY;
      l = 0.f;
    }
  }
}

__global__ void __launch_bounds__(kWarps * 32)
    win_bwd_f32_dq_kernel(const BwdParams P, int window, int sinks, const float* __restrict__ q, const float* __restrict__ k,
                          const float* __restrict__ v, const float* __restrict__ dout) {
  __shared__ float qs[kWarps][kMaxD], dos[kWarps][kMaxD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t rows_all = (int64_t)P.batch * P.heads_q * P.seq;
  const int64_t grow = (int64_t)blockIdx.x * kWarps + warp;
  if (grow >= rows_all) return;
  const int d = P.head_dim, N = P.n_shards;
  const int64_t bh = grow / P.seq;
  const int srow = (int)(grow % P.seq);
  const int p = srow / (int)P.s_n, i = srow % (int)P.s_n;
  const int b = (int)(bh / P.heads_q), h = (int)(bh % P.heads_q);
  const int64_t kv_base = ((int64_t)b * P.heads_kv + h / P.group) * P.seq;
  const int my_pos = (int)pos_of(P.layout, N, P.s_n, p, i);
  for (int c = lane; c < d; c += 32) {
    qs[warp][c] = q[grow * d + c];
    dos[warp][c] = dout[grow * d + c];
  }
  __syncwarp();
  const int64_t li = bwd_scalar_index(bh, p, i, N, P.n64);
  RA_BOUNDS(P.status, li >= 0 && li + 64 < (int64_t)P.batch * P.heads_q * N * P.n64 * 128, 71);
  const float2 ld = make_float2(P.lse2d[li], P.lse2d[li + 64]);
  float acc[kMaxD / 32];
#pragma unroll
  for (int x = 0; x < kMaxD / 32; ++x) acc[x] = 0.f;
  for (int t = 0; t < N; ++t) {
    const int r = (p - t + N) % N;
    const WinSpan sp = win_span(P.layout, N, (int)P.s_n, window, sinks, r, my_pos, my_pos);
    const float* kb = k + (kv_base + (int64_t)r * P.s_n) * d;
    const float* vb = v + (kv_base + (int64_t)r * P.s_n) * d;
    for (int run = 0; run < 2; ++run) {
      const int end = run ? sp.hi : sp.first;
      for (int j0 = run ? sp.lo : 0; j0 < end; j0 += 32) {
        const int j = j0 + lane;
        float ds = 0.f;
        if (j < end) {
          const float pj = exp2f(fmaf(dot_row(qs[warp], kb + (int64_t)j * d, d), P.scale_log2, -ld.x));
          ds = pj * (dot_row(dos[warp], vb + (int64_t)j * d, d) - ld.y);
        }
        const int nj = (end - j0 < 32) ? end - j0 : 32;
        for (int jj = 0; jj < nj; ++jj) {
          const float dsb = __shfl_sync(0xffffffffu, ds, jj);
          const float* kr = kb + (int64_t)(j0 + jj) * d;
#pragma unroll
          for (int x = 0; x < kMaxD / 32; ++x) {
            const int col = lane + 32 * x;
            if (col < d) acc[x] = fmaf(dsb, kr[col], acc[x]);
          }
        }
      }
    }
  }
  float* dst = static_cast<float*>(P.dq) + grow * d;
#pragma unroll
  for (int x = 0; x < kMaxD / 32; ++x) {
    const int col = lane + 32 * x;
    if (col < d) dst[col] = acc[x] * P.scale;
  }
}

__global__ void __launch_bounds__(kWarps * 32)
    win_bwd_f32_dkdv_kernel(const BwdParams P, int window, int sinks, const float* __restrict__ q, const float* __restrict__ k,
                            const float* __restrict__ v, const float* __restrict__ dout) {
  __shared__ float ks[kWarps][kMaxD], vs[kWarps][kMaxD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t rows_all = (int64_t)P.batch * P.heads_kv * P.seq;
  const int64_t grow = (int64_t)blockIdx.x * kWarps + warp;  // key row
  if (grow >= rows_all) return;
  const int d = P.head_dim, N = P.n_shards;
  const int64_t bk = grow / P.seq;
  const int srow = (int)(grow % P.seq);
  const int r = srow / (int)P.s_n, j = srow % (int)P.s_n;
  const int b = (int)(bk / P.heads_kv), hk = (int)(bk % P.heads_kv);
  const int key_pos = (int)pos_of(P.layout, N, P.s_n, r, j);
  for (int c = lane; c < d; c += 32) {
    ks[warp][c] = k[grow * d + c];
    vs[warp][c] = v[grow * d + c];
  }
  __syncwarp();
  float dk[kMaxD / 32], dv[kMaxD / 32];
#pragma unroll
  for (int x = 0; x < kMaxD / 32; ++x) dk[x] = dv[x] = 0.f;
  // the queries that see this key: up to window - 1 positions on, or all later ones
  const int64_t far = key_pos < sinks ? P.seq - 1 : (int64_t)key_pos + window - 1;
  const int last_pos = (int)(far < P.seq - 1 ? far : P.seq - 1);
  for (int t = 0; t < N; ++t) {
    const int p = (r + t) % N;  // the device this block sits on at step t
    const int i_lo = rows_le(P.layout, N, (int)P.s_n, p, key_pos - 1);
    const int i_hi = rows_le(P.layout, N, (int)P.s_n, p, last_pos);
    for (int g = 0; g < P.group; ++g) {
      const int64_t qh = (int64_t)b * P.heads_q + (int64_t)hk * P.group + g;
      const int64_t qrow0 = qh * P.seq + (int64_t)p * P.s_n;
      for (int i0 = i_lo; i0 < i_hi; i0 += 32) {
        const int i = i0 + lane;
        float pi = 0.f, ds = 0.f;
        if (i < i_hi) {
          const int64_t row = qrow0 + i;
          const int64_t li = bwd_scalar_index(qh, p, i, N, P.n64);
          RA_BOUNDS(P.status, row >= 0 && row < (int64_t)P.batch * P.heads_q * P.seq && li >= 0 &&
                                  li + 64 < (int64_t)P.batch * P.heads_q * N * P.n64 * 128, 72);
          const float2 ld = make_float2(P.lse2d[li], P.lse2d[li + 64]);
          pi = exp2f(fmaf(dot_row(q + row * d, ks[warp], d), P.scale_log2, -ld.x));
          ds = pi * (dot_row(dout + row * d, vs[warp], d) - ld.y);
        }
        const int ni = (i_hi - i0 < 32) ? i_hi - i0 : 32;
        for (int ii = 0; ii < ni; ++ii) {
          const float pb = __shfl_sync(0xffffffffu, pi, ii);
          const float db = __shfl_sync(0xffffffffu, ds, ii);
          const float* qr = q + (qrow0 + i0 + ii) * d;
          const float* dor = dout + (qrow0 + i0 + ii) * d;
#pragma unroll
          for (int x = 0; x < kMaxD / 32; ++x) {
            const int col = lane + 32 * x;
            if (col < d) {
              dv[x] = fmaf(pb, dor[col], dv[x]);
              dk[x] = fmaf(db, qr[col], dk[x]);
            }
          }
        }
      }
    }
  }
  float* dkd = static_cast<float*>(P.dk) + grow * d;
  float* dvd = static_cast<float*>(P.dv) + grow * d;
#pragma unroll
  for (int x = 0; x < kMaxD / 32; ++x) {
    const int col = lane + 32 * x;
    if (col < d) {
      dkd[col] = dk[x] * P.scale;
      dvd[col] = dv[x];
    }
  }
}

}  // namespace

cudaError_t launch_win_fwd_f32(const WinParams& prm, const float* q, const float* k, const float* v,
                               cudaStream_t stream) {
  const int64_t rows = (int64_t)prm.batch * prm.heads_q * prm.seq;
  const int64_t blocks = (rows + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  win_fwd_f32_kernel<<<(unsigned)blocks, kWarps * 32, 0, stream>>>(prm, q, k, v);
  return cudaGetLastError();
}

cudaError_t launch_win_bwd_f32(const BwdParams& prm, int window, int sinks, const float* q, const float* k,
                               const float* v, const float* dout, cudaStream_t stream) {
  const int64_t rows_q = (int64_t)prm.batch * prm.heads_q * prm.seq;
  const int64_t rows_kv = (int64_t)prm.batch * prm.heads_kv * prm.seq;
  const int64_t bq = (rows_q + kWarps - 1) / kWarps, bk = (rows_kv + kWarps - 1) / kWarps;
  if (bq > 0x7fffffff || bk > 0x7fffffff) return cudaErrorInvalidConfiguration;
  win_bwd_f32_dq_kernel<<<(unsigned)bq, kWarps * 32, 0, stream>>>(prm, window, sinks, q, k, v, dout);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  win_bwd_f32_dkdv_kernel<<<(unsigned)bk, kWarps * 32, 0, stream>>>(prm, window, sinks, q, k, v, dout);
  return cudaGetLastError();
}

}  // namespace ra
