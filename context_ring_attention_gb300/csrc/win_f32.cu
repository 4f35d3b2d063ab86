// Windowed attention in float32 on CUDA cores (any d <= 128): forward and gradients,
// for the small float32 problems.  The query at position i sees the keys j <= i with
// j > i - window or j < sinks; everything is kept in fp32 with the accurate
// exponential and logarithm (Module 23, "The Math: One Block at a Time").
//
// Rows are taken in the order of their positions, whatever the layout: a CTA owns 16
// consecutive queries (or keys, for dK and dV), and walks the positions that any of them
// meets in chunks of 32.  Four groups of four warps take every fourth chunk: a group brings
// its chunk to shared memory, a warp has 4 of the 16 rows, a lane scores one of the 32 rows
// against the 4, so that a value read from shared memory enters 4 products, and then holds
// d/32 output columns of the 4.  At the end the groups' sums are joined in order.
// What bounds these sizes is the latency of the chunks in turn, hence the groups: the
// chunk loop of a key tile that holds a sink spans the sequence.  Measured (96 tokens, 2
// heads, d = 32): forward 6.4 us, gradients 24 us in three launches.
// Ring steps and partials, which fold one shard's block at a time, keep a warp per row.
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
    // this step's block alone
    const int64_t at = (int64_t)(t - P.step_lo) * rows_all + grow;
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int x = 0; x < kMaxD / 32; ++x) {
      const int col = lane + 32 * x;
      if (col < d) P.o_parts[at * d + col] = acc[x] * inv;
      acc[x] = 0.f;
    }
    if (lane == 0) P.lse_parts[at] = l > 0.f ? m + logf(l) : -INFINITY;
    m = -INFINITY;
    l = 0.f;
  }
}

// ------------------------------------------------- rows by position, 16 a CTA --
constexpr int kOwn = 16;        // rows of a CTA
constexpr int kPer = 4;         // rows of a warp
constexpr int kChunk = 32;      // rows met at a time
constexpr int kGroups = 4;      // groups of kWarps warps that take the chunks in turn
constexpr int kThreads = kGroups * kWarps * 32;
static_assert(kOwn == kPer * kWarps, "rows of a CTA");

// Row of a head at which position x lies.
__device__ __forceinline__ int row_of(int layout, int n_shards, int s_n, int x) {
  if (layout == RA_LAYOUT_STRIPED) return x % n_shards * s_n + x / n_shards;
  if (layout == RA_LAYOUT_ZIGZAG) {
    const int c = s_n >> 1, chunk = x / c, at = x - chunk * c;
    return chunk < n_shards ? chunk * s_n + at : (2 * n_shards - 1 - chunk) * s_n + c + at;
  }
  return x;
}

// Shared memory of a CTA, in floats: own rows as [channel][16] (two tensors); per group a
// chunk as [32][d + 1] (two tensors) and the 4 weights of every row of the chunk per warp
// (two).  A group's chunks hold its sums at the end.
struct Smem {
  float *own0, *own1, *chunk0, *chunk1, *w0, *w1;
  int pitch, group_floats;
  __device__ __forceinline__ Smem(float* base, int d, int group) {
    pitch = d + 1;
    group_floats = floats_of_group(d);
    own0 = base;
    own1 = own0 + d * kOwn;
    w0 = own1 + d * kOwn + group * group_floats;  // (a multiple of 4 floats from base)
    w1 = w0 + kWarps * kChunk * kPer;
    chunk0 = w1 + kWarps * kChunk * kPer;
    chunk1 = chunk0 + kChunk * pitch;
  }
  __device__ __forceinline__ float* sums_of(const float* base, int d, int g) const {
    return const_cast<float*>(base) + 2 * d * kOwn + g * group_floats + (chunk0 - w0);
  }
  __host__ __device__ static int floats_of_group(int d) { return 2 * kWarps * kChunk * kPer + 2 * kChunk * (d + 1); }
  static size_t bytes(int d) { return (size_t)(2 * d * kOwn + kGroups * floats_of_group(d)) * 4; }
};
// Barrier of one group's warps.
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(kWarps * 32) : "memory");
}

// n rows (up to kRows) of two tensors' heads, rows of d, through put(row, channel, x, y); the
// rows from n on are zeros.  row: the lane's row in the heads (lane r: the r-th of the n).  A
// warp of a group takes every fourth row and requests all its elements before it uses one.
template <int kRows, class Put>
__device__ __forceinline__ void load_rows(int n, int d, const float* a, const float* b, int row, Put&& put) {
  const int warp = (threadIdx.x >> 5) % kWarps, lane = threadIdx.x & 31;
#pragma unroll
  for (int x = 0; x < kMaxD / 32; ++x) {
    const int col = lane + 32 * x;
    if (32 * x >= d) break;
    float u[kRows / kWarps], w[kRows / kWarps];
#pragma unroll
    for (int i = 0; i < kRows / kWarps; ++i) {
      const int r = warp + i * kWarps;
      const int64_t from = (int64_t)__shfl_sync(0xffffffffu, row, r) * d + col;
      const bool live = r < n && col < d;
      u[i] = live ? a[from] : 0.f;
      w[i] = live && b != nullptr ? b[from] : 0.f;
    }
    if (col < d)
#pragma unroll
      for (int i = 0; i < kRows / kWarps; ++i) put(warp + i * kWarps, col, u[i], w[i]);
  }
}
__device__ __forceinline__ void load_own(const Smem& sm, int d, int n, const float* a, const float* b, int row) {
  load_rows<kOwn>(n, d, a, b, row, [&](int r, int c, float x, float y) {
    sm.own0[c * kOwn + r] = x;
    sm.own1[c * kOwn + r] = y;
  });
}
__device__ __forceinline__ void load_chunk(const Smem& sm, int d, int n, const float* a, const float* b, int row) {
  load_rows<kChunk>(n, d, a, b, row, [&](int r, int c, float x, float y) {
    sm.chunk0[r * sm.pitch + c] = x;
    sm.chunk1[r * sm.pitch + c] = y;
  });
}
// Dot products of this lane's row of a chunk with the warp's 4 own rows.
__device__ __forceinline__ void dots(const float* own, const float* chunk, int pitch, int d, int warp, int lane,
                                     float (&out)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) out[i] = 0.f;
  const float* row = chunk + lane * pitch;
#pragma unroll 4
  for (int c = 0; c < d; ++c) {
    const float4 o = *reinterpret_cast<const float4*>(own + c * kOwn + warp * kPer);
    const float x = row[c];
    out[0] = fmaf(o.x, x, out[0]);
    out[1] = fmaf(o.y, x, out[1]);
    out[2] = fmaf(o.z, x, out[2]);
    out[3] = fmaf(o.w, x, out[3]);
  }
}
// acc[i][x] += sum over the chunk's rows j of w[j][i] * chunk[j][lane + 32 x].
__device__ __forceinline__ void add_rows(const float* w, const float* chunk, int pitch, int d, int n, int warp, int lane,
                                         float (&acc)[kPer][kMaxD / 32]) {
  const float4* wv = reinterpret_cast<const float4*>(w + warp * kChunk * kPer);
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const float4 p = wv[j];
#pragma unroll
    for (int x = 0; x < kMaxD / 32; ++x) {
      const int col = lane + 32 * x;
      if (col >= d) break;
      const float y = chunk[j * pitch + col];
      acc[0][x] = fmaf(p.x, y, acc[0][x]);
      acc[1][x] = fmaf(p.y, y, acc[1][x]);
      acc[2][x] = fmaf(p.z, y, acc[2][x]);
      acc[3][x] = fmaf(p.w, y, acc[3][x]);
    }
  }
}
__device__ __forceinline__ void put_weights(float* w, int warp, int lane, const float (&p)[kPer]) {
  *reinterpret_cast<float4*>(w + (warp * kChunk + lane) * kPer) = make_float4(p[0], p[1], p[2], p[3]);
}
__device__ __forceinline__ bool sees(int i, int j, int window, int sinks) {
  return j <= i && (j > i - window || j < sinks);
}

// Calls body(first position, rows) for this group's chunks of the positions that queries
// [i0, i1] see: the sinks' [0, first), then [lo, i1].
template <class Body>
__device__ __forceinline__ void for_each_chunk(int i0, int i1, int window, int sinks, int group, Body&& body) {
  const int lo = i0 - window + 1 > 0 ? i0 - window + 1 : 0;
  const int first = sinks < lo ? sinks : lo;
  int turn = 0;
  for (int run = 0; run < 2; ++run) {
    const int end = run ? i1 + 1 : first;
    for (int x = run ? lo : 0; x < end; x += kChunk, ++turn)
      if (turn % kGroups == group) body(x, end - x < kChunk ? end - x : kChunk);
  }
}
// Leaves the warp's sums in the group's area, from row 16 * which on.
__device__ __forceinline__ void leave_sums(float* sums, int which, int d, int warp, int lane,
                                           const float (&acc)[kPer][kMaxD / 32]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int x = 0; x < kMaxD / 32; ++x)
      if (lane + 32 * x < d) sums[(which * kOwn + warp * kPer + i) * d + lane + 32 * x] = acc[i][x];
}

// Fused and gathered forward: one CTA per 16 positions of a query head.
__global__ void __launch_bounds__(kThreads)
    win_fwd_f32_rows_kernel(const WinParams P, const float* __restrict__ q, const float* __restrict__ k,
                            const float* __restrict__ v) {
  extern __shared__ __align__(16) float smem_f[];
  const int group = threadIdx.x / (kWarps * 32);
  const Smem sm(smem_f, P.head_dim, group);
  const int warp = (threadIdx.x >> 5) % kWarps, lane = threadIdx.x & 31, d = P.head_dim;
  const int tiles = (P.seq + kOwn - 1) / kOwn;
  const int64_t bh = blockIdx.x / tiles;
  const int i0 = (int)(blockIdx.x - bh * tiles) * kOwn, n_own = min(kOwn, P.seq - i0);
  const int b = (int)(bh / P.heads_q), h = (int)(bh % P.heads_q);
  const int64_t kv = ((int64_t)b * P.heads_kv + h / P.group) * P.seq * d;
  auto q_row = [&](int x) { return row_of(P.q.layout, P.q.shards, P.q.s_n, x); };
  auto k_row = [&](int x) { return row_of(P.k.layout, P.k.shards, P.k.s_n, x); };
  if (group == 0) load_own(sm, d, n_own, q + bh * P.seq * d, nullptr, lane < n_own ? q_row(i0 + lane) : 0);

  __syncthreads();
  float m[kPer], l[kPer], acc[kPer][kMaxD / 32];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int x = 0; x < kMaxD / 32; ++x) acc[i][x] = 0.f;
  }
  for_each_chunk(i0, i0 + n_own - 1, P.window, P.sinks, group, [&](int x0, int n) {
    group_sync(group);  // the chunk before is done with
    load_chunk(sm, d, n, k + kv, v + kv, lane < n ? k_row(x0 + lane) : 0);
    group_sync(group);
    float s[kPer];
    dots(sm.own0, sm.chunk0, sm.pitch, d, warp, lane, s);
    bool scale_acc = false;
    float corr[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool seen = lane < n && sees(i0 + warp * kPer + i, x0 + lane, P.window, P.sinks);
      s[i] = seen ? s[i] * P.scale : -INFINITY;
      const float m_new = fmaxf(m[i], warp_max(s[i]));
      // a row whose scores so far are all -inf keeps p = 0
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      corr[i] = expf(m[i] - ref);
      scale_acc = scale_acc || m_new != m[i];
      s[i] = expf(s[i] - ref);
      l[i] = l[i] * corr[i] + warp_sum(s[i]);
      m[i] = m_new;
    }
    if (scale_acc) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int x = 0; x < kMaxD / 32; ++x) acc[i][x] *= corr[i];
    }
    put_weights(sm.w0, warp, lane, s);
    __syncwarp();
    add_rows(sm.w0, sm.chunk1, sm.pitch, d, n, warp, lane, acc);
  });
  // Join the groups: every row's maximum and sum of each, then the columns.
  __shared__ float gm[kGroups][kOwn], gl[kGroups][kOwn];
  group_sync(group);  // (its chunk is done with)
  leave_sums(sm.chunk0, 0, d, warp, lane, acc);
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      gm[group][warp * kPer + i] = m[i];
      gl[group][warp * kPer + i] = l[i];
    }
  __syncthreads();
  for (int r = threadIdx.x >> 5; r < n_own; r += kGroups * kWarps) {
    float mx = -INFINITY, sum = 0.f, f[kGroups];
#pragma unroll
    for (int z = 0; z < kGroups; ++z) mx = fmaxf(mx, gm[z][r]);
#pragma unroll
    for (int z = 0; z < kGroups; ++z) {
      f[z] = gm[z][r] == -INFINITY ? 0.f : expf(gm[z][r] - mx);
      sum = fmaf(f[z], gl[z][r], sum);
    }
    const int64_t row = bh * P.seq + q_row(i0 + r);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    for (int c = lane; c < d; c += 32) {
      float y = 0.f;
#pragma unroll
      for (int z = 0; z < kGroups; ++z) y = fmaf(f[z], sm.sums_of(smem_f, d, z)[r * d + c], y);
      static_cast<float*>(P.o)[row * d + c] = y * inv;
    }
    if (lane == 0 && P.lse != nullptr) P.lse[row] = sum > 0.f ? mx + logf(sum) : -INFINITY;
  }
}

// Index of a query row's lse2 (its D is 64 further).
__device__ __forceinline__ int64_t scalar_at(const BwdParams& P, int64_t bh, int row) {
  const int p = row / (int)P.s_n;
  return bwd_scalar_index(bh, p, row - p * (int)P.s_n, P.n_shards, P.n64);
}

// dQ: one CTA per 16 positions of a query head.
__global__ void __launch_bounds__(kThreads)
    win_bwd_f32_dq_kernel(const BwdParams P, int window, int sinks, const float* __restrict__ q,
                          const float* __restrict__ k, const float* __restrict__ v, const float* __restrict__ dout) {
  extern __shared__ __align__(16) float smem_f[];
  const int group = threadIdx.x / (kWarps * 32);
  const Smem sm(smem_f, P.head_dim, group);
  const int warp = (threadIdx.x >> 5) % kWarps, lane = threadIdx.x & 31, d = P.head_dim, seq = (int)P.seq;
  const int tiles = (seq + kOwn - 1) / kOwn;
  const int64_t bh = blockIdx.x / tiles;
  const int i0 = (int)(blockIdx.x - bh * tiles) * kOwn, n_own = min(kOwn, seq - i0);
  const int b = (int)(bh / P.heads_q), h = (int)(bh % P.heads_q);
  const int64_t kv = ((int64_t)b * P.heads_kv + h / P.group) * seq * d;
  auto row = [&](int x) { return row_of(P.layout, P.n_shards, (int)P.s_n, x); };
  if (group == 0) load_own(sm, d, n_own, q + bh * seq * d, dout + bh * seq * d, lane < n_own ? row(i0 + lane) : 0);
  __syncthreads();
  float l2[kPer], dd[kPer], acc[kPer][kMaxD / 32];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = warp * kPer + i;
    l2[i] = dd[i] = 0.f;
    if (r < n_own) {
      const int64_t li = scalar_at(P, bh, row(i0 + r));
      RA_BOUNDS(P.status, li >= 0 && li + 64 < (int64_t)P.batch * P.heads_q * P.n_shards * P.n64 * 128, 71);
      l2[i] = P.lse2d[li];
      dd[i] = P.lse2d[li + 64];
    }
#pragma unroll
    for (int x = 0; x < kMaxD / 32; ++x) acc[i][x] = 0.f;
  }
  for_each_chunk(i0, i0 + n_own - 1, window, sinks, group, [&](int x0, int n) {
    group_sync(group);
    load_chunk(sm, d, n, k + kv, v + kv, lane < n ? row(x0 + lane) : 0);
    group_sync(group);
    float s[kPer], dp[kPer];
    dots(sm.own0, sm.chunk0, sm.pitch, d, warp, lane, s);
    dots(sm.own1, sm.chunk1, sm.pitch, d, warp, lane, dp);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool seen = lane < n && sees(i0 + warp * kPer + i, x0 + lane, window, sinks);
      s[i] = seen ? exp2f(fmaf(s[i], P.scale_log2, -l2[i])) * (dp[i] - dd[i]) : 0.f;
    }
    put_weights(sm.w0, warp, lane, s);
    __syncwarp();
    add_rows(sm.w0, sm.chunk0, sm.pitch, d, n, warp, lane, acc);
  });
  group_sync(group);
  leave_sums(sm.chunk0, 0, d, warp, lane, acc);
  __syncthreads();
  for (int r = threadIdx.x >> 5; r < n_own; r += kGroups * kWarps) {
    float* dst = static_cast<float*>(P.dq) + (bh * seq + row(i0 + r)) * d;
    for (int c = lane; c < d; c += 32) {
      float y = 0.f;
#pragma unroll
      for (int z = 0; z < kGroups; ++z) y += sm.sums_of(smem_f, d, z)[r * d + c];
      dst[c] = y * P.scale;
    }
  }
}

// dK, dV: one CTA per 16 positions of a key/value head; it meets the queries from its first
// key on, up to window - 1 past its last one, or all of them when it holds a sink, of every
// query head of the group.
__global__ void __launch_bounds__(kThreads)
    win_bwd_f32_dkdv_kernel(const BwdParams P, int window, int sinks, const float* __restrict__ q,
                            const float* __restrict__ k, const float* __restrict__ v, const float* __restrict__ dout) {
  extern __shared__ __align__(16) float smem_f[];
  const int group = threadIdx.x / (kWarps * 32);
  const Smem sm(smem_f, P.head_dim, group);
  const int warp = (threadIdx.x >> 5) % kWarps, lane = threadIdx.x & 31, d = P.head_dim, seq = (int)P.seq;
  const int tiles = (seq + kOwn - 1) / kOwn;
  const int64_t bk = blockIdx.x / tiles;
  const int j0 = (int)(blockIdx.x - bk * tiles) * kOwn, n_own = min(kOwn, seq - j0);
  const int b = (int)(bk / P.heads_kv), hk = (int)(bk % P.heads_kv);
  auto row = [&](int x) { return row_of(P.layout, P.n_shards, (int)P.s_n, x); };
  if (group == 0) load_own(sm, d, n_own, k + bk * seq * d, v + bk * seq * d, lane < n_own ? row(j0 + lane) : 0);
  __syncthreads();
  float dk[kPer][kMaxD / 32], dv[kPer][kMaxD / 32];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int x = 0; x < kMaxD / 32; ++x) dk[i][x] = dv[i][x] = 0.f;
  const int64_t far = (int64_t)j0 + n_own - 1 + window;  // first position past their reach
  const int end = j0 < sinks || far > seq ? seq : (int)far;
  int turn = 0;
  for (int g = 0; g < P.group; ++g) {
    const int64_t qh = (int64_t)b * P.heads_q + (int64_t)hk * P.group + g;
    for (int x0 = j0; x0 < end; x0 += kChunk) {
      if (turn++ % kGroups != group) continue;
      const int n = min(kChunk, end - x0);
      group_sync(group);
      load_chunk(sm, d, n, q + qh * seq * d, dout + qh * seq * d, lane < n ? row(x0 + lane) : 0);
      float l2 = 0.f, dd = 0.f;
      if (lane < n) {
        const int64_t li = scalar_at(P, qh, row(x0 + lane));
        RA_BOUNDS(P.status, li >= 0 && li + 64 < (int64_t)P.batch * P.heads_q * P.n_shards * P.n64 * 128, 72);
        l2 = P.lse2d[li];
        dd = P.lse2d[li + 64];
      }
      group_sync(group);
      float s[kPer], dp[kPer];
      dots(sm.own0, sm.chunk0, sm.pitch, d, warp, lane, s);
      dots(sm.own1, sm.chunk1, sm.pitch, d, warp, lane, dp);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const bool seen = lane < n && sees(x0 + lane, j0 + warp * kPer + i, window, sinks);
        s[i] = seen ? exp2f(fmaf(s[i], P.scale_log2, -l2)) : 0.f;
        dp[i] = seen ? s[i] * (dp[i] - dd) : 0.f;
      }
      put_weights(sm.w0, warp, lane, s);
      put_weights(sm.w1, warp, lane, dp);
      __syncwarp();
      add_rows(sm.w0, sm.chunk1, sm.pitch, d, n, warp, lane, dv);
      add_rows(sm.w1, sm.chunk0, sm.pitch, d, n, warp, lane, dk);
    }
  }
  group_sync(group);
  leave_sums(sm.chunk0, 0, d, warp, lane, dk);
  leave_sums(sm.chunk0, 1, d, warp, lane, dv);
  __syncthreads();
  for (int r = threadIdx.x >> 5; r < n_own; r += kGroups * kWarps) {
    const int64_t at = (bk * seq + row(j0 + r)) * d;
    for (int c = lane; c < d; c += 32) {
      float y = 0.f, z2 = 0.f;
#pragma unroll
      for (int z = 0; z < kGroups; ++z) {
        y += sm.sums_of(smem_f, d, z)[r * d + c];
        z2 += sm.sums_of(smem_f, d, z)[(kOwn + r) * d + c];
      }
      static_cast<float*>(P.dk)[at + c] = y * P.scale;
      static_cast<float*>(P.dv)[at + c] = z2;
    }
  }
}

// Dynamic shared memory beyond 48 KiB has to be asked for, once per device.
template <class Kernel>
cudaError_t allow_smem(Kernel kernel, std::atomic<int>* ready) {
  const char* why = "";
  return prepare_once(kernel, ready, kThreads, 0, (int)Smem::bytes(kMaxD), &why);
}

int64_t tiles_of(int64_t heads, int64_t seq) { return heads * ((seq + kOwn - 1) / kOwn); }

}  // namespace

cudaError_t launch_win_fwd_f32(const WinParams& prm, const float* q, const float* k, const float* v,
                               cudaStream_t stream) {
  if (prm.o_parts == nullptr) {
    static std::atomic<int> ready[kMaxDevices];
    const cudaError_t e = allow_smem(win_fwd_f32_rows_kernel, ready);
    const int64_t blocks = tiles_of((int64_t)prm.batch * prm.heads_q, prm.seq);
    if (e != cudaSuccess) return e;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    win_fwd_f32_rows_kernel<<<(unsigned)blocks, kThreads, Smem::bytes(prm.head_dim), stream>>>(prm, q, k, v);
    return cudaGetLastError();
  }
  const int64_t rows = (int64_t)prm.batch * prm.heads_q * prm.seq;
  const int64_t blocks = (rows + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  win_fwd_f32_kernel<<<(unsigned)blocks, kWarps * 32, 0, stream>>>(prm, q, k, v);
  return cudaGetLastError();
}

cudaError_t launch_win_bwd_f32(const BwdParams& prm, int window, int sinks, const float* q, const float* k,
                               const float* v, const float* dout, cudaStream_t stream) {
  static std::atomic<int> ready_q[kMaxDevices], ready_k[kMaxDevices];
  const int64_t bq = tiles_of((int64_t)prm.batch * prm.heads_q, prm.seq);
  const int64_t bk = tiles_of((int64_t)prm.batch * prm.heads_kv, prm.seq);
  if (bq > 0x7fffffff || bk > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaError_t e = allow_smem(win_bwd_f32_dq_kernel, ready_q);
  if (e == cudaSuccess) e = allow_smem(win_bwd_f32_dkdv_kernel, ready_k);
  if (e != cudaSuccess) return e;
  const size_t smem = Smem::bytes(prm.head_dim);
  win_bwd_f32_dq_kernel<<<(unsigned)bq, kThreads, smem, stream>>>(prm, window, sinks, q, k, v, dout);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  win_bwd_f32_dkdv_kernel<<<(unsigned)bk, kThreads, smem, stream>>>(prm, window, sinks, q, k, v, dout);
  return cudaGetLastError();
}

}  // namespace ra
