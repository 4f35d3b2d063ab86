// Eviction by accumulated attention weight (include/ra.h, ra_paged_evict): of every sequence
// and key/value head the `keep` slots that stay are the first ones, the most recent ones, and
// of the others the heaviest, ties to the lowest slot; they move together in their order.
//
// Two kernels.  The first decides: a CTA per head and sequence finds the weight of the last
// slot that stays by its bits, 11 at a time from the top (a histogram in shared memory of the
// slots that agree so far), and lists the slots in order with one scan.  Counts are whole
// numbers: their order does not matter.  The second moves rows: a CTA has 64 bytes of every
// row of a head's keys or values, so that the list is walked in order by CTAs that do not
// depend on each other.  A row's new place is never behind its old one; a CTA that has read all
// rows up to some place may write up to it, also where old and new pages are the same.
// Bound by HBM: the kept rows are read and written once.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "paged_internal.h"

namespace ra {
namespace {

constexpr int kPickThreads = 1024;
constexpr int kBins = 2048;       // 11 bits a pass
constexpr int kMaxKnown = 49152;  // weights that the CTA keeps in shared memory

// Whole numbers in the order of the weights: NaN lowest, then -inf .. +inf, -0 as +0.
__device__ __forceinline__ uint32_t rank_of(float w) {
  if (w != w) return 0u;
  const uint32_t x = __float_as_uint(w + 0.f);
  return (x & 0x80000000u) ? ~x : x | 0x80000000u;
}

// Inclusive sums over the CTA's threads; all of them in `total`.  sums: 32 places.
__device__ __forceinline__ uint64_t scan(uint64_t x, uint64_t* sums, uint64_t& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint64_t s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  total = sums[31];
  if (warp > 0) x += sums[warp - 1];
  __syncthreads();
  return x;
}

__global__ void __launch_bounds__(kPickThreads) pick_kernel(const PagedEvictParams P, int known) {
  extern __shared__ uint32_t ranks[];  // [known]
  __shared__ uint32_t bins[kBins];
  __shared__ uint64_t sums[32];
  __shared__ uint32_t found[2];
  const int head = (int)blockIdx.x, b = (int)blockIdx.y, tid = threadIdx.x;
  int n = paged_seq(P.t, b).length;
  if (n > P.weight_width || min(n, P.keep) > P.new_width * P.t.page_rows) {
    if (tid == 0) atomicOr(P.t.status, kPagedStatusRange);
    n = 0;
  }
  const int m = min(n, P.keep);
  if (head == 0 && tid == 0) P.new_length[b] = m;
  const int64_t row = (int64_t)b * P.t.heads_kv + head;
  const float* w = P.weight_in + row * P.weight_width;
  float* out = P.weight != nullptr ? P.weight + row * P.weight_width : nullptr;
  int32_t* kept = P.kept + row * P.keep;
  for (int64_t j = m + tid; j < P.keep; j += kPickThreads) kept[j] = -1;
  if (n <= P.keep) {
    for (int j = tid; j < n; j += kPickThreads) {
      kept[j] = j;
      if (out != nullptr && out != w) out[j] = w[j];
    }
    return;
  }
  // The slots [lo, hi) compete for `places`.
  const int lo = P.first, hi = n - P.recent, places = P.keep - P.first - P.recent;
  const bool in_smem = n <= known;
  if (in_smem)
    for (int j = tid; j < n; j += kPickThreads) ranks[j] = rank_of(w[j]);
  auto rank_at = [&](int j) { return in_smem ? ranks[j] : rank_of(w[j]); };

  // The lowest rank that stays, and how many slots of that very rank do.
  uint32_t prefix = 0u, left = (uint32_t)places;
  if (places > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kPickThreads) bins[i] = 0u;
      __syncthreads();
      for (int j = lo + tid; j < hi; j += kPickThreads) {
        const uint32_t r = rank_at(j);
        if (pass == 0 || (r >> (shift + width)) == prefix) atomicAdd(&bins[(r >> shift) & ((1u << width) - 1u)], 1u);
      }
      __syncthreads();
      // From the highest bin down: the one in which `left` slots are reached.
      const int top = kBins - 1 - 2 * tid;
      const uint32_t a = bins[top], c = bins[top - 1];
      uint64_t total;
      const uint64_t sum = scan((uint64_t)a + c, sums, total);
      const uint64_t before = sum - a - c;
      if (before < left && sum >= left) {
        const bool second = before + a < left;
        found[0] = (uint32_t)(second ? top - 1 : top);
        found[1] = (uint32_t)(left - before - (second ? a : 0u));
      }
      __syncthreads();
      prefix = (prefix << width) | found[0];
      left = found[1];
      __syncthreads();
    }
  }
  // In order: slots that stay for certain, and of those of the lowest rank the first `left`.
  uint32_t sure_before = 0u, ties_before = 0u;
  for (int64_t j0 = 0; j0 < n; j0 += kPickThreads) {
    const int64_t j = j0 + tid;
    bool sure = false, tie = false;
    float wj = 0.f;
    if (j < n) {
      if (out != nullptr) wj = w[j];
      if (j < lo || j >= hi) {
        sure = true;
      } else if (places > 0) {
        const uint32_t r = rank_at((int)j);
        sure = r > prefix;
        tie = r == prefix;
      }
    }
    uint64_t total;  // (ends with barriers: the chunk's weights are read before any is written)
    const uint64_t sum = scan(((uint64_t)sure << 32) | (uint64_t)tie, sums, total);
    const uint32_t s = sure_before + (uint32_t)(sum >> 32) - (sure ? 1u : 0u);
    const uint32_t t = ties_before + (uint32_t)sum - (tie ? 1u : 0u);
    if (sure || (tie && t < left)) {
      const uint32_t to = s + min(t, left);
      RA_BOUNDS(P.t.status, to < (uint32_t)P.keep, 118);
      kept[to] = (int32_t)j;
      if (out != nullptr) out[to] = wj;
    }
    sure_before += (uint32_t)(total >> 32);
    ties_before += (uint32_t)total;
  }
}

constexpr int kMoveThreads = 256;
constexpr int kPiece = 64;                        // bytes of a row that a CTA moves
constexpr int kPassRows = kMoveThreads / (kPiece / 16);
constexpr int kUnroll = 4;                        // rows of a thread under way, twice

struct MoveRow {
  int64_t from, to;  // byte offsets; from < 0: nothing
};
__device__ __forceinline__ MoveRow move_row(const PagedEvictParams& P, int row_bytes, int b, int head, int which,
                                            const int32_t* kept, int m, int j) {
  if (j >= m) return {-1, 0};
  const int s = __ldg(kept + j);
  const int pr = P.t.page_rows;
  const int from_page = paged_page(P.t, b, s / pr);
  const int to_page = __ldg(P.new_table + b * P.new_width + j / pr);
  if (to_page < 0 || to_page >= P.t.pages) {
    atomicOr(P.t.status, kPagedStatusRange);
    return {-1, 0};
  }
  if (from_page < 0) return {-1, 0};
  const int64_t from = paged_row(P.t, from_page, which, head, s % pr), to = paged_row(P.t, to_page, which, head, j % pr);
  if (from == to) return {-1, 0};
  RA_BOUNDS(P.t.status, s >= j && from >= 0 && to >= 0, 119);
  return {from * row_bytes, to * row_bytes};
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const PagedEvictParams P, int row_bytes) {
  const int pieces = row_bytes / kPiece;
  const int which = (int)blockIdx.x / pieces, piece = (int)blockIdx.x % pieces;
  const int head = (int)blockIdx.y, b = (int)blockIdx.z;
  const int m = __ldg(P.new_length + b);
  const int32_t* kept = P.kept + ((int64_t)b * P.t.heads_kv + head) * P.keep;
  uint8_t* cache = static_cast<uint8_t*>(P.t.cache) + piece * kPiece + (threadIdx.x & 3) * 16;
  const int r0 = threadIdx.x >> 2;
  constexpr int kStep = kPassRows * kUnroll;
  uint4 x[2][kUnroll];
  int64_t to[2][kUnroll];
  auto load = [&](int j0, uint4 (&v)[kUnroll], int64_t (&t)[kUnroll]) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const MoveRow r = move_row(P, row_bytes, b, head, which, kept, m, j0 + i * kPassRows + r0);
      t[i] = r.from < 0 ? -1 : r.to;
      if (r.from >= 0) v[i] = __ldcg(reinterpret_cast<const uint4*>(cache + r.from));
    }
  };
  auto store = [&](const uint4 (&v)[kUnroll], const int64_t (&t)[kUnroll]) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
      if (t[i] >= 0) *reinterpret_cast<uint4*>(cache + t[i]) = v[i];
  };
  load(0, x[0], to[0]);
  for (int j0 = 0; j0 < m; j0 += 2 * kStep) {
    load(j0 + kStep, x[1], to[1]);
    __syncthreads();  // all rows up to here are read: their places may be written
    store(x[0], to[0]);
    load(j0 + 2 * kStep, x[0], to[0]);
    __syncthreads();
    store(x[1], to[1]);
  }
}

}  // namespace

cudaError_t launch_paged_evict(int dtype, const PagedEvictParams& prm, cudaStream_t stream) {
  const int known = (int)std::min<int64_t>(prm.weight_width, kMaxKnown);
  static std::atomic<int> ready[kMaxDevices];
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool cached = dev >= 0 && dev < kMaxDevices;
  if (!cached || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKnown * 4);
    if (e != cudaSuccess) return e;
    if (cached) ready[dev].store(1, std::memory_order_release);
  }
  const dim3 grid((unsigned)prm.t.heads_kv, (unsigned)prm.t.batch);
  pick_kernel<<<grid, kPickThreads, known * 4, stream>>>(prm, known);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int row_bytes = prm.d * (dtype == RA_DTYPE_BF16 ? 2 : 4);
  const dim3 moves((unsigned)(2 * row_bytes / kPiece), (unsigned)prm.t.heads_kv, (unsigned)prm.t.batch);
  move_kernel<<<moves, kMoveThreads, 0, stream>>>(prm, row_bytes);
  return cudaGetLastError();
}

}  // namespace ra
