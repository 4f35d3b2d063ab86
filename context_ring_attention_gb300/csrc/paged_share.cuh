// How the row kernels of the paged cache share out a packed batch: the sequences' query tiles
// (kRowsTile rows of one key/value head) laid in a row, each as long as the key blocks that it
// meets, and cut into as many equal shares as there are CTAs.  An item cut between CTAs is
// joined from its parts afterwards, in order.
#pragma once

#include "paged_internal.h"

namespace ra {

// Item t of a sequence: rows [row0, row0 + rows) of its count * group, at slots s0..s1.
struct PagedItem {
  int row0, rows, s0, s1;
};
template <int kR>
__device__ __forceinline__ PagedItem paged_item(const PagedSeq& q, int group, int t) {
  PagedItem it;
  it.row0 = t * kR;
  it.rows = min(kR, q.count * group - it.row0);
  it.s0 = q.slot0() + it.row0 / group;
  it.s1 = q.slot0() + (it.row0 + it.rows - 1) / group;
  return it;
}
// Units of an item: its key blocks; one where it meets none, so that a CTA writes its rows.
template <int kR, int kB>
__device__ __forceinline__ int paged_units(const PagedSeq& q, int group, int window, int sinks, int t) {
  const PagedItem it = paged_item<kR>(q, group, t);
  return max(1, PagedBlocks<kB>(paged_span(window, sinks, it.s0, it.s1)).n);
}

// prefix[1 ..] from the sequences' own numbers to their sums (a whole warp calls it).
__device__ __forceinline__ void paged_scan(int batch, int64_t* prefix) {
  const int lane = threadIdx.x & 31;
  int64_t before = 0;
  for (int b0 = 0; b0 < batch; b0 += 32) {
    int64_t x = b0 + lane < batch ? prefix[b0 + lane + 1] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (b0 + lane < batch) prefix[b0 + lane + 1] = before + x;
    before += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) prefix[0] = 0;
}

// Sums of the sequences' units: prefix[b] of the sequences before b, prefix[batch] of all.
// Every thread of the CTA calls it; it ends with a barrier.
template <int kR, int kB, int kWarps>
__device__ void paged_prefix(const PagedTable& t, int group, int window, int sinks, int64_t* prefix) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int b0 = warp * 32; b0 < t.batch; b0 += kWarps * 32) {
    // A lane has a sequence of one or two items (a decoding step's) for itself; the others' items
    // are shared out among the lanes.
    PagedSeq q{0, 0, 0};
    if (b0 + lane < t.batch) q = paged_seq(t, b0 + lane);
    const int tiles = paged_mine(t, q, group) ? (q.count * group + kR - 1) / kR : 0;
    int64_t sum = 0;
    if (tiles <= 2)
      for (int i = 0; i < tiles; ++i) sum += paged_units<kR, kB>(q, group, window, sinks, i);
    for (uint32_t many = __ballot_sync(0xffffffffu, tiles > 2); many; many &= many - 1) {
      const int src = __ffs(many) - 1;
      const PagedSeq o{0, __shfl_sync(0xffffffffu, q.count, src), __shfl_sync(0xffffffffu, q.length, src)};
      const int n = __shfl_sync(0xffffffffu, tiles, src);
      int64_t all = 0;
      for (int i = lane; i < n; i += 32) all += paged_units<kR, kB>(o, group, window, sinks, i);
#pragma unroll
      for (int e = 16; e > 0; e >>= 1) all += __shfl_xor_sync(0xffffffffu, all, e);
      if (lane == src) sum = all;
    }
    if (b0 + lane < t.batch) prefix[b0 + lane + 1] = sum;
  }
  __syncthreads();
  if (warp == 0) paged_scan(t.batch, prefix);
  __syncthreads();
}

// The last sequence that begins at x or before it and is not empty there.
__device__ __forceinline__ int paged_find(const int64_t* prefix, int batch, int64_t x) {
  int b = 0;
  for (int end = batch; end - b > 1;) {
    const int mid = (b + end) >> 1;
    (prefix[mid] <= x ? b : end) = mid;
  }
  return b;
}

// Item of sequence q that holds its unit y (a whole warp calls it): the item, and its first unit.
template <int kR, int kB>
__device__ __forceinline__ int paged_find_item(const PagedSeq& q, int group, int window, int sinks, int64_t y,
                                               int64_t& first) {
  const int lane = threadIdx.x & 31;
  const int tiles = (q.count * group + kR - 1) / kR;
  first = 0;
  for (int t0 = 0; t0 < tiles; t0 += 32) {
    const int64_t own = t0 + lane < tiles ? paged_units<kR, kB>(q, group, window, sinks, t0 + lane) : 0;
    int64_t x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t z = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += z;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, first + x > y);
    if (past) {
      const int src = __ffs(past) - 1;
      first += __shfl_sync(0xffffffffu, x - own, src);
      return t0 + src;
    }
    first += __shfl_sync(0xffffffffu, x, 31);
  }
  return tiles;
}

}  // namespace ra
