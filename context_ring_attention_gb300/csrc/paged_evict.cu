// Eviction by accumulated attention weight (include/ra.h, ra_paged_evict): of every sequence
// and key/value head the `keep` slots that stay are the first ones, the most recent ones, and
// of the others the heaviest, ties to the lowest slot; they move together in their order.
//
// Two kernels.  The first decides: a cluster of CTAs per head and sequence (one CTA for short
// ones) finds the weight of the last slot that stays by its bits, 11 at a time from the top (a
// histogram in shared memory of the slots that agree so far, summed over the cluster), and lists
// the slots in order with a scan.  Counts are whole numbers: their order does not matter.
//
// The second moves rows, bound by HBM: the kept rows are read and written once.  Into other pages
// the CTAs take runs of rows.  In place a row's new one is never behind its old one, so that whoever
// has read all rows up to some place may write up to it: a cluster walks the whole list in order,
// its CTAs some rows of each step, for a piece of every row of a head's keys or values, reading a
// step ahead.  Where each row lies is looked up for many rows at once, before their turn.
//
// Measured (8 heads, D 128, bf16): 16 sequences of 4352 slots to 4096 (543 MB) into other pages 107
// us, in place 108; the choice alone takes 15.  33001 slots to 8192 (69 MB) into other pages 31 to 33
// us, of which the choice 20: bound by the latency of its three passes, barriers and the scan; in place
// 35 to 41.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "paged_internal.h"

namespace ra {
namespace {

namespace cg = cooperative_groups;

constexpr int kPickThreads = 1024;
constexpr int kBins = 2048;       // 11 bits a pass
constexpr int kMaxKnown = 49152;  // weights that a CTA keeps in shared memory
// 33001 slots of 8 heads to 8192 with clusters of up to 1, 2, 4 and 8 CTAs a head 43, 34, 31 and 31 us, to
// 32768 103, 81, 71 and 68; 100000 to 8192 403, 202, 42 and 37.
constexpr int kMaxCluster = 4;

// Whole numbers in the order of the weights: NaN lowest, then -inf .. +inf, -0 as +0.
__device__ __forceinline__ uint32_t rank_of(float w) {
  if (w != w) return 0u;
  const uint32_t x = __float_as_uint(w + 0.f);
  return (x & 0x80000000u) ? ~x : x | 0x80000000u;
}

// Inclusive sums over the CTA's threads; all of them in `total`.  sums: 32 places that the scan
// before did not have.  One barrier.
__device__ __forceinline__ uint64_t scan(uint64_t x, uint64_t* sums, uint64_t& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  uint64_t s = sums[lane];  // (every warp adds the warps up for itself)
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const uint64_t before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
  return warp > 0 ? x + before : x;
}

__global__ void __launch_bounds__(kPickThreads) pick_kernel(const PagedEvictParams P, int known) {
  extern __shared__ __align__(16) float weights[];  // [known]
  __shared__ uint32_t bins[3][kBins];  // of each pass
  __shared__ uint64_t sums[2][32];
  __shared__ uint32_t found[3][2];
  __shared__ uint64_t own_count;  // of this CTA's slots: sure << 32 | ties
  next_may_come();
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int head = (int)blockIdx.x / ctas, b = (int)blockIdx.y, tid = threadIdx.x;
  int n = paged_seq(P.t, b).length;
  if (n > P.weight_width || min(n, P.keep) > P.new_width * P.t.page_rows) {
    if (tid == 0) atomicOr(P.t.status, kPagedStatusRange);
    n = 0;
  }
  const int m = min(n, P.keep), all = ctas * kPickThreads, me = rank * kPickThreads + tid;
  if (head == 0 && me == 0) P.new_length[b] = m;
  const int64_t row = (int64_t)b * P.t.heads_kv + head;
  const float* w = P.weight_in + row * P.weight_width;
  float* out = P.weight != nullptr ? P.weight + row * P.weight_width : nullptr;
  int32_t* kept = P.kept + row * P.keep;
  for (int64_t j = m + me; j < P.keep; j += all) kept[j] = -1;
  if (n <= P.keep) {
    for (int j = me; j < n; j += all) {
      kept[j] = j;
      if (out != nullptr && out != w) out[j] = w[j];
    }
    return;
  }
  // This CTA's slots [s0, s1), their weights in shared memory where they fit.  (In place a weight
  // may be written over before another CTA has read it: then one CTA takes all, in order.)
  int s0 = (int)((int64_t)n * rank / ctas) & ~3, s1 = rank + 1 == ctas ? n : (int)((int64_t)n * (rank + 1) / ctas) & ~3;
  const bool in_smem = (n + ctas - 1) / ctas + 4 <= known;
  if (!in_smem && out == w) s0 = rank == 0 ? 0 : n, s1 = n;
  for (int i = tid; i < 3 * kBins; i += kPickThreads) (&bins[0][0])[i] = 0u;
  if (in_smem)
    for (int j = s0 + tid; j < s1; j += kPickThreads) weights[j - s0] = w[j];
  auto weight_at = [&](int j) { return in_smem ? weights[j - s0] : w[j]; };
  // The slots [lo, hi) compete for `places`.
  const int lo = P.first, hi = n - P.recent, places = P.keep - P.first - P.recent;

  // The lowest rank that stays, and how many slots of that very rank do.
  uint32_t prefix = 0u, left = (uint32_t)places;
  __syncthreads();
  if (places > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11;
      for (int j = max(s0, lo) + tid; j < min(s1, hi); j += kPickThreads) {
        const uint32_t r = rank_of(weight_at(j));
        if (pass == 0 || (r >> (shift + width)) == prefix) atomicAdd(&bins[pass][(r >> shift) & ((1u << width) - 1u)], 1u);
      }
      if (ctas > 1) cluster.sync();
      else __syncthreads();
      // From the highest bin down: the one in which `left` slots are reached.
      const int top = kBins - 1 - 2 * tid;
      uint32_t a = 0u, c = 0u;
      for (int i = 0; i < ctas; ++i) {
        const uint2 two = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&bins[pass][0], i) + top - 1);
        a += two.y, c += two.x;
      }
      uint64_t total;
      const uint64_t sum = scan((uint64_t)a + c, sums[pass & 1], total);
      const uint64_t before = sum - a - c;
      if (before < left && sum >= left) {
        const bool second = before + a < left;
        found[pass][0] = (uint32_t)(second ? top - 1 : top);
        found[pass][1] = (uint32_t)(left - before - (second ? a : 0u));
      }
      __syncthreads();
      prefix = (prefix << width) | found[pass][0];
      left = found[pass][1];
    }
  }
  // Slots that stay for certain, and those of the lowest rank, of which the first `left` do.
  auto kinds = [&](int j, bool& sure, bool& tie) {
    sure = tie = false;
    if (j >= s1) return;
    if (j < lo || j >= hi) {
      sure = true;
    } else if (places > 0) {
      const uint32_t r = rank_of(weight_at(j));
      sure = r > prefix;
      tie = r == prefix;
    }
  };
  auto emit = [&](int j, bool sure, bool tie, float wj, uint32_t& s, uint32_t& t) {
    if (sure || (tie && t < left)) {
      const uint32_t to = s + min(t, left);
      RA_BOUNDS(P.t.status, to < (uint32_t)P.keep, 118);
      kept[to] = j;
      if (out != nullptr) out[to] = wj;
    }
    s += sure, t += tie;
  };
  // A thread has a run of slots, of an odd number so that a warp's reads fall into different banks.
  const int own = ((s1 - s0 + kPickThreads - 1) / kPickThreads) | 1;
  const int j0 = (int)min((int64_t)s0 + (int64_t)own * tid, (int64_t)s1), j1 = min(j0 + own, s1);
  uint64_t mine = 0, total;
  for (int j = j0; j < j1; ++j) {
    bool sure, tie;
    kinds(j, sure, tie);
    mine += ((uint64_t)sure << 32) | (uint64_t)tie;
  }
  uint64_t before = scan(mine, sums[1], total) - mine;
  if (ctas > 1) {  // those of the CTAs before this one
    if (tid == 0) own_count = total;
    cluster.sync();
    for (int i = 0; i < rank; ++i) before += *cluster.map_shared_rank(&own_count, i);
    cluster.sync();  // (no CTA leaves while another reads its count)
  }
  if (in_smem || out != w) {
    uint32_t s = (uint32_t)(before >> 32), t = (uint32_t)before;
    for (int j = j0; j < j1; ++j) {
      bool sure, tie;
      kinds(j, sure, tie);
      emit(j, sure, tie, out != nullptr ? weight_at(j) : 0.f, s, t);
    }
    return;
  }
  // In place, more weights than shared memory holds (one CTA has them all): in order, a step's
  // weights read before any is written.
  before = 0;
  for (int64_t step = s0; step < s1; step += kPickThreads) {
    const int j = (int)min(step + tid, (int64_t)s1);
    bool sure, tie;
    kinds(j, sure, tie);
    const float wj = j < s1 ? weight_at(j) : 0.f;
    const uint64_t one = ((uint64_t)sure << 32) | (uint64_t)tie;
    __syncthreads();  // (the scan before has been read)
    const uint64_t sum = before + scan(one, sums[0], total) - one;
    uint32_t s = (uint32_t)(sum >> 32), t = (uint32_t)sum;
    emit(j, sure, tie, wj, s, t);
    before += total;
  }
}

constexpr int kMoveThreads = 256;
constexpr int kUnroll = 4;      // rows of a thread under way, twice
constexpr int kMaxTeam = 8;
constexpr int kBlock = 2048;    // rows whose places are looked up at a time: four steps or more

static_assert(kBlock >= 4 * (kMoveThreads / 4) * kUnroll, "a step's places are written two barriers before they are read");

// team: CTAs of a cluster.
__global__ void __launch_bounds__(kMoveThreads, 4) move_kernel(const PagedEvictParams P, int row_bytes, int pieces, int team) {
  __shared__ int2 places[2][kBlock];  // rows of the cache: from, to (from < 0: nothing to move)
  const int head = (int)blockIdx.y, b = (int)blockIdx.z;
  after_previous();
  const int m = P.new_length[b];
  if (m == 0) return;
  // The pages are the same, or none of them is: the first entry tells.
  const bool in_place = __ldg(P.new_table + b * P.new_width) == __ldg(P.t.page_table + b * P.t.width);
  // In place: cluster 2 * piece + which has a piece of every row, its CTAs a step of rows in turn.
  // Else: CTA 2 * run + which a run of rows.
  const int unit = in_place ? (int)blockIdx.x / team : (int)blockIdx.x, which = unit & 1, part = unit >> 1;
  const int rank = in_place ? (int)blockIdx.x % team : 0;
  if (!in_place) pieces = team = 1;
  else if (part >= pieces) return;  // (a whole cluster)
  const int piece = in_place ? part : 0, runs = in_place ? 1 : (int)gridDim.x >> 1, run = in_place ? 0 : part;
  const int piece_bytes = row_bytes / pieces, lanes = piece_bytes / 16, pass = kMoveThreads / lanes;
  const int r0 = (int)((int64_t)m * run / runs), r1 = (int)((int64_t)m * (run + 1) / runs);
  const int sub = threadIdx.x / lanes, step = pass * kUnroll;  // rows of this CTA a step: a power of two
  const int bits = __ffs(step) - 1;
  const int32_t* kept = P.kept + ((int64_t)b * P.t.heads_kv + head) * P.keep;
  const int pr = P.t.page_rows;
  auto look_up = [&](int block) {
    for (int i = threadIdx.x; i < kBlock; i += kMoveThreads) {
      const int k = block * kBlock + i, j = r0 + ((((k >> bits) * team + rank) << bits) | (k & (step - 1)));
      int2 at = make_int2(-1, 0);
      if (j < r1) {
        const int s = kept[j];
        const int from_page = paged_page(P.t, b, s / pr), to_page = __ldg(P.new_table + b * P.new_width + j / pr);
        if (to_page < 0 || to_page >= P.t.pages) {
          atomicOr(P.t.status, kPagedStatusRange);
        } else if (from_page >= 0) {
          at = make_int2((int)paged_row(P.t, from_page, which, head, s % pr), (int)paged_row(P.t, to_page, which, head, j % pr));
          if (at.x == at.y) at.x = -1;
          RA_BOUNDS(P.t.status, s >= j && at.y >= 0, 119);
        }
      }
      places[block & 1][i] = at;
    }
  };
  uint8_t* cache = static_cast<uint8_t*>(P.t.cache) + piece * piece_bytes + (threadIdx.x % lanes) * 16;
  const int steps = (r1 - r0 + step * team - 1) / (step * team), per_block = kBlock >> bits;  // (a power of two)
  uint4 x[2][kUnroll];
  auto place = [&](int s, int i) { return places[(s << bits) / kBlock & 1][((s & (per_block - 1)) << bits) + i * pass + sub]; };
  auto load = [&](int s, uint4 (&v)[kUnroll]) {
    if (s >= steps) return;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int from = place(s, i).x;
      if (from >= 0) v[i] = __ldcg(reinterpret_cast<const uint4*>(cache + (int64_t)from * row_bytes));
    }
  };
  auto store = [&](int s, const uint4 (&v)[kUnroll]) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int2 at = place(s, i);
      if (at.x >= 0) *reinterpret_cast<uint4*>(cache + (int64_t)at.y * row_bytes) = v[i];
    }
  };
  // Step s is stored once step s + 1 is read and all threads, of the whole cluster, have read step s.
  auto turn = [&](int s, const uint4 (&now)[kUnroll], uint4 (&next)[kUnroll]) {
    load(s + 1, next);
    if (team > 1) cg::this_cluster().sync();
    else __syncthreads();
    store(s, now);
    // (all threads have stored the block before this one; the next one is read two barriers on)
    if ((s & (per_block - 1)) == 0) look_up((s << bits) / kBlock + 1);
  };
  look_up(0);
  __syncthreads();
  load(0, x[0]);
  for (int s = 0; s < steps; s += 2) {
    turn(s, x[0], x[1]);
    if (s + 1 < steps) turn(s + 1, x[1], x[0]);
  }
}

}  // namespace

cudaError_t launch_paged_evict(int dtype, const PagedEvictParams& prm, int sm_count, cudaStream_t stream) {
  const int known = (int)std::min<int64_t>(prm.weight_width + 4, kMaxKnown);
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
  // A cluster where a sequence may be long and the heads are few (they are one wave then).
  const int64_t heads = (int64_t)prm.t.heads_kv * prm.t.batch;
  int ctas = 1;
  while (ctas < kMaxCluster && prm.weight_width > 4096 * ctas && 2 * ctas * heads <= sm_count) ctas *= 2;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3((unsigned)(prm.t.heads_kv * ctas), (unsigned)prm.t.batch);
  config.blockDim = dim3(kPickThreads);
  config.dynamicSmemBytes = (size_t)std::min<int64_t>(known, prm.weight_width / ctas + 8) * 4;
  config.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  config.attrs = &attr;
  config.numAttrs = 1;
  e = cudaLaunchKernelEx(&config, pick_kernel, prm, (int)(config.dynamicSmemBytes / 4));
  if (e != cudaSuccess) return e;
  const int row_bytes = prm.d * (dtype == RA_DTYPE_BF16 ? 2 : 4);
  // Pieces of 64 bytes at least, as many as fill the GPU twice; runs of rows until there are six
  // CTAs an SM (two to sixteen are within 4%; below 128 rows a run is too short for its start).
  int pieces = 1;
  while (row_bytes / pieces > 64 && 2 * pieces * heads < 2 * sm_count) pieces *= 2;
  const int64_t most = (prm.keep + 127) / 128;
  const int runs = (int)std::max<int64_t>(1, std::min(most, (int64_t)sm_count * 6 / (2 * pieces * heads)));
  // In place, clusters where the pieces leave the GPU idle (one sequence of 33001 slots to 8192:
  // clusters of 1, 2, 4, 8 CTAs 82, 65, 51, 41 us; to 32768: 247, 179, 123, 88).
  const int step = kMoveThreads * 16 * pieces / row_bytes * kUnroll;
  int team = 1;
  while (team < kMaxTeam && (int64_t)team * step < prm.keep && 2 * 2 * team * pieces * heads <= 4 * sm_count) team *= 2;
  cudaLaunchConfig_t move{};
  move.gridDim = dim3((unsigned)(2 * pieces * ((runs + team - 1) / team * team)), (unsigned)prm.t.heads_kv, (unsigned)prm.t.batch);
  move.blockDim = dim3(kMoveThreads);
  move.stream = stream;
  cudaLaunchAttribute how[2]{};
  how[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // as launch_behind
  how[0].val.programmaticStreamSerializationAllowed = 1;
  how[1].id = cudaLaunchAttributeClusterDimension;
  how[1].val.clusterDim.x = (unsigned)team;
  how[1].val.clusterDim.y = how[1].val.clusterDim.z = 1;
  move.attrs = how;
  move.numAttrs = 2;
  return cudaLaunchKernelEx(&move, move_kernel, prm, row_bytes, pieces, team);
}

}  // namespace ra
