// Windowed attention forward, bf16, d = 128, on the sm_100-family tensor cores.
//
// What it computes: for the query at position i, with s_ij = scale * q_i.k_j over the
// keys it sees (j <= i and (j > i - window or j < sinks)),
//   m = max_j s_ij,  l = sum_j e^(s_ij - m),  O_i = sum_j e^(s_ij - m) v_j / l,
//   LSE_i = m + ln l,
// folded tile by tile with the running maximum and sum of Module 23, "The Math: One
// Block at a Time".  The planner lists, for every pair of query tiles, the key rows
// that some query of it sees, shard by shard in ring order (win_internal.h); a key
// tile starts at the first row that is seen (striped layouts walked by position: at the
// start of its stripe), not at a multiple of 128.
//
// A windowed item meets few key tiles (9 for a 1024-token window, against hundreds of
// a full causal prefix), so what matters is the seam between two items.  The stream of
// (item, key tile) pairs is one stream: the products of the next item's first key tile
// are issued as those of any next tile are, while the softmax of the current item's
// last tile runs; a query tile's shared memory is handed back to the loads as soon as
// its last score product is done; the next item's first K and V tiles are requested
// before its queries.  Items cost nearly the same, so CTA b takes items b, b + grid,
// ... of a list sorted by cost and key/value head: no counter, and launches of one
// plan need no reset between them.
//
// Measured, 32 query and 8 key/value heads: 32768 tokens in 8 zigzag shards, window 4096 and 4
// sinks, 1.30 to 1.39 ms by the clock, 0.77 to 0.82 of the tensor cores' measured rate on the
// visible pairs; 131072 tokens in 32 contiguous shards, window 1024 and 64 sinks, 1.87 to 1.98
// ms (0.61 to 0.64: a pair of query tiles meets 10 key tiles, of which the two at the window's
// edges and the sinks' are partly empty); 900 tokens of 4 heads 13 us.  The first workload's
// eight partials in one launch 2.58 ms (4.3 GB of fp32 rows, a thread writing its own row in
// 16-byte pieces), ring steps 0.12 ms (no keys) to 0.64, the ring driver 3.95.  What bounds it: each softmax thread has a row of 128 scores to bring from
// tensor memory and back per product pair, and the two query tiles' softmax and products
// overlap only so far (tensor cores 59% busy at 32768 tokens and a window of 1024).
//
// Roles (one persistent CTA per SM, 12 warps): warp 0 TMA producer, warp 1 tcgen05
// issuer (both converged, one elected lane issues), warp 2 the work items' records, warp 3
// (partials) the rows of items that meet no key in the launch's steps, warps 4-7 softmax of
// query tile 0, warps 8-11 of query tile 1 (one thread per row).
// TMEM: S0 cols 0-127 (P0 in 64-127), S1 128-255 (P1 in 192-255), O0 256-383,
// O1 384-511 (all 512 columns).
//
// Every mbarrier wait is bounded (~1 s).  On expiry the CTA raises an abort flag,
// records the role in the plan's status word, drains its own in-flight TMA loads and
// MMAs (bounded again), frees TMEM and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "sm100_ptx.cuh"
#include "win_internal.h"

namespace ra {
namespace {

constexpr int kThreads = 384;  // 3 warpgroups: {producer, MMA, 2 idle}, softmax 0, softmax 1
constexpr uint32_t kRegsLaunch = 168;
constexpr uint32_t kRegsOther = 120;
constexpr uint32_t kRegsSoftmax = 192;
static_assert(128 * kRegsOther + 256 * kRegsSoftmax <= kThreads * kRegsLaunch, "register split");
constexpr uint32_t kTileBytes = 128 * 128 * 2;  // one 128 x 128 bf16 tile
constexpr uint32_t kHalfBytes = 128 * 64 * 2;   // 128 rows x one 128-byte swizzle column
constexpr int kStages = 3;                      // K/V ring: 4 and 5 were no faster (131072 tokens: 2061, 2106 against 2043 us)
constexpr int kItemSlots = 4;                   // work items under way from the record warp to the others
constexpr int kSlotRanges = 12;                 // ranges of an item kept with it (more are read from memory)
constexpr uint32_t kStageRow = 144;             // 128 bytes of an output row, and 16 so that the lanes'
                                                // 16-byte writes fall into different banks
constexpr uint32_t kOffQ = 0;                   // Q0, Q1
constexpr uint32_t kOffKV = 2 * kTileBytes;
constexpr uint32_t kOffOut = kOffKV + kStages * kTileBytes;  // half rows of O on their way out
constexpr uint32_t kOffRec = kOffOut + 256 * kStageRow;
struct alignas(16) Record {
  WinItem it;
  int32_t x0, xn;  // its ranges within this launch: P.ranges[x0 .. x0 + xn)
  int32_t pad[2];
  WinRange ranges[kSlotRanges];
};
constexpr uint32_t kOffBar = kOffRec + kItemSlots * (uint32_t)sizeof(Record);

enum : int {
  kQFull = 0,               // one per query tile
  kQEmpty = kQFull + 2,
  kKVFull = kQEmpty + 2,
  kKVEmpty = kKVFull + kStages,
  kSFull = kKVEmpty + kStages,
  kPFull = kSFull + 2,
  kOFull = kPFull + 2,
  kDone = kOFull + 2,
  kItemFull = kDone + 1,
  kItemEmpty = kItemFull + kItemSlots,
  kNumBars = kItemEmpty + kItemSlots
};
constexpr uint32_t kItemConsumers = 10;  // producer, MMA and 8 softmax warps
constexpr uint32_t kOffSlot = kOffBar + 8 * kNumBars;  // TMEM base written by tcgen05.alloc
constexpr uint32_t kOffAbort = kOffSlot + 4;
constexpr uint32_t kSmemBytes = kOffBar + 256 + 1024;  // + slack to align the base to 1 KiB
static_assert(8 * kNumBars + 8 <= 256 && kOffBar % 16 == 0 && kSmemBytes <= 232448, "shared memory");

constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t col_s(int g) { return g ? 128u : 0u; }
__device__ __forceinline__ uint32_t col_o(int g) { return g ? 384u : 256u; }
// P (bf16, two per 32-bit column) overwrites the upper half of its tile's S columns
// once the softmax has read S; the next S MMA of that tile is issued after the PV
// MMA that reads P.
constexpr uint32_t kColP = 64;

constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(128, 128, false, false);  // Q, K both K-major
constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(128, 128, false, true);  // V is MN-major
constexpr uint64_t kWaitBudgetNs = 1000000000ull;
constexpr uint32_t kSuspendHintNs = 2000u;  // a waiting thread sleeps up to this long per try
constexpr float kRescaleSlack = 8.0f;  // log2 units: keep a stale max while p <= 2^8
constexpr float kLn2 = 0.6931471805599453f;

struct Ctl {
  uint32_t bars;
  volatile uint32_t* abort;
  uint32_t* status;
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * (uint32_t)i; }
};

// Bounded wait for phase `parity` of a barrier; false on abort or expiry.
__device__ __forceinline__ bool wait_bar(const Ctl& c, uint32_t bar, uint32_t parity, uint32_t who) {
  if (ptx::mbar_test(bar, parity)) return true;
  const uint64_t t0 = ptx::global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (ptx::mbar_wait_hint(bar, parity, kSuspendHintNs)) return true;
    if ((it & 15u) == 0) {
      if (*c.abort) return false;
      if (ptx::global_timer_ns() - t0 > kWaitBudgetNs) {
        *c.abort = 1u;
        atomicOr(c.status, who);
        return false;
      }
    }
  }
}

// Teardown wait: ignores the abort flag, still bounded.
__device__ __forceinline__ void drain_bar(const Ctl& c, uint32_t bar, uint32_t parity) {
  const uint64_t t0 = ptx::global_timer_ns();
  while (!ptx::mbar_test(bar, parity)) {
    if (ptx::global_timer_ns() - t0 > kWaitBudgetNs) {
      atomicOr(c.status, kStatusTimeoutTeardown);
      return;
    }
  }
}

#define RA_WAIT(n, phase, who) __all_sync(0xffffffffu, wait_bar(c, c.bar(n), (phase) & 1u, who))

// 4-D tiled load (element of a row, row of the stripe, stripe, head); a converged warp
// executes it and one elected lane issues.
__device__ __forceinline__ void tma_load_4d_warp_hint(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                                      int32_t i, int32_t bh, uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(0), "r"(i), "r"(bh), "l"(policy)
      : "memory");
}
// ------------------------------------------------------------------- records --
// The item's ranges that belong to the steps of this launch (they are in the order of their
// steps): P.ranges[x0 .. x0 + xn).  A whole warp calls it, w is the item's record, 16 bytes a lane.
__device__ __forceinline__ void ranges_of_launch(const WinParams& P, const int4& w, int lane, int& x0, int& xn) {
  x0 = __shfl_sync(0xffffffffu, w.z, 1);  // range0
  xn = __shfl_sync(0xffffffffu, w.w, 1);  // n_ranges
  if (P.step_lo == 0 && P.step_hi >= P.k.shards) return;
  int before = 0, in = 0;
  for (int k = 0; k < xn; k += 32) {
    const int step = k + lane < xn ? P.ranges[x0 + k + lane].step : P.step_hi;
    before += __popc(__ballot_sync(0xffffffffu, step < P.step_lo));
    in += __popc(__ballot_sync(0xffffffffu, step >= P.step_lo && step < P.step_hi));
  }
  x0 += before;
  xn = in;
}
__device__ __forceinline__ int4 item_words(const WinParams& P, int idx, int lane) {
  return lane < 3 ? reinterpret_cast<const int4*>(P.items + idx)[lane] : make_int4(0, 0, 0, 0);
}

// Warp 2 brings the items and their ranges of this CTA into shared memory, a few items
// ahead: reading them where they are needed took each role 1 to 2 us at every item.  Items that
// meet no key in the launch's steps are not among them: the MMA warp asks for the next item
// before it issues the last product that the softmax warps wait for, and a row of such items,
// each to be given back by all roles, would fill the slots meanwhile, for good.
__device__ void run_records(const WinParams& P, const Ctl& c, Record* recs, int lane) {
  int idx = (int)blockIdx.x;
  for (uint32_t u = 0;; ++u, idx += (int)gridDim.x) {
    int4 w;
    int x0 = 0, xn = 0;
    for (; idx < P.n_items; idx += (int)gridDim.x) {
      w = item_words(P, idx, lane);
      ranges_of_launch(P, w, lane, x0, xn);
      if (xn > 0) break;
    }
    const uint32_t slot = u % kItemSlots;
    if (!RA_WAIT(kItemEmpty + (int)slot, (u / kItemSlots) ^ 1u, kStatusTimeoutProducer)) return;
    Record& r = recs[slot];
    const bool end = idx >= P.n_items;
    if (end) {
      if (lane == 0) r.it.bh0 = -1;
    } else {
      if (lane < 3) reinterpret_cast<int4*>(&r.it)[lane] = w;
      if (lane == 0) {
        r.x0 = x0;
        r.xn = xn;
      }
      if (lane < kSlotRanges && lane < xn)
        *reinterpret_cast<int4*>(&r.ranges[lane]) = *reinterpret_cast<const int4*>(&P.ranges[x0 + lane]);
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(c.bar(kItemFull + (int)slot));
    if (end) return;
  }
}

// Row of [batch, heads, S] that row `row` of an item's tile g is (-1: none).
__device__ __forceinline__ int64_t row_of_tile(const WinParams& P, const WinItem& it, int g, int row) {
  const int i = (g ? it.row1 : it.row0) + row;
  if (i >= it.row_end || row >= P.q.tile) return -1;
  const int head_row = it.shard * P.q.s_n + i;
  return (int64_t)(g ? it.bh1 : it.bh0) * P.seq +
         (P.q.stripe == 1 ? head_row : head_row % P.q.stripe * (P.seq / P.q.stripe) + head_row / P.q.stripe);
}

// Partials, warp 3: the rows of the items that meet no key in the launch's steps, O_t = 0 and
// LSE_t = -inf in each of them.  (Partials are walked shard by shard: a tile's rows follow each
// other in the tensor.)
__device__ void run_empty(const WinParams& P, int lane) {
  const int64_t rows_all = (int64_t)P.batch * P.heads_q * P.seq;
  for (int idx = (int)blockIdx.x; idx < P.n_items; idx += (int)gridDim.x) {
    const int4 w = item_words(P, idx, lane);
    int x0, xn;
    ranges_of_launch(P, w, lane, x0, xn);
    if (xn > 0) continue;
    const WinItem it = P.items[idx];
    for (int g = 0; g < (it.bh1 >= 0 ? 2 : 1); ++g) {
      const int left = it.row_end - (g ? it.row1 : it.row0), rows = left < P.q.tile ? left : P.q.tile;
      const int64_t first = row_of_tile(P, it, g, 0);
      RA_BOUNDS(P.status, P.q.stripe == 1 && first >= 0 && first + rows <= rows_all, 66);
      for (int part = 0; part < P.step_hi - P.step_lo; ++part) {
        float4* o = reinterpret_cast<float4*>(P.o_parts + ((int64_t)part * rows_all + first) * 128) + lane;
#pragma unroll 8
        for (int row = 0; row < rows; ++row) o[row * 32] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int row = lane; row < rows; row += 32) P.lse_parts[(int64_t)part * rows_all + first + row] = -INFINITY;
      }
    }
  }
}

// Consumer side: the record of this role's u-th item (nullptr at the end or on abort), and
// giving it back.
__device__ __forceinline__ const Record* next_record(const Ctl& c, const Record* recs, uint32_t u, uint32_t who) {
  const uint32_t slot = u % kItemSlots;
  if (!RA_WAIT(kItemFull + (int)slot, u / kItemSlots, who)) return nullptr;
  return recs[slot].it.bh0 < 0 ? nullptr : recs + slot;
}
__device__ __forceinline__ void release_record(const Ctl& c, uint32_t u, int lane) {
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(c.bar(kItemEmpty + (int)(u % kItemSlots)));
}
__device__ __forceinline__ WinRange range_at(const WinParams& P, const Record* r, int k) {
  return k < kSlotRanges ? r->ranges[k] : P.ranges[r->x0 + k];
}

// ------------------------------------------------------------------ producer --
struct ProducerState {
  uint32_t kv_issued, q_issued[2];
};

__device__ void run_producer(const WinParams& P, const Ctl& c, uint32_t sbase, const Record* recs,
                             const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv, ProducerState& st,
                             int lane) {
  const uint64_t keep = ptx::l2_policy_evict_last();   // K/V: re-read by the CTAs running together
  const uint64_t once = ptx::l2_policy_evict_first();  // Q: read once
  const uint32_t kv_bytes = (uint32_t)P.k.tile * 256u, q_bytes = (uint32_t)P.q.tile * 256u;
  auto load_kv = [&](int32_t i, int32_t bh) {  // K tile, then V tile
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const uint32_t s = st.kv_issued % kStages, use = st.kv_issued / kStages;
      if (!RA_WAIT(kKVEmpty + (int)s, use ^ 1u, kStatusTimeoutProducer)) return false;
      const uint32_t dst = sbase + kOffKV + s * kTileBytes;
      const CUtensorMap* map = which ? tv : tk;
      ptx::mbar_arrive_expect_tx_warp(c.bar(kKVFull + (int)s), kv_bytes);
      tma_load_4d_warp_hint(dst, map, c.bar(kKVFull + (int)s), 0, i, bh, keep);
      tma_load_4d_warp_hint(dst + kHalfBytes, map, c.bar(kKVFull + (int)s), 64, i, bh, keep);
      ++st.kv_issued;
    }
    return true;
  };
  for (uint32_t u = 0;; ++u) {
    const Record* r = next_record(c, recs, u, kStatusTimeoutProducer);
    if (r == nullptr) return;
    const WinItem it = r->it;
    RA_BOUNDS(c.status, it.shard >= 0 && it.shard < P.q.shards && it.row0 >= 0 && it.row0 < P.q.s_n && it.row1 < P.q.s_n, 60);
    const int kv_bh = it.bh0 / P.heads_q * P.heads_kv + (it.bh0 % P.heads_q) / P.group;
    RA_BOUNDS(c.status, kv_bh >= 0 && kv_bh < P.batch * P.heads_kv, 61);
    bool q_loaded = false;
    for (int k = 0; k < r->xn; ++k) {
      const WinRange rg = range_at(P, r, k);
      const int slot = P.kv_rotated ? it.shard : rg.r;  // where the block of the step sits
      RA_BOUNDS(c.status, slot >= 0 && slot < P.k.shards && rg.row0 >= 0 && rg.row0 < rg.end && rg.end <= P.k.s_n &&
                              rg.row0 % P.k.stripe == 0, 61);
      int32_t i = (slot * P.k.s_n + rg.row0) / P.k.stripe;
      for (int n = range_tiles(rg, P.k.tile); n > 0; --n, i += P.k.tile / P.k.stripe) {
        RA_BOUNDS(c.status, i >= 0 && i < P.seq / P.k.stripe, 61);
        if (!load_kv(i, kv_bh)) return;
        if (q_loaded) continue;
        q_loaded = true;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (g == 1 && it.bh1 < 0) break;
          if (!RA_WAIT(kQEmpty + g, st.q_issued[g] ^ 1u, kStatusTimeoutProducer)) return;
          const int32_t iq = (it.shard * P.q.s_n + (g ? it.row1 : it.row0)) / P.q.stripe;
          const int32_t bh = g ? it.bh1 : it.bh0;
          RA_BOUNDS(c.status, iq >= 0 && iq < P.seq / P.q.stripe && bh < P.batch * P.heads_q, 62);
          ptx::mbar_arrive_expect_tx_warp(c.bar(kQFull + g), q_bytes);
          tma_load_4d_warp_hint(sbase + kOffQ + g * kTileBytes, tq, c.bar(kQFull + g), 0, iq, bh, once);
          tma_load_4d_warp_hint(sbase + kOffQ + g * kTileBytes + kHalfBytes, tq, c.bar(kQFull + g), 64, iq, bh, once);
          ++st.q_issued[g];
        }
      }
    }
    release_record(c, u, lane);
  }
}

// ----------------------------------------------------------------------- MMA --
constexpr uint32_t kTileDesc = kTileBytes >> 4;  // one tile in descriptor address units

__device__ __forceinline__ void issue_s(uint32_t q0, uint32_t k0, uint32_t tmem, int g, uint32_t ks) {
  const uint32_t a0 = q0 + (uint32_t)g * kTileDesc, b0 = k0 + ks * kTileDesc;
#pragma unroll
  for (uint32_t kk = 0; kk < 8; ++kk) {  // 8 steps of K = 16 over d = 128
    const uint32_t off = ((kk >> 2) * kHalfBytes + (kk & 3u) * 32u) >> 4;
    ptx::mma_bf16_ss_lo_warp(tmem + col_s(g), a0 + off, b0 + off, kIdescS, kk > 0 ? 1u : 0u);
  }
}

// (Products of fewer keys for the sinks' tile, by a descriptor and a count held in
// registers, cost 2.5% in the issue and gained nothing: the tile's time is the softmax's.)
__device__ __forceinline__ void issue_pv(uint32_t v0, uint32_t tmem, int g, uint32_t vs, bool accumulate) {
  const uint32_t a0 = tmem + col_s(g) + kColP;  // P in tensor memory
  const uint32_t b0 = v0 + vs * kTileDesc;
#pragma unroll
  for (uint32_t kk = 0; kk < 8; ++kk)  // 8 steps of 16 keys = 8 TMEM columns of P
    // V is [keys][d]: 16 keys = 2 groups of 8 rows (SBO 1 KiB); d halves 16 KiB apart (LBO).
    ptx::mma_bf16_ts_lo_warp(tmem + col_o(g), a0 + kk * 8u, b0 + ((kk * 2048u) >> 4), kIdescPV,
                             (accumulate || kk > 0) ? 1u : 0u);
}

// A segment is a run of key tiles folded into one (O, LSE): a whole item, or
// (partials) one ring step of it.
struct Seg {
  int n;             // key tiles
  bool two;          // two query tiles
  bool first, last;  // first / last segment of its item
};
template <bool kPartials>
struct SegWalk {
  uint32_t u;      // record in hand, or the next one
  int k;           // partials: next range of it; -1: none in hand
  const Record* r;
  __device__ __forceinline__ void begin() {
    u = 0;
    k = -1;
  }
  __device__ __forceinline__ bool next(const WinParams& P, const Ctl& c, const Record* recs, int lane, Seg& s) {
    if (!kPartials) {
      r = next_record(c, recs, u, kStatusTimeoutMma);
      if (r == nullptr) return false;
      s = {r->it.n_tiles, r->it.bh1 >= 0, true, true};
      release_record(c, u++, lane);
      return true;
    }
    s.first = k < 0;
    if (k < 0) {
      r = next_record(c, recs, u, kStatusTimeoutMma);
      if (r == nullptr) return false;
      k = 0;
    }
    s.two = r->it.bh1 >= 0;
    const int step = range_at(P, r, k).step;
    s.n = 0;
    for (; k < r->xn; ++k) {
      const WinRange rg = range_at(P, r, k);
      if (rg.step != step) break;
      s.n += range_tiles(rg, P.k.tile);
    }
    s.last = k == r->xn;
    if (s.last) {
      release_record(c, u++, lane);
      k = -1;
    }
    return true;
  }
};

template <bool kPartials>
__device__ void run_mma(const WinParams& P, const Ctl& c, uint32_t sbase, const Record* recs, uint32_t tmem, int lane) {
  const uint32_t q0 = ptx::desc_lo(sbase + kOffQ, 16);
  const uint32_t k0 = ptx::desc_lo(sbase + kOffKV, 16);
  const uint32_t v0 = ptx::desc_lo(sbase + kOffKV, kHalfBytes);
  // the column map (S0, S1, O0, O1 = 0, 128, 256, 384) needs all 512 columns from 0
  RA_BOUNDS(c.status, tmem == 0u && col_o(1) + 128u <= kTmemCols, 63);
  uint32_t kv = 0, pj[2] = {0, 0}, qj[2] = {0, 0};
  SegWalk<kPartials> walk;
  walk.begin();
  Seg cur, nxt;
  if (!walk.next(P, c, recs, lane, cur)) return;
  // Scores of a segment's key tile: the queries arrive with an item's first tile, and
  // their shared memory is free for the next item's after its last.
  auto scores = [&](const Seg& s, int kt, int g, uint32_t ks) {
    if (s.first && kt == 0) {
      if (!RA_WAIT(kQFull + g, qj[g], kStatusTimeoutMma)) return false;
      ++qj[g];
    }
    issue_s(q0, k0, tmem, g, ks);
    ptx::mma_commit_warp(c.bar(kSFull + g));
    if (s.last && kt == s.n - 1) ptx::mma_commit_warp(c.bar(kQEmpty + g));
    return true;
  };
  uint32_t ks = kv % kStages;
  // Waits on TMA-filled buffers need no tcgen05 fence: the mbarrier completion
  // already orders the async-proxy writes before the MMAs that read them.
  if (!RA_WAIT(kKVFull + (int)ks, kv / kStages, kStatusTimeoutMma)) return;
  if (!scores(cur, 0, 0, ks)) return;
  if (cur.two && !scores(cur, 0, 1, ks)) return;
  ptx::mma_commit_warp(c.bar(kKVEmpty + (int)ks));
  ++kv;
  for (int kt = 0;;) {
    const bool seg_last = kt == cur.n - 1;
    bool has_next = true;
    int nkt = kt + 1;
    nxt = cur;
    if (seg_last) {
      has_next = walk.next(P, c, recs, lane, nxt);
      nkt = 0;
    }
    const uint32_t vs = kv % kStages;
    if (!RA_WAIT(kKVFull + (int)vs, kv / kStages, kStatusTimeoutMma)) return;
    ++kv;
    if (!RA_WAIT(kPFull + 0, pj[0], kStatusTimeoutMma)) return;
    ++pj[0];
    ptx::tc_fence_after();
    issue_pv(v0, tmem, 0, vs, kt > 0);
    if (seg_last) ptx::mma_commit_warp(c.bar(kOFull + 0));
    if (has_next) {
      ks = kv % kStages;
      if (!RA_WAIT(kKVFull + (int)ks, kv / kStages, kStatusTimeoutMma)) return;
      ptx::tc_fence_after();
      if (!scores(nxt, nkt, 0, ks)) return;
    }
    if (cur.two) {
      if (!RA_WAIT(kPFull + 1, pj[1], kStatusTimeoutMma)) return;
      ++pj[1];
      ptx::tc_fence_after();
      issue_pv(v0, tmem, 1, vs, kt > 0);
      if (seg_last) ptx::mma_commit_warp(c.bar(kOFull + 1));
    }
    ptx::mma_commit_warp(c.bar(kKVEmpty + (int)vs));
    if (!has_next) break;
    if (nxt.two && !scores(nxt, nkt, 1, ks)) return;
    ptx::mma_commit_warp(c.bar(kKVEmpty + (int)ks));
    ++kv;
    cur = nxt;
    kt = nkt;
  }
}

// ------------------------------------------------------------------- softmax --
// The lowest n bits (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : ~(~0u << n)); }

// The finished rows of a segment.  bf16 rows go out through shared memory, half a row at a
// time, so that 8 lanes write 128 consecutive bytes: written from where they stand, every
// 16-byte store of a warp touches 32 lines, and the rows of an item took 1.4 to 2.2 us.
// (Sent from shared memory as a bulk copy per row they took 2.6.)
template <bool kPartials>
__device__ __forceinline__ void store_segment(const WinParams& P, uint32_t tO, uint8_t* stage, float m, float l,
                                              float fix, bool valid, int64_t out_row, int part, int lane) {
  const float inv = l > 0.f ? 1.0f / (l + fix) : 0.f;
  const float lse = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
  const int64_t rows_all = (int64_t)P.batch * P.heads_q * P.seq;
  const int to = valid ? (int)out_row : -1;  // (rows fit in 31 bits)
#pragma unroll 1
  for (int cc = 0; cc < 2; ++cc) {
    uint32_t v[64];
    __syncwarp();
    ptx::tmem_ld32x2(tO + cc * 64, tO + cc * 64 + 32, v);
    if (kPartials) {
      if (!valid) continue;
      float4* dst = reinterpret_cast<float4*>(P.o_parts + ((int64_t)part * rows_all + out_row) * 128);
#pragma unroll
      for (int q = 0; q < 16; ++q)
        dst[cc * 16 + q] = make_float4(__uint_as_float(v[4 * q]) * inv, __uint_as_float(v[4 * q + 1]) * inv,
                                       __uint_as_float(v[4 * q + 2]) * inv, __uint_as_float(v[4 * q + 3]) * inv);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = ptx::pack_bf16x2(__uint_as_float(v[8 * q + 2 * e]) * inv, __uint_as_float(v[8 * q + 2 * e + 1]) * inv);
        *reinterpret_cast<uint4*>(stage + lane * kStageRow + q * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 8; ++q) {  // rows 4q .. 4q + 3
        const int r = 4 * q + (lane >> 3);
        const uint4 x = *reinterpret_cast<const uint4*>(stage + r * kStageRow + (lane & 7) * 16);
        const int row = __shfl_sync(0xffffffffu, to, r);
        if (row >= 0) reinterpret_cast<uint4*>(P.o)[(int64_t)row * 16 + cc * 8 + (lane & 7)] = x;
      }
    }
  }
  if (valid) {
    if (kPartials) P.lse_parts[(int64_t)part * rows_all + out_row] = lse;
    else if (P.lse != nullptr) P.lse[out_row] = lse;
  }
}

// A ring step in which the item's rows meet no key: O_t = 0, LSE_t = -inf.
__device__ __forceinline__ void store_empty(const WinParams& P, bool valid, int64_t out_row, int part) {
  if (!valid) return;
  const int64_t rows_all = (int64_t)P.batch * P.heads_q * P.seq;
  float4* dst = reinterpret_cast<float4*>(P.o_parts + ((int64_t)part * rows_all + out_row) * 128);
  for (int q = 0; q < 32; ++q) dst[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  P.lse_parts[(int64_t)part * rows_all + out_row] = -INFINITY;
}

template <bool kPartials>
__device__ void run_softmax(const WinParams& P, const Ctl& c, uint8_t* stage, const Record* recs, uint32_t tmem, int g,
                            int wq, int lane) {
  const int row = wq * 32 + lane;  // TMEM lane = query row of the tile
  const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
  const uint32_t tS = tmem + lane_off + col_s(g);
  const uint32_t tO = tmem + lane_off + col_o(g);
  RA_BOUNDS(c.status, wq >= 0 && wq < 4 && (tS & 0xFFFFu) + 128u <= kTmemCols && (tO & 0xFFFFu) + 128u <= kTmemCols &&
                          (tS & 0xFFFFu) + kColP + 64u <= kTmemCols, 64);
  const float sl2 = P.scale_log2;
  uint32_t sj = 0, oj = 0;

  for (uint32_t u = 0;; ++u) {
    const Record* rec = next_record(c, recs, u, kStatusTimeoutSoftmax);
    if (rec == nullptr) return;
    const WinItem it = rec->it;
    const int xn = g == 1 && it.bh1 < 0 ? -1 : rec->xn;
    if (xn < 0) {
      release_record(c, u, lane);
      continue;
    }
    const int64_t out_row = row_of_tile(P, it, g, row);
    const bool valid = out_row >= 0;
    const int my_pos = (g ? it.pos1 : it.pos0) + row * P.q.apart;  // (of rows that are not valid: any)
    RA_BOUNDS(c.status, !valid || ((g ? it.bh1 : it.bh0) >= 0 && out_row < (int64_t)P.batch * P.heads_q * P.seq), 65);

    float m = -INFINITY, l = 0.f, fix = 0.f;
    bool first = true;
    int next_part = P.step_lo;  // partials: steps below are written
    for (int k = 0; k < xn; ++k) {
      const WinRange rg = range_at(P, rec, k);
      const bool seg_end = k == xn - 1 || (kPartials && range_at(P, rec, k + 1).step != rg.step);
      if (kPartials)
        for (; next_part < rg.step; ++next_part) store_empty(P, valid, out_row, next_part - P.step_lo);
      const WinColumns seen = range_columns(rg, P.k.apart, P.window, P.sinks, my_pos);
      const int n = range_tiles(rg, P.k.tile);
      for (int kt = 0; kt < n; ++kt) {
        const int y = kt * P.k.tile;
        const bool last = seg_end && kt == n - 1;
        // columns [c_lo, c_hi), and those below c_s, are seen
        const int c_hi = seen.hi - y < P.k.tile ? seen.hi - y : P.k.tile, c_lo = seen.lo - y;
        const int c_s = seen.sk - y < c_hi ? seen.sk - y : c_hi;
        const bool full = c_hi >= kTileRows && (c_lo <= 0 || c_s >= kTileRows);

        bool ok = wait_bar(c, c.bar(kSFull + g), sj & 1u, kStatusTimeoutSoftmax);
        ++sj;
        if (!__all_sync(0xffffffffu, ok)) return;
        ptx::tc_fence_after();

        // The tile's weights into tensor memory, their sum into part, the rounding of the
        // largest into top_fix; m moves when the tile's largest score exceeds it by the
        // slack.  Two copies of the code: without a mask the loop over the columns stays
        // free of branches, which the tiles inside the window need.
        bool resc = false;
        float alpha = 1.0f, part_sum, top_fix;
        auto weights = [&](auto edge) {
          // The whole 128-column score row in registers (one TMEM round trip); the
          // reducing load also returns the largest score of each 32 columns.
          uint32_t raw[128];
          float mx4[4];
          ptx::tmem_ld128_max(tS, raw, mx4);
          float* s = reinterpret_cast<float*>(raw);
          // At an edge of the window, on the diagonal and in the sinks, 32 columns at a
          // time: columns that no row of the warp sees are left out of the exponentials,
          // those that all see need no mask, and in the others the keys that are not seen
          // score -inf.
          uint32_t live = 15u;
          if (decltype(edge)::value) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t bits = (below(c_hi - 32 * q) & ~below(c_lo - 32 * q)) | below(c_s - 32 * q);
              if (!__any_sync(0xffffffffu, bits != 0u)) {
                live &= ~(1u << q);
                mx4[q] = -INFINITY;
              } else if (!__all_sync(0xffffffffu, bits == ~0u)) {
#pragma unroll
                for (int e = 0; e < 32; ++e) s[32 * q + e] = ((bits >> e) & 1u) ? s[32 * q + e] : -INFINITY;
                float a[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] = ptx::max3(s[32 * q + e], s[32 * q + e + 4], s[32 * q + e + 8]);
#pragma unroll
                for (int n2 = 12; n2 < 28; n2 += 8)
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    a[e] = ptx::max3(a[e], s[32 * q + n2 + e], s[32 * q + n2 + e + 4]);
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] = fmaxf(a[e], s[32 * q + 28 + e]);
                mx4[q] = fmaxf(ptx::max3(a[0], a[1], a[2]), a[3]);
              }
            }
          }
          const float mx = fmaxf(ptx::max3(mx4[0], mx4[1], mx4[2]), mx4[3]);
          const float mt = mx * sl2;  // in log2 units; -inf stays -inf
          float m_new = m;
          if (first) {
            m_new = mt;
            l = fix = 0.f;
          } else if (mt > m + kRescaleSlack) {
            m_new = mt;
            resc = true;
          }
          alpha = resc ? ptx::ex2_approx(m - m_new) : 1.0f;
          m = m_new;
          const float mref = (m == -INFINITY) ? 0.f : m;

          // p = 2^(s*scale*log2e - m) (masked -inf -> 0), row sum, P to tensor memory as bf16.
          const float2 sc2 = make_float2(sl2, sl2);
          const float2 neg = make_float2(-mref, -mref);
          float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                           make_float2(0.f, 0.f)};
          // Packed P word e overwrites register e, whose score was already consumed.
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (!decltype(edge)::value || ((live >> q) & 1u)) {
#pragma unroll
              for (int e = 16 * q; e < 16 * q + 16; ++e) {
                float2 x2 = ptx::fma2(make_float2(s[2 * e], s[2 * e + 1]), sc2, neg);
                x2.x = ptx::ex2_approx(x2.x);
                x2.y = ptx::ex2_approx(x2.y);
                acc[e & 3] = ptx::add2(acc[e & 3], x2);
                raw[e] = ptx::pack_bf16x2(x2.x, x2.y);
              }
            } else {
#pragma unroll
              for (int e = 16 * q; e < 16 * q + 16; ++e) raw[e] = 0u;
            }
          }
          ptx::tmem_st64(tS + kColP, *reinterpret_cast<const uint32_t(*)[64]>(raw));
          const float2 a01 = ptx::add2(acc[0], acc[1]);
          const float2 a23 = ptx::add2(acc[2], acc[3]);
          const float2 a = ptx::add2(a01, a23);
          part_sum = a.x + a.y;
          // The PV product weighs each key by its bf16-rounded p while l sums the fp32 p.
          // `fix` holds the rounding of every tile's largest p: O is divided by l + fix, so
          // that when one key dominates a row its rounding cancels; the LSE is that of l.
          const float p_top = ptx::ex2_approx(ptx::fma2(make_float2(mx, mx), sc2, neg).x);
          const float p_top_bf = __uint_as_float(ptx::pack_bf16x2(p_top, 0.f) << 16);
          top_fix = p_top_bf - p_top;
        };
        if (__all_sync(0xffffffffu, full)) weights(std::false_type());
        else weights(std::true_type());
        if (!first && __any_sync(0xffffffffu, resc)) {
          // O and l were accumulated against the old max: bring them to the new one
          // (after the scores are consumed, so their registers are free).
#pragma unroll 1
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t v[32];
            __syncwarp();
            ptx::tmem_ld32(tO + cc * 32, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
            ptx::tmem_st32(tO + cc * 32, v);
          }
          l *= alpha;
          fix *= alpha;
        }
        l += part_sum;
        fix += top_fix;
        first = false;
        ptx::tc_fence_before();
        ptx::mbar_arrive(c.bar(kPFull + g));

        if (last) {
          ok = wait_bar(c, c.bar(kOFull + g), oj & 1u, kStatusTimeoutSoftmax);
          ++oj;
          if (!__all_sync(0xffffffffu, ok)) return;
          ptx::tc_fence_after();
          store_segment<kPartials>(P, tO, stage, m, l, fix, valid, out_row, rg.step - P.step_lo, lane);
          ptx::tc_fence_before();
          next_part = rg.step + 1;
          m = -INFINITY;
          l = fix = 0.f;
          first = true;
        }
        __syncwarp();
      }
    }
    if (kPartials)
      for (; next_part < P.step_hi; ++next_part) store_empty(P, valid, out_row, next_part - P.step_lo);
    release_record(c, u, lane);
  }
}

template <bool kPartials>
__global__ void __launch_bounds__(kThreads, 1)
    win_fwd_bf16_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, const WinParams P) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Ctl c{sbase + kOffBar, reinterpret_cast<volatile uint32_t*>(sgen + kOffAbort), P.status};
  Record* recs = reinterpret_cast<Record*>(sgen + kOffRec);

  // The rows that shorter boxes never fill meet weights of zero: they have to be finite.
  if (P.k.tile < kTileRows) {
    for (uint32_t at = threadIdx.x * 16; at < kStages * kTileBytes; at += kThreads * 16)
      ptx::st_shared_v4(sbase + kOffKV + at, 0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kItemSlots; ++s) {
      ptx::mbar_init(c.bar(kItemFull + s), 1);
      ptx::mbar_init(c.bar(kItemEmpty + s), kItemConsumers);
    }
    for (int g = 0; g < 2; ++g) {
      ptx::mbar_init(c.bar(kQFull + g), 1);
      ptx::mbar_init(c.bar(kQEmpty + g), 1);
      ptx::mbar_init(c.bar(kSFull + g), 1);
      ptx::mbar_init(c.bar(kPFull + g), 128);
      ptx::mbar_init(c.bar(kOFull + g), 1);
    }
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(c.bar(kKVFull + s), 1);
      ptx::mbar_init(c.bar(kKVEmpty + s), 1);
    }
    ptx::mbar_init(c.bar(kDone), 1);
    *c.abort = 0u;
    ptx::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::tma_prefetch_desc(&tq);
    ptx::tma_prefetch_desc(&tk);
    ptx::tma_prefetch_desc(&tv);
  }
  if (warp == 1) {
    ptx::tmem_alloc(sbase + kOffSlot, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sgen + kOffSlot);

  ProducerState ps{0u, {0u, 0u}};
  if (warp < 4) {
    ptx::regs_release<kRegsOther>();
    if (warp == 0) {
      run_producer(P, c, sbase, recs, &tq, &tk, &tv, ps, lane);  // whole warp; one elected lane issues
      __syncwarp();
    } else if (warp == 1) {
      run_mma<kPartials>(P, c, sbase, recs, tmem, lane);
      // Every MMA this warp issued must retire before TMEM is freed.
      ptx::mma_commit_warp(c.bar(kDone));
      drain_bar(c, c.bar(kDone), 0);
      __syncwarp();
    } else if (warp == 2) {
      run_records(P, c, recs, lane);
    } else if (kPartials) {
      run_empty(P, lane);
    }
  } else {
    ptx::regs_acquire<kRegsSoftmax>();
    run_softmax<kPartials>(P, c, sgen + kOffOut + (warp - 4) * 32 * kStageRow, recs, tmem, (warp - 4) >> 2, warp & 3, lane);
  }

  if (warp == 0 && lane == 0 && *c.abort) {  // (every lane of warp 0 holds the same counts)
    // Let this CTA's own TMA loads land before its shared memory goes away.
    for (uint32_t s = 0; s < (uint32_t)kStages; ++s) {
      if (ps.kv_issued > s) {
        const uint32_t uses = (ps.kv_issued - 1 - s) / kStages + 1;  // loads issued to slot s
        drain_bar(c, c.bar(kKVFull + (int)s), (uses - 1) & 1u);
      }
    }
    for (int g = 0; g < 2; ++g)
      if (ps.q_issued[g] > 0) drain_bar(c, c.bar(kQFull + g), (ps.q_issued[g] - 1) & 1u);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encoder() {
  static EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// [heads, S, 128] bf16 rows as (element, row of a stripe, stripe, head), boxes of 64 elements
// x the tile's rows, 128-byte swizzle.  Rows past the end of a head read as zeros.
bool encode_view(CUtensorMap* map, const void* base, const WinView& view, int64_t seq, int64_t heads) {
  EncodeTiledFn enc = get_encoder();
  if (!enc) return false;
  const uint64_t per = (uint64_t)(seq / view.stripe);
  const cuuint64_t dims[4] = {128, (cuuint64_t)view.stripe, per, (cuuint64_t)heads};
  const cuuint64_t strides[3] = {view.stripe == 1 ? 256 : per * 256, 256, (uint64_t)seq * 256};
  const cuuint32_t box[4] = {64, (cuuint32_t)view.stripe, (cuuint32_t)(view.tile / view.stripe), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kPartials>
cudaError_t launch_kernel(const WinParams& prm, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          int grid, cudaStream_t stream, const char** why) {
  static std::atomic<int> ready[kMaxDevices];
  cudaError_t e = prepare_once(win_fwd_bf16_kernel<kPartials>, ready, kThreads, 128 * kRegsOther + 256 * kRegsSoftmax,
                               (int)kSmemBytes, why);
  if (e != cudaSuccess) return e;
  win_fwd_bf16_kernel<kPartials><<<grid, kThreads, kSmemBytes, stream>>>(tq, tk, tv, prm);
  e = cudaGetLastError();
  if (e != cudaSuccess) *why = "windowed tensor-core forward launch failed";
  return e;
}

}  // namespace

cudaError_t launch_win_fwd_bf16(const WinParams& prm, const void* q, const void* k, const void* v, int grid,
                                cudaStream_t stream, const char** why) {
  CUtensorMap tq, tk, tv;
  const int64_t hq = (int64_t)prm.batch * prm.heads_q, hk = (int64_t)prm.batch * prm.heads_kv;
  if (!encode_view(&tq, q, prm.q, prm.seq, hq) || !encode_view(&tk, k, prm.k, prm.seq, hk) ||
      !encode_view(&tv, v, prm.k, prm.seq, hk)) {
    *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  return prm.o_parts != nullptr ? launch_kernel<true>(prm, tq, tk, tv, grid, stream, why)
                                : launch_kernel<false>(prm, tq, tk, tv, grid, stream, why);
}

}  // namespace ra
