// Windowed attention backward, bf16, d = 128, on the sm_100-family tensor cores.
//
// With the forward's LSE the probabilities of the visible pairs (j <= i and
// (j > i - window or j < sinks)) are recomputed tile by tile,
//   P = 2^(scale*log2(e) * q.k - LSE*log2(e)),   dP = dO V^T,
//   dS = P * (dP - D)   with D = rowsum(dO * O),
//   dV = P^T dO,   dK = scale * dS^T Q,   dQ = scale * dS K,
// a key/value head's dK and dV gathered over the query heads of its group.  Two passes of
// one kernel template, as in the causal backward (bwd_bf16_sm103.cu):
//   pass 0 (dK, dV): an item is one key tile; it meets the query tiles that see one of its
//     keys, every query head of the group in turn;
//   pass 1 (dQ): an item is one query tile; it meets the key tiles that one of its queries
//     sees.
// The planner lists the rows an item meets as ranges (win_internal.h), in the order of
// positions where the layout allows it.  A key tile that holds a sink is met by every later
// query of the sequence, up to hundreds of times what the other tiles meet, and would end
// the launch alone: its far queries (past the window's reach) are cut into pieces the size
// of an ordinary item, which leave their sums in fp32 for a last kernel to add in order.
// (8k tokens, window 512, 4 sinks: 552 us with the tile as one item.)  Where there are few
// tiles in all, the others' queries are cut in the same way.
//
// How (one persistent CTA per SM, 12 warps):
//   warp 0     TMA producer: pass 0's own tiles (K, V) once per item, then 64-row tiles of
//              the streamed tensors (Q, dO and the tile's 64 LSE*log2(e) and D values in
//              pass 0; K, V in pass 1) into a ring of stages.
//   warp 1     tcgen05 issuer (converged warp, one elected lane): per streamed tile two
//              products (M = 128, N = 64) give the scores and dP -- SS in pass 0 (keys are
//              the TMEM lanes), TS in pass 1 with Q and dO read from tensor memory -- then
//              TS products (M = 128, N = 128, K = 64) add P^T dO and dS^T Q (pass 0) or
//              dS K (pass 1), reading P and dS from tensor memory and the streamed tile,
//              still in shared memory, as an MN-major operand.
//   warp 2     the items' records, a few items ahead of the others.
//   warps 4-7 / 8-11  elementwise: one thread per TMEM lane turns scores and dP into P and
//              dS (bf16, written back into tensor memory), for the even / odd streamed
//              tiles; in pass 1 they first store the item's Q (warps 4-7) and dO (8-11)
//              rows into tensor memory; at the end of an item they write the accumulators
//              (pass 0: warps 4-7 dV, 8-11 dK; pass 1: half of dQ each).
// TMEM: two tile buffers of 128 columns (scores 0-63, dP 64-127; P over 0-31 and dS over
// 64-95 once computed), so the next tile's products run while the elementwise warps work on
// the previous one; pass 0 keeps dV at 256 and dK at 384, pass 1 dQ at 256, Q at 384 and dO
// at 448.
// Every wait is bounded (~1 s); on expiry the CTA records it in the status word, drains its
// own copies and MMAs, frees TMEM and returns.
//
// Measured: 32768 tokens in 8 zigzag shards, 32 query and 8 key/value heads, window 4096, 4
// sinks: 5.46 ms (pass 0 3.10, pass 1 2.23, preparation 0.08), 945 TFLOP/s of the formula's 10 d
// a visible pair, 1355 of the 14 d executed (0.70 of the measured rate).  What bounds it: pass 0's
// products with N = 64 read the 128-row own tile from shared memory for every streamed tile;
// pass 1's chain of score product, elementwise step and dQ product is exposed (tensor cores 53%
// and 45% busy).  900 tokens of 4 heads: 21 us in three launches, the passes side by side.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "sm100_ptx.cuh"
#include "win_internal.h"

namespace ra {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kRegsLaunch = 168;
constexpr uint32_t kRegsOther = 120;
constexpr uint32_t kRegsCompute = 192;
static_assert(128 * kRegsOther + 256 * kRegsCompute <= kThreads * kRegsLaunch, "register split");

constexpr int kStreamRows = 64;                   // rows of a streamed tile, at most
constexpr uint32_t kFixBytes = 128 * 128 * 2;     // one 128 x 128 bf16 tile
constexpr uint32_t kFixHalf = 128 * 64 * 2;       // its 128-byte swizzle column
constexpr uint32_t kStrBytes = 64 * 128 * 2;      // one 64 x 128 bf16 tile
constexpr uint32_t kStrHalf = 64 * 64 * 2;
constexpr uint32_t kLseBytes = 128 * 4;           // 64 lse2 values, then 64 D values
constexpr int kItemSlots = 4;                     // records under way
constexpr int kSlotRanges = 12;                   // ranges of an item kept with it
constexpr uint32_t kItemConsumers = 10;           // producer, MMA and 8 elementwise warps
constexpr uint32_t kStageRow = 80;                // 64 bytes of an output row, and 16 against bank conflicts

struct alignas(16) Record {
  WinBwdItem it;
  WinBwdRange ranges[kSlotRanges];
};

template <int kPass>
struct Cfg {
  static constexpr int kStages = kPass == 0 ? 3 : 5;
  static constexpr int kBufs = 2;  // score/dP buffers in tensor memory
  static constexpr uint32_t kStageBytes = kPass == 0 ? 2 * kStrBytes + 1024 : 2 * kStrBytes;
  static constexpr uint32_t kOffFix = 0;  // pass 0 only: K, V (pass 1 keeps Q, dO in tensor memory)
  static constexpr uint32_t kOffStage = kPass == 0 ? 2 * kFixBytes : 0;
  static constexpr uint32_t kOffOut = kOffStage + kStages * kStageBytes;  // output rows on their way out
  static constexpr uint32_t kOffRec = kOffOut + 256 * kStageRow;
  static constexpr uint32_t kOffBar = kOffRec + kItemSlots * (uint32_t)sizeof(Record);
  static constexpr uint32_t kSmemBytes = kOffBar + 512 + 1024;  // barriers + slots, 1 KiB alignment slack
};

enum : int {
  kFixFull = 0,
  kFixEmpty = 1,
  kAccFull = 2,
  kAccEmpty = 3,
  kDone = 4,
  kSFull = 5,       // 2 (one per buffer)
  kPFull = 7,       // 2
  kItemFull = 9,    // kItemSlots
  kItemEmpty = kItemFull + kItemSlots,
  kStFull = kItemEmpty + kItemSlots,  // kStages
};
template <int kPass>
struct Bars {
  static constexpr int kStEmpty = kStFull + Cfg<kPass>::kStages;
  static constexpr int kNum = kStEmpty + Cfg<kPass>::kStages;
};

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColAcc0 = 256, kColAcc1 = 384;  // dV (or dQ), dK
constexpr uint32_t kColQ = 384, kColDO = 448;       // pass 1
__device__ __forceinline__ uint32_t col_buf(uint32_t b) { return b * 128u; }
constexpr uint32_t kColDP = 64;   // dP within a buffer; dS is written over its first 32 columns
constexpr uint32_t kIdescSS = ptx::idesc_bf16_f32(128, 64, false, false);
constexpr uint32_t kIdescTS = ptx::idesc_bf16_f32(128, 128, false, true);
constexpr uint64_t kWaitBudgetNs = 1000000000ull;
constexpr uint32_t kSuspendHintNs = 2000u;

struct Ctl {
  uint32_t bars;
  volatile uint32_t* abort;
  uint32_t* status;
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * (uint32_t)i; }
};

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
__device__ void run_records(const WinBwdParams& P, const Ctl& c, Record* recs, int lane, uint32_t first, uint32_t stride) {
  constexpr int kWords = sizeof(WinBwdItem) / 16;
  for (uint32_t u = 0;; ++u) {
    const int idx = (int)(first + u * stride);
    const uint32_t slot = u % kItemSlots;
    if (!RA_WAIT(kItemEmpty + (int)slot, (u / kItemSlots) ^ 1u, kStatusTimeoutProducer)) return;
    Record& r = recs[slot];
    const bool end = idx >= P.n_items;
    if (end) {
      if (lane == 0) r.it.bh = -1;
    } else {
      const int4 w = lane < kWords ? reinterpret_cast<const int4*>(P.items + idx)[lane] : make_int4(0, 0, 0, 0);
      if (lane < kWords) reinterpret_cast<int4*>(&r.it)[lane] = w;
      const int x0 = __shfl_sync(0xffffffffu, w.x, 1), xn = __shfl_sync(0xffffffffu, w.y, 1);  // range0, n_ranges
      if (lane < kSlotRanges && lane < xn)
        *reinterpret_cast<int4*>(&r.ranges[lane]) = *reinterpret_cast<const int4*>(&P.ranges[x0 + lane]);
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(c.bar(kItemFull + (int)slot));
    if (end) return;
  }
}
__device__ __forceinline__ const Record* next_record(const Ctl& c, const Record* recs, uint32_t u, uint32_t who) {
  const uint32_t slot = u % kItemSlots;
  if (!RA_WAIT(kItemFull + (int)slot, u / kItemSlots, who)) return nullptr;
  return recs[slot].it.bh < 0 ? nullptr : recs + slot;
}
__device__ __forceinline__ void release_record(const Ctl& c, uint32_t u, int lane) {
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(c.bar(kItemEmpty + (int)(u % kItemSlots)));
}
__device__ __forceinline__ WinBwdRange range_at(const WinBwdParams& P, const Record* r, int k) {
  return k < kSlotRanges ? r->ranges[k] : P.ranges[r->it.range0 + k];
}

// ---------------------------------------------------------------- producer --
struct ProducerState {
  uint32_t str_issued;  // streamed tiles issued
  uint32_t fix_issued;  // items whose own tiles were issued
};

// (head, range, tile) in order: the streamed tiles of an item, for each of its heads.
template <int kPass>
__device__ void run_producer(const WinBwdParams& P, const Ctl& c, uint32_t sbase, const Record* recs,
                             const CUtensorMap* tx0, const CUtensorMap* tx1, const CUtensorMap* ty0,
                             const CUtensorMap* ty1, ProducerState& st, int lane) {
  using C = Cfg<kPass>;
  const uint64_t keep = ptx::l2_policy_evict_last();
  const uint32_t str_bytes = (uint32_t)P.str.tile * 256u, fix_bytes = (uint32_t)P.own.tile * 256u;
  uint32_t s_it = 0;
  for (uint32_t u = 0;; ++u) {
    const Record* r = next_record(c, recs, u, kStatusTimeoutProducer);
    if (r == nullptr) return;
    const WinBwdItem it = r->it;
    RA_BOUNDS(c.status, it.shard >= 0 && it.shard < P.own.shards && it.row0 >= 0 && it.row0 < P.own.s_n, 81);
    if (kPass == 0) {
      if (!RA_WAIT(kFixEmpty, u ^ 1u, kStatusTimeoutProducer)) return;
      const int32_t i = (it.shard * P.own.s_n + it.row0) / P.own.stripe;
      RA_BOUNDS(c.status, i >= 0 && i < P.seq / P.own.stripe && it.bh < P.batch * P.heads_kv, 82);
      ptx::mbar_arrive_expect_tx_warp(c.bar(kFixFull), 2 * fix_bytes);
      tma_load_4d_warp_hint(sbase + C::kOffFix, tx0, c.bar(kFixFull), 0, i, it.bh, keep);
      tma_load_4d_warp_hint(sbase + C::kOffFix + kFixHalf, tx0, c.bar(kFixFull), 64, i, it.bh, keep);
      tma_load_4d_warp_hint(sbase + C::kOffFix + kFixBytes, tx1, c.bar(kFixFull), 0, i, it.bh, keep);
      tma_load_4d_warp_hint(sbase + C::kOffFix + kFixBytes + kFixHalf, tx1, c.bar(kFixFull), 64, i, it.bh, keep);
      st.fix_issued = u + 1;
    }
    for (int g = it.g0; g < it.g1; ++g) {
      // bh of the streamed rows: pass 0 (bh = b * Hkv + kv head) query head g of the group,
      // pass 1 (bh = b * Hq + h) the key/value head
      const int32_t bh = kPass == 0 ? it.bh / P.heads_kv * P.heads_q + it.bh % P.heads_kv * P.group + g
                                    : it.bh / P.heads_q * P.heads_kv + it.bh % P.heads_q / P.group;
      for (int k = 0; k < it.n_ranges; ++k) {
        const WinBwdRange rg = range_at(P, r, k);
        RA_BOUNDS(c.status, rg.r >= 0 && rg.r < P.str.shards && rg.row0 >= 0 && rg.row0 % P.str.tile == 0 &&
                                rg.row0 < rg.end && rg.end <= P.str.s_n, 83);
        int32_t i = (rg.r * P.str.s_n + rg.row0) / P.str.stripe;
        int64_t lse_at = win_scalar_block(P, bh, rg.r, rg.row0 / P.str.tile) * 128;
        for (int n = range_tiles64(rg, P.str.tile); n > 0; --n, i += P.str.tile / P.str.stripe, lse_at += 128) {
          RA_BOUNDS(c.status, i >= 0 && i < P.seq / P.str.stripe && lse_at >= 0 &&
                                  (kPass == 1 || lse_at + 128 <= P.n_scalars), 84);
          const uint32_t s = s_it % C::kStages;
          if (!RA_WAIT(kStFull + C::kStages + (int)s, (s_it / C::kStages) ^ 1u, kStatusTimeoutProducer)) return;
          const uint32_t dst = sbase + C::kOffStage + s * C::kStageBytes;
          ptx::mbar_arrive_expect_tx_warp(c.bar(kStFull + (int)s), 2 * str_bytes + (kPass == 0 ? kLseBytes : 0u));
          tma_load_4d_warp_hint(dst, ty0, c.bar(kStFull + (int)s), 0, i, bh, keep);
          tma_load_4d_warp_hint(dst + kStrHalf, ty0, c.bar(kStFull + (int)s), 64, i, bh, keep);
          tma_load_4d_warp_hint(dst + kStrBytes, ty1, c.bar(kStFull + (int)s), 0, i, bh, keep);
          tma_load_4d_warp_hint(dst + kStrBytes + kStrHalf, ty1, c.bar(kStFull + (int)s), 64, i, bh, keep);
          if (kPass == 0)  // the tile's 64 lse2 and 64 D values (one 512-byte block)
            ptx::bulk_load_warp(dst + 2 * kStrBytes, P.lse2d + lse_at, kLseBytes, c.bar(kStFull + (int)s));
          st.str_issued = ++s_it;
        }
      }
    }
    release_record(c, u, lane);
  }
}

// --------------------------------------------------------------------- MMA --
template <int kPass>
__device__ __forceinline__ void issue_ss(uint32_t tmem, int buf, uint32_t fix_lo, uint32_t str_lo) {
  // Scores: own tile 0 x streamed tile 0; dP: own tile 1 x streamed tile 1.  Pass 0's
  // own tiles (K, V) are in shared memory; pass 1's (Q, dO) in tensor memory, two bf16
  // of d per column, so its products read only the streamed 64-row tile from shared
  // memory.
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const uint32_t a0 = fix_lo + (which ? (kFixBytes >> 4) : 0u);
    const uint32_t b0 = str_lo + (which ? (kStrBytes >> 4) : 0u);
    const uint32_t d = tmem + col_buf(buf) + (which ? kColDP : 0u);
#pragma unroll
    for (uint32_t kk = 0; kk < 8; ++kk) {  // 8 steps of K = 16 over d = 128
      const uint32_t ob = ((kk >> 2) * kStrHalf + (kk & 3u) * 32u) >> 4;
      if (kPass == 0) {
        const uint32_t oa = ((kk >> 2) * kFixHalf + (kk & 3u) * 32u) >> 4;
        ptx::mma_bf16_ss_lo_warp(d, a0 + oa, b0 + ob, kIdescSS, kk > 0 ? 1u : 0u);
      } else {
        ptx::mma_bf16_ts_lo_warp(d, tmem + (which ? kColDO : kColQ) + kk * 8u, b0 + ob, kIdescSS, kk > 0 ? 1u : 0u);
      }
    }
  }
}

// acc += A[tmem, 64 K-columns as 32 words] * B[streamed 64-row tile, MN-major].
__device__ __forceinline__ void issue_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, bool accumulate) {
#pragma unroll
  for (uint32_t kk = 0; kk < 4; ++kk)  // 4 steps of 16 rows = 8 TMEM columns of A
    ptx::mma_bf16_ts_lo_warp(d, a_tmem + kk * 8u, b_lo + ((kk * 2048u) >> 4), kIdescTS,
                             (accumulate || kk > 0) ? 1u : 0u);
}

template <int kPass>
__device__ void run_mma(const WinBwdParams& P, const Ctl& c, uint32_t sbase, const Record* recs, uint32_t tmem, int lane) {
  using C = Cfg<kPass>;
  constexpr uint32_t NB = (uint32_t)C::kBufs;
  const uint32_t fix_lo = ptx::desc_lo(sbase + C::kOffFix, 16);
  // two 128-column buffers, then the accumulators (and pass 1's Q, dO) up to column 512
  RA_BOUNDS(c.status, tmem == 0u && col_buf(C::kBufs) <= kColAcc0 && kColDO + 64u <= kTmemCols, 85);
  uint32_t s_it = 0;  // streamed tiles so far (global tile index J of this CTA)
  auto str_lo = [&](uint32_t J, uint32_t lbo) {
    return ptx::desc_lo(sbase + C::kOffStage + (J % C::kStages) * C::kStageBytes, lbo);
  };
  // Scores and dP of tile J into buffer J % NB.
  auto issue_tile_ss = [&](uint32_t J) {
    if (!RA_WAIT(kStFull + (int)(J % C::kStages), J / C::kStages, kStatusTimeoutMma)) return false;
    issue_ss<kPass>(tmem, (int)(J % NB), fix_lo, str_lo(J, 16));
    ptx::mma_commit_warp(c.bar(kSFull + (int)(J % NB)));
    return true;
  };
  for (uint32_t u = 0;; ++u) {
    const Record* r = next_record(c, recs, u, kStatusTimeoutMma);
    if (r == nullptr) break;
    const uint32_t n = (uint32_t)r->it.n_tiles;  // at least one
    release_record(c, u, lane);
    if (!RA_WAIT(kFixFull, u, kStatusTimeoutMma)) return;
    ptx::tc_fence_after();  // pass 1: Q and dO were stored into tensor memory by other warps
    // Run NB - 1 tiles ahead: buffer (J + NB - 1) % NB was last used by tile J - 1,
    // whose TS products are issued (the tensor pipe executes in issue order).
    for (uint32_t a = 0; a + 1 < NB && a < n; ++a)
      if (!issue_tile_ss(s_it + a)) return;
    for (uint32_t i = 0; i < n; ++i) {
      const uint32_t J = s_it + i;
      if (i + NB - 1 < n && !issue_tile_ss(J + NB - 1)) return;
      if (!RA_WAIT(kPFull + (int)(J % NB), J / NB, kStatusTimeoutMma)) return;
      if (i == 0 && u > 0 && !RA_WAIT(kAccEmpty, u - 1, kStatusTimeoutMma)) return;
      ptx::tc_fence_after();
      // Streamed tile 0 (Q in pass 0, K in pass 1) and tile 1 (dO in pass 0) as MN-major B.
      const uint32_t y0 = str_lo(J, kStrHalf), y1 = y0 + (kStrBytes >> 4);
      const uint32_t buf = tmem + col_buf(J % NB);
      if (kPass == 0) {
        issue_ts(tmem + kColAcc0, buf, y1, i > 0);           // dV += P^T dO
        issue_ts(tmem + kColAcc1, buf + kColDP, y0, i > 0);  // dK += dS^T Q
      } else {
        issue_ts(tmem + kColAcc0, buf + kColDP, y0, i > 0);  // dQ += dS K
      }
      ptx::mma_commit_warp(c.bar(kStFull + C::kStages + (int)(J % C::kStages)));
    }
    ptx::mma_commit_warp(c.bar(kAccFull));
    ptx::mma_commit_warp(c.bar(kFixEmpty));
    s_it += n;
  }
}

// -------------------------------------------------------------- elementwise --
// Write 64 accumulator columns [col0, col0 + 64) of the warp's 32 rows, times mul, as bf16:
// through shared memory, 32 columns at a time, so that 4 lanes write 64 consecutive bytes.
// to: this lane's row of dst, or -1.
__device__ __forceinline__ void store_rows(uint32_t t_acc, uint8_t* stage, void* dst, int to, int col0, float mul,
                                           int lane) {
#pragma unroll 1
  for (int cc = 0; cc < 2; ++cc) {
    uint32_t v[32];
    __syncwarp();
    ptx::tmem_ld32(t_acc + (uint32_t)(col0 + cc * 32), v);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = ptx::pack_bf16x2(__uint_as_float(v[8 * q + 2 * e]) * mul, __uint_as_float(v[8 * q + 2 * e + 1]) * mul);
      *reinterpret_cast<uint4*>(stage + lane * kStageRow + q * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // rows 8q .. 8q + 7
      const int r = 8 * q + (lane >> 2);
      const uint4 x = *reinterpret_cast<const uint4*>(stage + r * kStageRow + (lane & 3) * 16);
      const int row = __shfl_sync(0xffffffffu, to, r);
      if (row >= 0) reinterpret_cast<uint4*>(dst)[(int64_t)row * 16 + (col0 + cc * 32) / 8 + (lane & 3)] = x;
    }
  }
}

// The 128 accumulator columns of this lane's row, times mul, as fp32 partial sums.
__device__ __forceinline__ void store_part(uint32_t t_acc, float* dst, float mul, bool valid) {
#pragma unroll 1
  for (int cc = 0; cc < 4; ++cc) {
    uint32_t v[32];
    __syncwarp();
    ptx::tmem_ld32(t_acc + (uint32_t)(cc * 32), v);
    if (!valid) continue;
    float4* d = reinterpret_cast<float4*>(dst + cc * 32);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      d[q] = make_float4(__uint_as_float(v[4 * q]) * mul, __uint_as_float(v[4 * q + 1]) * mul,
                         __uint_as_float(v[4 * q + 2]) * mul, __uint_as_float(v[4 * q + 3]) * mul);
  }
}

// The lowest n bits (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : ~(~0u << n)); }

// P and dS for one pair of columns (live: both unmasked).
__device__ __forceinline__ void p_ds_pair(float2 s2, float2 dp2, float2 l2, float2 d2, float2 sl2, bool live0,
                                          bool live1, uint32_t& pw, uint32_t& dw) {
  float2 x = ptx::fma2(s2, sl2, make_float2(-l2.x, -l2.y));
  x.x = live0 ? ptx::ex2_approx(x.x) : 0.f;
  x.y = live1 ? ptx::ex2_approx(x.y) : 0.f;
  const float2 ds = ptx::mul2(x, ptx::add2(dp2, make_float2(-d2.x, -d2.y)));
  pw = ptx::pack_bf16x2(x.x, x.y);
  dw = ptx::pack_bf16x2(ds.x, ds.y);
}

template <int kPass>
__device__ void run_elementwise(const WinBwdParams& P, const Ctl& c, uint8_t* sgen, const Record* recs, uint32_t tmem,
                                int g, int wq, int lane) {
  using C = Cfg<kPass>;
  constexpr uint32_t NB = (uint32_t)C::kBufs;
  const int row = wq * 32 + lane;  // TMEM lane: key row (pass 0) or query row (pass 1)
  const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
  uint8_t* stage = sgen + C::kOffOut + (g * 4 + wq) * 32 * kStageRow;
  const float2 sl2 = make_float2(P.scale_log2, P.scale_log2);
  uint32_t s_it = 0;
  for (uint32_t u = 0;; ++u) {
    const Record* rec = next_record(c, recs, u, kStatusTimeoutSoftmax);
    if (rec == nullptr) return;
    const WinBwdItem it = rec->it;
    const int i_own = it.row0 + row;  // local row of the item's own tile
    const bool valid = i_own < it.row_end && row < P.own.tile;
    const int my_pos = it.pos0 + row * P.own.apart;  // (of rows that are not valid: any)
    const int head_row = it.shard * P.own.s_n + i_own;
    const int64_t out_row = (int64_t)it.bh * P.seq +
                            (P.own.stripe == 1 ? head_row
                                               : head_row % P.own.stripe * (P.seq / P.own.stripe) + head_row / P.own.stripe);
    RA_BOUNDS(c.status,
              !valid || (out_row >= 0 && out_row < (int64_t)P.batch * (kPass == 0 ? P.heads_kv : P.heads_q) * P.seq), 87);
    RA_BOUNDS(c.status, wq >= 0 && wq < 4 && (lane_off >> 16) + 32u <= 128u, 88);
    float2 own_l = make_float2(0.f, 0.f), own_d = make_float2(0.f, 0.f);  // pass 1: this row's lse2, D
    if (kPass == 1) {
      if (valid) {
        const int64_t li = win_scalar_block(P, it.bh, it.shard, i_own / P.str.tile) * 128 + i_own % P.str.tile;
        RA_BOUNDS(c.status, li >= 0 && li + 64 < P.n_scalars, 89);
        own_l = make_float2(P.lse2d[li], P.lse2d[li]);
        own_d = make_float2(P.lse2d[li + 64], P.lse2d[li + 64]);
      }
      // This row of Q (warps 4-7) or dO (warps 8-11) into tensor memory, once the
      // previous item's products are done with it.
      const bool okq = wait_bar(c, c.bar(kFixEmpty), (u & 1u) ^ 1u, kStatusTimeoutSoftmax);
      if (!__all_sync(0xffffffffu, okq)) return;
      uint32_t words[64];
      const uint4* src = reinterpret_cast<const uint4*>(g ? P.dout : P.q) + (valid ? out_row * 16 : 0);
#pragma unroll
      for (int q4 = 0; q4 < 16; ++q4) {
        const uint4 v4 = valid ? src[q4] : make_uint4(0u, 0u, 0u, 0u);
        words[4 * q4] = v4.x;
        words[4 * q4 + 1] = v4.y;
        words[4 * q4 + 2] = v4.z;
        words[4 * q4 + 3] = v4.w;
      }
      ptx::tmem_st64(tmem + lane_off + (g ? kColDO : kColQ), words);
      ptx::tc_fence_before();
      ptx::mbar_arrive(c.bar(kFixFull));
    }

    uint32_t J = s_it;
    for (int head = it.g0; head < it.g1; ++head)
      for (int k = 0; k < it.n_ranges; ++k) {
        const WinBwdRange rg = range_at(P, rec, k);
        const int n = range_tiles64(rg, P.str.tile);
        const WinBwdColumns own = range_columns<kPass>(P, rg, my_pos);
        for (int kt = 0; kt < n; ++kt, ++J) {
          if ((int)(J & 1u) != g) continue;
          // Columns [c_lo, c_hi) and [c_f, c_s) of this tile are live for this row.
          const int y = kt * P.str.tile;
          const int c_hi = own.hi - y < P.str.tile ? own.hi - y : P.str.tile, c_lo = own.lo - y;
          const int c_s = own.sk - y < c_hi ? own.sk - y : c_hi, c_f = own.from - y;
          const bool ok = wait_bar(c, c.bar(kSFull + (int)(J % NB)), (J / NB) & 1u, kStatusTimeoutSoftmax);
          if (!__all_sync(0xffffffffu, ok)) return;
          ptx::tc_fence_after();
          const uint32_t tb = tmem + lane_off + col_buf(J % NB);
          // pass 0: the tile's 64 lse2 values, then its 64 D values, in shared memory
          const float4* l4 =
              reinterpret_cast<const float4*>(sgen + C::kOffStage + (J % C::kStages) * C::kStageBytes + 2 * kStrBytes);
          uint32_t pw[32], dw[32];
          auto weights = [&](auto edge) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // columns 32*half .. 32*half + 31
              uint32_t raw[64];                       // scores in 0-31, dP in 32-63
              ptx::tmem_ld32x2(tb + 32u * half, tb + kColDP + 32u * half, raw);
              uint32_t bits = ~0u;
              if (decltype(edge)::value)
                bits = (below(c_hi - 32 * half) & ~below(c_lo - 32 * half)) | (below(c_s - 32 * half) & ~below(c_f - 32 * half));
#pragma unroll
              for (int q = 0; q < 8; ++q) {  // columns c0 .. c0+3 of the tile
                const int c0 = 32 * half + 4 * q;
                float4 L, D;
                if (kPass == 0) {
                  L = l4[c0 / 4];
                  D = l4[16 + c0 / 4];
                } else {
                  L = make_float4(own_l.x, own_l.x, own_l.x, own_l.x);
                  D = make_float4(own_d.x, own_d.x, own_d.x, own_d.x);
                }
                auto live = [&](int e) { return !decltype(edge)::value || ((bits >> (4 * q + e)) & 1u); };
                const int r0 = 4 * q;
                p_ds_pair(make_float2(__uint_as_float(raw[r0]), __uint_as_float(raw[r0 + 1])),
                          make_float2(__uint_as_float(raw[32 + r0]), __uint_as_float(raw[32 + r0 + 1])),
                          make_float2(L.x, L.y), make_float2(D.x, D.y), sl2, live(0), live(1), pw[c0 / 2], dw[c0 / 2]);
                p_ds_pair(make_float2(__uint_as_float(raw[r0 + 2]), __uint_as_float(raw[r0 + 3])),
                          make_float2(__uint_as_float(raw[32 + r0 + 2]), __uint_as_float(raw[32 + r0 + 3])),
                          make_float2(L.z, L.w), make_float2(D.z, D.w), sl2, live(2), live(3), pw[c0 / 2 + 1],
                          dw[c0 / 2 + 1]);
              }
            }
          };
          const bool full = c_hi >= kStreamRows && (c_lo <= 0 || (c_s >= kStreamRows && c_f <= 0));
          if (__all_sync(0xffffffffu, full)) weights(std::false_type());
          else weights(std::true_type());
          if (kPass == 0) ptx::tmem_st32(tb, pw);  // P^T for dV (pass 1 needs only dS)
          ptx::tmem_st32(tb + kColDP, dw);
          ptx::tc_fence_before();
          ptx::mbar_arrive(c.bar(kPFull + (int)(J % NB)));
        }
      }
    RA_BOUNDS(c.status, J == s_it + (uint32_t)it.n_tiles, 86);
    s_it = J;
    release_record(c, u, lane);

    // Item done: write the accumulators (pass 0: dV by warps 4-7, dK by 8-11;
    // pass 1: dQ columns 0-63 by warps 4-7, 64-127 by 8-11).
    const bool ok = wait_bar(c, c.bar(kAccFull), u & 1u, kStatusTimeoutSoftmax);
    if (!__all_sync(0xffffffffu, ok)) return;
    ptx::tc_fence_after();
    const int to = valid ? (int)out_row : -1;  // (rows fit in 31 bits)
    if (kPass == 0) {
      const uint32_t t_acc = tmem + lane_off + (g ? kColAcc1 : kColAcc0);
      const float mul = g ? P.scale : 1.0f;
      if (it.part >= 0) {
        // (a piece of far queries leaves only the sinks' rows)
        const bool mine = valid && row < it.part_rows;
        store_part(t_acc, P.parts + it.part + ((int64_t)g * it.part_rows + (mine ? row : 0)) * 128, mul, mine);
      } else {
        store_rows(t_acc, stage, g ? P.dk : P.dv, to, 0, mul, lane);
        store_rows(t_acc, stage, g ? P.dk : P.dv, to, 64, mul, lane);
      }
    } else {
      store_rows(tmem + lane_off + kColAcc0, stage, P.dq, to, g * 64, P.scale, lane);
    }
    ptx::tc_fence_before();
    ptx::mbar_arrive(c.bar(kAccEmpty));
    __syncwarp();
  }
}

// A CTA of one pass, taking items first, first + stride, ...
template <int kPass>
__device__ __forceinline__ void run_pass(const CUtensorMap& tx0, const CUtensorMap& tx1, const CUtensorMap& ty0,
                                         const CUtensorMap& ty1, const WinBwdParams& P, uint32_t first, uint32_t stride) {
  using C = Cfg<kPass>;
  using B = Bars<kPass>;
  static_assert(8 * B::kNum + 8 <= 512 && C::kOffBar % 16 == 0 && C::kSmemBytes <= 232448, "shared memory");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t off_slot = C::kOffBar + 8 * B::kNum;
  Ctl c{sbase + C::kOffBar, reinterpret_cast<volatile uint32_t*>(sgen + off_slot + 4), P.status};
  Record* recs = reinterpret_cast<Record*>(sgen + C::kOffRec);

  // Rows that shorter boxes never fill meet weights of zero: they have to be finite.
  if (P.str.tile < kStreamRows || P.own.tile < 128) {
    for (uint32_t at = threadIdx.x * 16; at < C::kOffOut; at += kThreads * 16)
      ptx::st_shared_v4(sbase + at, 0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
  }

  if (threadIdx.x == 0) {
    ptx::mbar_init(c.bar(kFixFull), kPass == 0 ? 1 : 256);  // TMA (pass 0) or the 256 writers (pass 1)
    ptx::mbar_init(c.bar(kFixEmpty), 1);
    ptx::mbar_init(c.bar(kAccFull), 1);
    ptx::mbar_init(c.bar(kAccEmpty), 256);
    ptx::mbar_init(c.bar(kDone), 1);
    for (int b = 0; b < C::kBufs; ++b) {
      ptx::mbar_init(c.bar(kSFull + b), 1);
      ptx::mbar_init(c.bar(kPFull + b), 128);
    }
    for (int s = 0; s < kItemSlots; ++s) {
      ptx::mbar_init(c.bar(kItemFull + s), 1);
      ptx::mbar_init(c.bar(kItemEmpty + s), kItemConsumers);
    }
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(c.bar(kStFull + s), 1);
      ptx::mbar_init(c.bar(B::kStEmpty + s), 1);
    }
    *c.abort = 0u;
    ptx::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    if (kPass == 0) {
      ptx::tma_prefetch_desc(&tx0);
      ptx::tma_prefetch_desc(&tx1);
    }
    ptx::tma_prefetch_desc(&ty0);
    ptx::tma_prefetch_desc(&ty1);
  }
  if (warp == 1) {
    ptx::tmem_alloc(sbase + off_slot, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sgen + off_slot);

  ProducerState ps{0u, 0u};
  if (warp < 4) {
    ptx::regs_release<kRegsOther>();
    if (warp == 0) {
      run_producer<kPass>(P, c, sbase, recs, &tx0, &tx1, &ty0, &ty1, ps, lane);
      __syncwarp();
    } else if (warp == 1) {
      run_mma<kPass>(P, c, sbase, recs, tmem, lane);
      ptx::mma_commit_warp(c.bar(kDone));
      drain_bar(c, c.bar(kDone), 0);
      __syncwarp();
    } else if (warp == 2) {
      run_records(P, c, recs, lane, first, stride);
    }
  } else {
    ptx::regs_acquire<kRegsCompute>();
    run_elementwise<kPass>(P, c, sgen, recs, tmem, (warp - 4) >> 2, warp & 3, lane);
  }

  if (warp == 0 && lane == 0 && *c.abort) {
    // Let this CTA's own TMA loads land before its shared memory goes away.
    for (uint32_t s = 0; s < (uint32_t)C::kStages; ++s) {
      if (ps.str_issued > s) {
        const uint32_t uses = (ps.str_issued - 1 - s) / C::kStages + 1;
        drain_bar(c, c.bar(kStFull + (int)s), (uses - 1) & 1u);
      }
    }
    if (ps.fix_issued > 0) drain_bar(c, c.bar(kFixFull), (ps.fix_issued - 1) & 1u);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// Maps of a pass: own tiles of K and V (pass 0), streamed tiles of Q and dO (pass 0) or K and
// V (pass 1; its own rows of Q and dO are read without a map).
struct Maps {
  CUtensorMap own_k, own_v, y0, y1;
};

template <int kPass>
__global__ void __launch_bounds__(kThreads, 1)
    win_bwd_bf16_kernel(const __grid_constant__ Maps t, const __grid_constant__ WinBwdParams P) {
  run_pass<kPass>(t.own_k, t.own_v, t.y0, t.y1, P, blockIdx.x, gridDim.x);
}
// Both passes side by side: the first `n0` CTAs take pass 0's items, the others pass 1's.
__global__ void __launch_bounds__(kThreads, 1)
    win_bwd_both_kernel(const __grid_constant__ Maps t0, const __grid_constant__ Maps t1,
                        const __grid_constant__ WinBwdParams P0, const __grid_constant__ WinBwdParams P1, uint32_t n0) {
  if (blockIdx.x < n0) run_pass<0>(t0.own_k, t0.own_v, t0.y0, t0.y1, P0, blockIdx.x, n0);
  else run_pass<1>(t1.own_k, t1.own_v, t1.y0, t1.y1, P1, blockIdx.x - n0, gridDim.x - n0);
}

// -------------------------------------------------------------- preparation --
// lse2 = LSE * log2(e) and D = rowsum(dO * O) of every query row, in blocks of 64: the rows of
// one streamed tile (P.str.tile of them, zeros behind), 64 lse2 values, then 64 D values.  A
// warp takes 4 rows at a time, 8 lanes a row, and reads them in 16-byte loads.
constexpr int kPrepWarps = 8;
__global__ void __launch_bounds__(kPrepWarps * 32)
    win_bwd_prep_kernel(const WinBwdParams P, int64_t blocks, const uint4* __restrict__ o, const uint4* __restrict__ dout,
                        const float* __restrict__ lse, float* __restrict__ out) {
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const int64_t rows4 = blocks * 16;  // groups of 4 rows
  const int per_shard = P.blocks;
  for (int64_t r4 = (int64_t)blockIdx.x * kPrepWarps + (threadIdx.x >> 5); r4 < rows4; r4 += (int64_t)gridDim.x * kPrepWarps) {
    const int64_t blk = r4 >> 4;
    const int col = (int)(r4 & 15) * 4 + (lane >> 3);  // row of the block
    const int64_t bs = blk / per_shard;                // bh * shards + shard
    const int tile = (int)(blk - bs * per_shard);
    const int i = tile * P.str.tile + col;
    float l2 = 0.f, dd = 0.f;
    if (col < P.str.tile && i < P.str.s_n) {
      const int64_t bh = bs / P.str.shards;
      const int head_row = (int)(bs - bh * P.str.shards) * P.str.s_n + i;
      const int64_t row = bh * P.seq + (P.str.stripe == 1 ? head_row
                                                          : head_row % P.str.stripe * (P.seq / P.str.stripe) +
                                                                head_row / P.str.stripe);
      l2 = sub == 0 ? lse[row] * 1.4426950408889634f : 0.f;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint4 a = __ldcs(o + row * 16 + n * 8 + sub), b = __ldcs(dout + row * 16 + n * 8 + sub);
        const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dd = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y[e] << 16), dd);
          dd = fmaf(__uint_as_float(x[e] & 0xffff0000u), __uint_as_float(y[e] & 0xffff0000u), dd);
        }
      }
    }
#pragma unroll
    for (int s = 4; s > 0; s >>= 1) dd += __shfl_xor_sync(0xffffffffu, dd, s);
    if (sub == 0) {
      out[blk * 128 + col] = l2;
      out[blk * 128 + 64 + col] = dd;
    }
  }
}

// Adds the parts of the key tiles that were cut, in order: a CTA takes 8 rows of a tile's dV or
// dK, a warp a row, a lane 4 columns.
constexpr int kJoinRows = 8;
__global__ void __launch_bounds__(kJoinRows * 32) win_bwd_join_kernel(const WinBwdParams P, const WinBwdSplit* __restrict__ splits) {
  const WinBwdSplit sp = splits[blockIdx.x];
  const int row = blockIdx.y * kJoinRows + (threadIdx.x >> 5), which = blockIdx.z, lane = threadIdx.x & 31;
  const int i = sp.row0 + row;
  if (i >= sp.row_end || row >= P.own.tile) return;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int64_t first, int rows, int n) {
    const float4* from = reinterpret_cast<const float4*>(P.parts + first + ((int64_t)which * rows + row) * 128) + lane;
#pragma unroll 8
    for (int x = 0; x < n; ++x) {
      const float4 y = from[(int64_t)x * 2 * rows * 32];
      sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
    }
  };
  add(sp.near, 128, sp.n_near);
  if (row < sp.far_rows) add(sp.far, sp.far_rows, sp.n_far);
  const int head_row = sp.shard * P.own.s_n + i;
  const int64_t out = (int64_t)sp.bh * P.seq + (P.own.stripe == 1 ? head_row
                                                                  : head_row % P.own.stripe * (P.seq / P.own.stripe) +
                                                                        head_row / P.own.stripe);
  reinterpret_cast<uint2*>(which ? P.dk : P.dv)[out * 32 + lane] =
      make_uint2(ptx::pack_bf16x2(sum.x, sum.y), ptx::pack_bf16x2(sum.z, sum.w));
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

// [heads, S, 128] bf16 rows in a view, boxes of 64 elements x `tile` rows (encode_view of the
// forward).  Rows past the end of a head read as zeros.
bool encode_view(CUtensorMap* map, const void* base, const WinView& view, int64_t seq, int64_t heads) {
  EncodeTiledFn enc = get_encoder();
  if (!enc) return false;
  const uint64_t per = (uint64_t)(seq / view.stripe);
  const cuuint64_t dims[4] = {128, (cuuint64_t)view.stripe, per, (cuuint64_t)heads};
  const cuuint64_t strides[3] = {view.stripe == 1 ? 256 : per * 256, 256, (uint64_t)seq * 256};
  const cuuint32_t box[4] = {64, (cuuint32_t)view.stripe, (cuuint32_t)(view.tile / view.stripe), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kPass>
cudaError_t launch_pass(const WinBwdParams& prm, const Maps& maps, int grid, cudaStream_t stream, const char** why) {
  using C = Cfg<kPass>;
  static std::atomic<int> ready[kMaxDevices];
  cudaError_t e = prepare_once(win_bwd_bf16_kernel<kPass>, ready, kThreads, 128 * kRegsOther + 256 * kRegsCompute,
                               (int)C::kSmemBytes, why);
  if (e != cudaSuccess) return e;
  win_bwd_bf16_kernel<kPass><<<grid, kThreads, C::kSmemBytes, stream>>>(maps, prm);
  e = cudaGetLastError();
  if (e != cudaSuccess) *why = "windowed tensor-core backward launch failed";
  return e;
}

cudaError_t launch_both(const WinBwdParams (&prm)[2], const Maps (&maps)[2], const int (&grid)[2], cudaStream_t stream,
                        const char** why) {
  constexpr int kSmem = Cfg<0>::kSmemBytes > Cfg<1>::kSmemBytes ? Cfg<0>::kSmemBytes : Cfg<1>::kSmemBytes;
  static std::atomic<int> ready[kMaxDevices];
  cudaError_t e = prepare_once(win_bwd_both_kernel, ready, kThreads, 128 * kRegsOther + 256 * kRegsCompute, kSmem, why);
  if (e != cudaSuccess) return e;
  win_bwd_both_kernel<<<grid[0] + grid[1], kThreads, kSmem, stream>>>(maps[0], maps[1], prm[0], prm[1], (uint32_t)grid[0]);
  e = cudaGetLastError();
  if (e != cudaSuccess) *why = "windowed tensor-core backward launch failed";
  return e;
}

}  // namespace

cudaError_t launch_win_bwd_prep(const WinBwdParams& prm, const void* o, const float* lse, float* out, int sms,
                                cudaStream_t stream) {
  const int64_t blocks = prm.n_scalars / 128;
  const int64_t want = (blocks * 16 + kPrepWarps - 1) / kPrepWarps, cap = (int64_t)sms * 8 * 4;
  win_bwd_prep_kernel<<<(unsigned)(want < cap ? want : cap), kPrepWarps * 32, 0, stream>>>(
      prm, blocks, static_cast<const uint4*>(o), static_cast<const uint4*>(prm.dout), lse, out);
  return cudaGetLastError();
}

cudaError_t launch_win_bwd_join(const WinBwdParams& prm, const WinBwdSplit* splits, int n, cudaStream_t stream) {
  win_bwd_join_kernel<<<dim3((unsigned)n, 128 / kJoinRows, 2), kJoinRows * 32, 0, stream>>>(prm, splits);
  return cudaGetLastError();
}

cudaError_t launch_win_bwd_bf16(const WinBwdParams (&prm)[2], const void* q, const void* k, const void* v,
                                const void* dout, const int (&grid)[2], bool both, cudaStream_t stream, const char** why) {
  Maps maps[2];
  const WinBwdParams& p = prm[0];
  const int64_t hq = (int64_t)p.batch * p.heads_q, hk = (int64_t)p.batch * p.heads_kv;
  if (!encode_view(&maps[0].own_k, k, p.own, p.seq, hk) || !encode_view(&maps[0].own_v, v, p.own, p.seq, hk) ||
      !encode_view(&maps[0].y0, q, p.str, p.seq, hq) || !encode_view(&maps[0].y1, dout, p.str, p.seq, hq) ||
      !encode_view(&maps[1].y0, k, p.str, p.seq, hk) || !encode_view(&maps[1].y1, v, p.str, p.seq, hk)) {
    *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  maps[1].own_k = maps[0].own_k;  // (not used)
  maps[1].own_v = maps[0].own_v;
  if (both) return launch_both(prm, maps, grid, stream, why);
  const cudaError_t e = launch_pass<0>(prm[0], maps[0], grid[0], stream, why);
  return e != cudaSuccess ? e : launch_pass<1>(prm[1], maps[1], grid[1], stream, why);
}

}  // namespace ra
