// Attention of chunks over the paged cache, bf16, on the sm_100-family tensor cores.
//
// For the query rows of an item and the cached keys j that they see,
//   m = max_j s_j,  s_j = scale * q.k_j,  l = sum_j e^(s_j - m),  O = sum_j e^(s_j - m) v_j / l,
//   LSE = m + ln l,
// folded key tile by key tile of 128 slots with the running maximum and sum.
//
// An item is two query tiles of one sequence and key/value head.  A tile has 128 / group tokens
// with the rows of all heads of the group, so that every K and V tile that is loaded serves the
// whole group of twice as many tokens, and a single token fills as much of a tile as it can.
// A key tile is brought in pieces of the largest power of two (16 to 128 rows) that divides a
// page; pieces that nobody sees, and pages that are none, come as zeros from beyond the
// tensor's end.  Rows of a V tile that no token of the item sees are cleared in shared memory
// before the product: what pages hold there may be anything, and 0 * NaN is NaN.
//
// Shares: all items laid in a row, each as long as its key tiles, are cut into equal shares, one
// for each CTA or several (rounds) where the cache is larger than the L2: the CTAs of a round
// then walk the keys of a few heads, which stay there.  An item that is cut is written as parts,
// which a second kernel joins in order.
//
// Roles (one CTA per SM, 12 warps): warp 0 TMA producer, warp 1 tcgen05 issuer (both converged,
// one elected lane issues), warp 2 the items' records, warps 4-7 softmax of query tile 0, warps
// 8-11 of query tile 1 (one thread per row).
// TMEM: S0 cols 0-127 (P0 in 64-127), S1 128-255 (P1 in 192-255), O0 256-383, O1 384-511.
//
// Bound by the tensor cores (71% of the elapsed cycles busy) with the softmax between their
// products.  Measured: 2048 tokens of 32 and 8 heads, D 128, over 32k 651 us (1.06e12 operations,
// 1.64 PFLOP/s), the join with it; with the warp-level instruction 7.5 ms.
//
// Every mbarrier wait is bounded (~1 s).  On expiry the CTA raises an abort flag, records the
// role in the handle's status word, drains its own in-flight TMA loads and MMAs (bounded
// again), frees TMEM and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "paged_sm103.cuh"

namespace ra {
namespace {

constexpr int kWarps = 12;
constexpr int kThreads = kWarps * 32;  // 3 warpgroups: {producer, MMA, records, idle}, softmax 0, softmax 1
constexpr uint32_t kRegsLaunch = 168;
constexpr uint32_t kRegsOther = 120;
constexpr uint32_t kRegsSoftmax = 192;
static_assert(128 * kRegsOther + 256 * kRegsSoftmax <= kThreads * kRegsLaunch, "register split");
constexpr int kTile = 128;      // rows of a query tile and of a key tile
constexpr int kStages = 3;      // K/V ring
constexpr int kItemSlots = 4;   // items under way from the record warp to the others
constexpr int kNotes = 8;       // key tiles' notes from the producer: no role is that far apart
constexpr int kMinUnits = 2;    // key tiles of a share
constexpr uint32_t kStageRow = 144;  // 128 bytes of an output row, and 16 so that the lanes'
                                     // 16-byte writes fall into different banks

// An item's share as the roles need it.
struct alignas(16) Record {
  int32_t head, token;   // key/value head; first token of tile 0 in the packed batch
  int32_t n0, n1;        // tokens of the two tiles (n1 0: none)
  int32_t slot, b;       // slot of that token; sequence
  PagedSpan span;        // slots that any token of the item sees
  int32_t blk_head, blk_skip;  // its key tiles (PagedBlocks)
  int32_t k0, n;         // those of this share: [k0, k0 + n); n 0: no more items
  int32_t part;          // where to leave the sums, or -1: the item is whole
  __device__ __forceinline__ int at(int k) const { return k < blk_head ? k : k + blk_skip; }
};

template <int D>
struct Smem {
  static constexpr uint32_t kTileBytes = kTile * D * 2;
  static constexpr uint32_t kHalf = kTile * 128;  // 128 rows x one 128-byte swizzle column
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffKV = 2 * kTileBytes;
  static constexpr uint32_t kOffOut = kOffKV + kStages * kTileBytes;
  static constexpr uint32_t kOffRec = kOffOut + 256 * kStageRow;
  static constexpr uint32_t kOffBar = kOffRec + kItemSlots * (uint32_t)sizeof(Record);
  static constexpr uint32_t kOffPrefix = kOffBar + 320;
  static constexpr uint32_t kFixed = kOffPrefix + 1024;  // + slack to align the base to 1 KiB
};
static_assert(sizeof(Record) % 16 == 0, "records");

enum : int {
  kQFull = 0,  // one per query tile
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
constexpr uint32_t kOffSlot = 8 * kNumBars, kOffAbort = kOffSlot + 4, kOffNotes = kOffSlot + 8;  // behind the barriers
static_assert(kOffNotes + 4 * kNotes <= 320 && kOffNotes % 4 == 0, "barriers");

constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t col_s(int g) { return g ? 128u : 0u; }
__device__ __forceinline__ uint32_t col_o(int g) { return g ? 384u : 256u; }
// P (bf16, two per 32-bit column) overwrites the upper half of its tile's S columns once the
// softmax has read S; the next S MMA of that tile is issued after the PV MMA that reads P.
constexpr uint32_t kColP = 64;
constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(kTile, kTile, false, false);  // Q, K both K-major
constexpr float kRescaleSlack = 8.0f;  // log2 units: keep a stale max while p <= 2^8
constexpr float kLn2 = 0.6931471805599453f;

// --------------------------------------------------------------------- shares --
// Tokens of an item and its key tiles.
struct Item {
  int t0, tokens, s0, s1;
};
__device__ __forceinline__ Item item_of(const PagedSeq& q, int per_item, int i) {
  const int t0 = i * per_item, n = min(per_item, q.count - t0);
  return {t0, n, q.slot0() + t0, q.slot0() + t0 + n - 1};
}
__device__ __forceinline__ int item_units(const PagedChunkParams& P, const PagedSeq& q, int per_item, int i) {
  const Item it = item_of(q, per_item, i);
  return PagedBlocks<kTile>(paged_span(P.window, P.sinks, it.s0, it.s1)).n;  // (a token sees itself: >= 1)
}

struct Shares {
  int64_t all, per_head;  // units of all heads, of one
  int ctas, count;        // CTAs that take shares, shares
  __device__ __forceinline__ int64_t begin(int s) const { return all * s / count; }
};

// CTAs of this kernel's, where the row kernel reads other sequences' keys beside it: the two then
// end together.  A key tile takes a CTA 1.4 us, beside the reads 1.7; the reads take the time of their bytes at 6.6 TB/s
// if five eighths of the SMs are left to them, and longer in proportion if fewer are.  (One chunk of
// 512 tokens and 31 single ones under a window of 8192: one kernel after the other 226 us.  With 1.7,
// 1.2, 0.85 and 0.6 us a tile: 512 tokens, D 128, 186, 211, 261 and 345 us; D 64, whose tiles are half as long,
// 119, 119, 118 and 155; 64 tokens, one query tile an item: D 128 176, 204, 243 and 282, D 64 100, 98, 117 and 142.)
__device__ __forceinline__ int ctas_beside(int64_t units, double bytes, int sms) {
  const float work = 1.7f * (float)units, reads = (float)(bytes / 6.6e6);  // us
  const float few = 0.375f * (float)sms, need = 0.625f * (float)sms;
  const float n = work <= few * reads ? 1.1f * work / reads + 1.f : (float)sms * work / (need * reads + work);
  return max(1, min(sms, (int)ceilf(n)));
}

// Prefix sums of the sequences' units (one head), and the number of shares: as many as CTAs, times
// the rounds.  Every thread calls it; it ends with a barrier.
__device__ Shares shares_of(const PagedChunkParams& P, int per_item, int64_t* prefix, int64_t* scratch) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t again = 0, others = 0;  // slots that more than one item reads; that other kernels' sequences read
  for (int b0 = warp * 32; b0 < P.t.batch; b0 += kWarps * 32) {
    PagedSeq q{0, 0, 0};
    if (b0 + lane < P.t.batch) q = paged_seq(P.t, b0 + lane);
    const bool mine = paged_mine(P.t, q, P.group);
    const int items = mine ? (q.count + per_item - 1) / per_item : 0;
    if (!mine && q.count > 0) {
      const PagedSpan sp = paged_span(P.window, P.sinks, q.slot0(), q.length - 1);
      others += sp.sink + sp.hi - sp.lo;
    }
    if (items > 1) again += q.length;
    int64_t sum = 0;
    for (uint32_t some = __ballot_sync(0xffffffffu, items > 0); some; some &= some - 1) {
      const int src = __ffs(some) - 1;
      const PagedSeq o{0, __shfl_sync(0xffffffffu, q.count, src), __shfl_sync(0xffffffffu, q.length, src)};
      const int64_t all = warp_total(__shfl_sync(0xffffffffu, items, src), [&](int i) { return item_units(P, o, per_item, i); });
      if (lane == src) sum = all;
    }
    if (b0 + lane < P.t.batch) prefix[b0 + lane + 1] = sum;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    again += __shfl_xor_sync(0xffffffffu, again, o);
    others += __shfl_xor_sync(0xffffffffu, others, o);
  }
  if (lane == 0) scratch[warp] = again, scratch[kWarps + warp] = others;
  __syncthreads();
  if (warp == 0) paged_scan(P.t.batch, prefix);
  __syncthreads();
  again = others = 0;
  for (int i = 0; i < kWarps; ++i) again += scratch[i], others += scratch[kWarps + i];
  Shares s;
  s.per_head = prefix[P.t.batch];
  s.all = s.per_head * P.t.heads_kv;
  s.ctas = (int)gridDim.x;
  if (others > 0) s.ctas = ctas_beside(s.all, (double)others * P.t.heads_kv * P.row_bytes * 2, s.ctas);
  // (Rounds of 100 tiles a share at least: below that the parts cost more than the reads.  256 tokens
  // over 128k with 32 tiles 545 us, 64 459, 100 429; 512 over 64k 487, 402, 423.  2048 tokens over 32k
  // and 128k without rounds 693 and 3188 us, of 64 MB 656 and 2756, of 44 MB 653 and 2734.)
  const int64_t rounds = max((int64_t)1, min(min((int64_t)P.rounds, s.all / (100 * (int64_t)s.ctas)),
                                             again * P.t.heads_kv * P.row_bytes * 2 / kRoundBytes));
  s.count = (int)max((int64_t)1, min(rounds * s.ctas, s.all / kMinUnits));
  return s;
}

// Warp 2: this CTA's shares as records, a few ahead of the other roles.
__device__ void run_records(const PagedChunkParams& P, const Ctl& c, Record* recs, const int64_t* prefix, const Shares& sh,
                            int per_tile, int lane) {
  const int per_item = 2 * per_tile;
  // Nothing to join so far (all shares': a wait that runs out leaves none as they were).
  for (int s = (int)blockIdx.x + lane * sh.ctas; s < sh.count; s += 32 * sh.ctas) P.joins[s] = {0, 0, 0, 0};
  __syncwarp();
  uint32_t u = 0;
  for (int s = (int)blockIdx.x; s < sh.count; s += sh.ctas) {
    int64_t x = sh.begin(s);
    const int64_t x1 = sh.begin(s + 1);
    int b = -1, head = 0, i = 0;
    PagedSeq q{0, 0, 0};
    int64_t item_x = 0;
    while (x < x1) {
      if (b < 0) {  // where the share begins
        head = (int)(x / sh.per_head);
        const int64_t y = x - head * sh.per_head;
        b = paged_find(prefix, P.t.batch, y);
        q = paged_seq(P.t, b);
        const int items = (q.count + per_item - 1) / per_item;
        i = warp_find(items, y - prefix[b], item_x, [&](int i) { return item_units(P, q, per_item, i); });
        item_x += head * sh.per_head + prefix[b];
      } else {  // to the next item
        item_x = x;
        ++i;
        if (i * per_item >= q.count) {
          int64_t y = x - head * sh.per_head;
          if (y == sh.per_head) {
            ++head;
            y = 0;
          }
          b = paged_find(prefix, P.t.batch, y);
          q = paged_seq(P.t, b);
          i = 0;
        }
      }
      const Item it = item_of(q, per_item, i);
      const PagedSpan span = paged_span(P.window, P.sinks, it.s0, it.s1);
      const PagedBlocks<kTile> blocks(span);
      const int u0 = (int)(x - item_x), u1 = (int)min((int64_t)blocks.n, x1 - item_x);
      RA_BOUNDS(c.status, it.tokens > 0 && u0 >= 0 && u0 < u1 && head < P.t.heads_kv && q.token0 + it.t0 + it.tokens <= P.t.tokens, 120);
      const bool cut = u0 > 0 || u1 < blocks.n;
      const uint32_t slot = u % kItemSlots;
      if (!RA_WAIT(kItemEmpty + (int)slot, (u / kItemSlots) ^ 1u, kStatusTimeoutProducer)) return;
      if (lane == 0) {
        Record& r = recs[slot];
        r.head = head;
        r.token = q.token0 + it.t0;
        r.n0 = min(it.tokens, per_tile);
        r.n1 = it.tokens - r.n0;
        r.slot = it.s0;
        r.b = b;
        r.span = span;
        r.blk_head = blocks.head;
        r.blk_skip = blocks.skip;
        r.k0 = u0;
        r.n = u1 - u0;
        r.part = cut ? 2 * s + (u0 > 0 ? 0 : 1) : -1;
        if (cut && u0 == 0) {
          const int last = (int)(((item_x + blocks.n) * sh.count - 1) / sh.all);
          P.joins[s] = {head, r.token, it.tokens, last};
        }
        ptx::mbar_arrive(c.bar(kItemFull + (int)slot));
      }
      __syncwarp();
      ++u;
      x = item_x + u1;
    }
  }
  const uint32_t slot = u % kItemSlots;
  if (!RA_WAIT(kItemEmpty + (int)slot, (u / kItemSlots) ^ 1u, kStatusTimeoutProducer)) return;
  if (lane == 0) {
    recs[slot].n = 0;
    ptx::mbar_arrive(c.bar(kItemFull + (int)slot));
  }
}

// Consumer side: the record of this role's u-th item (nullptr at the end or on abort), and
// giving it back.
__device__ __forceinline__ const Record* next_record(const Ctl& c, const Record* recs, uint32_t u, uint32_t who) {
  const uint32_t slot = u % kItemSlots;
  if (!RA_WAIT(kItemFull + (int)slot, u / kItemSlots, who)) return nullptr;
  return recs[slot].n == 0 ? nullptr : recs + slot;
}
__device__ __forceinline__ void release_record(const Ctl& c, uint32_t u, int lane) {
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(c.bar(kItemEmpty + (int)(u % kItemSlots)));
}

// ------------------------------------------------------------------ producer --
struct ProducerState {
  uint32_t kv_issued, q_issued[2];
};

template <int D>
__device__ void run_producer(const PagedChunkParams& P, const Ctl& c, uint32_t sbase, const Record* recs, uint32_t* notes,
                             const CUtensorMap* tq, const CUtensorMap* tkv, ProducerState& st, int per_tile, int lane) {
  using S = Smem<D>;
  const int piece = P.piece, pieces = kTile / piece;
  const int rows_all = P.t.pages * 2 * P.t.heads_kv * P.t.page_rows;  // the first row that reads as zeros
  const uint32_t q_bytes = (uint32_t)(per_tile * P.group * D * 2);
  const uint64_t keep = ptx::l2_policy_evict_last();  // the items of a sequence read the same keys and values
  uint32_t tile = 0;
  for (uint32_t u = 0;; ++u) {
    const Record* r = next_record(c, recs, u, kStatusTimeoutProducer);
    if (r == nullptr) return;
    // The pages of the next 32 pieces, a lane each, read a group of tiles ahead (under load a read
    // takes longer than a tile).
    const int group = 32 / pieces, end = r->k0 + r->n;  // tiles of a group
    bool want;
    auto read = [&](int k) {
      k += lane / pieces;
      const int j = k < end ? r->at(k) * kTile + lane % pieces * piece : 0;
      want = k < end && ((j < r->span.hi && j + piece > r->span.lo) || j < r->span.sink);  // somebody sees it
      return want ? __ldg(P.t.page_table + r->b * P.t.width + j / P.t.page_rows) : -1;
    };
    int page_next = read(r->k0), rows = 0;
    uint32_t bad = 0u;
    for (int k = r->k0; k < end; ++k, ++tile) {
      const int at = (k - r->k0) % group;
      if (at == 0) {
        // A lane's row of keys, or the row of zeros.
        const int mine = k + lane / pieces, j = mine < end ? r->at(mine) * kTile + lane % pieces * piece : 0;
        const bool there = page_next >= 0 && page_next < P.t.pages;
        if (want && !there) atomicOr(P.t.status, kPagedStatusRange);
        bad = __ballot_sync(0xffffffffu, want && !there);
        rows = there ? (int)paged_row(P.t, page_next, 0, r->head, j % P.t.page_rows) : rows_all;
        page_next = read(k + group);
      }
      const int y_now = __shfl_sync(0xffffffffu, rows, at * pieces + lane % pieces);
      const uint32_t bad_now = (bad >> (at * pieces)) & ((1u << pieces) - 1u);
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const uint32_t s = st.kv_issued % kStages, use = st.kv_issued / kStages;
        if (!RA_WAIT(kKVEmpty + (int)s, use ^ 1u, kStatusTimeoutProducer)) return;
        if (which == 0 && lane == 0) notes[tile % kNotes] = bad_now;
        __syncwarp();
        const uint32_t dst = sbase + S::kOffKV + s * S::kTileBytes + lane * piece * 128;
        const int row = y_now == rows_all ? rows_all : y_now + which * P.t.heads_kv * P.t.page_rows;
        RA_BOUNDS(c.status, row >= 0 && row <= rows_all && (row == rows_all || row + piece <= rows_all), 121);
        ptx::mbar_arrive_expect_tx_warp(c.bar(kKVFull + (int)s), S::kTileBytes);
        __syncwarp();
        if (lane < pieces) {
          tma_load_2d_hint(dst, tkv, c.bar(kKVFull + (int)s), 0, row, keep);
          if (D == 128) tma_load_2d_hint(dst + S::kHalf, tkv, c.bar(kKVFull + (int)s), 64, row, keep);
        }
        __syncwarp();
        ++st.kv_issued;
      }
      if (k > r->k0) continue;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (g == 1 && r->n1 == 0) break;
        if (!RA_WAIT(kQEmpty + g, st.q_issued[g] ^ 1u, kStatusTimeoutProducer)) return;
        const uint32_t dst = sbase + S::kOffQ + g * S::kTileBytes;
        const int h = r->head * P.group, t = r->token + g * per_tile;
        ptx::mbar_arrive_expect_tx_warp(c.bar(kQFull + g), q_bytes);
        tma_load_3d_warp(dst, tq, c.bar(kQFull + g), 0, h, t);
        if (D == 128) tma_load_3d_warp(dst + S::kHalf, tq, c.bar(kQFull + g), 64, h, t);
        ++st.q_issued[g];
      }
    }
    release_record(c, u, lane);
  }
}

// ----------------------------------------------------------------------- MMA --
template <int D>
__device__ __forceinline__ void issue_s(uint32_t q0, uint32_t k0, uint32_t tmem, int g, uint32_t ks) {
  using S = Smem<D>;
  const uint32_t a0 = q0 + (uint32_t)g * (S::kTileBytes >> 4), b0 = k0 + ks * (S::kTileBytes >> 4);
#pragma unroll
  for (uint32_t kk = 0; kk < D / 16; ++kk) {  // steps of K = 16 over d
    const uint32_t off = ((kk >> 2) * S::kHalf + (kk & 3u) * 32u) >> 4;
    ptx::mma_bf16_ss_lo_warp(tmem + col_s(g), a0 + off, b0 + off, kIdescS, kk > 0 ? 1u : 0u);
  }
}
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t v0, uint32_t tmem, int g, uint32_t vs, bool accumulate) {
  constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(kTile, D, false, true);  // V is MN-major
  const uint32_t a0 = tmem + col_s(g) + kColP;
  const uint32_t b0 = v0 + vs * (Smem<D>::kTileBytes >> 4);
#pragma unroll
  for (uint32_t kk = 0; kk < 8; ++kk)  // 8 steps of 16 keys = 8 TMEM columns of P
    ptx::mma_bf16_ts_lo_warp(tmem + col_o(g), a0 + kk * 8u, b0 + ((kk * 2048u) >> 4), kIdescPV,
                             (accumulate || kk > 0) ? 1u : 0u);
}

// An item as the MMA warp walks it.
struct Seg {
  PagedSpan span;
  int head, skip, k0, n;
  bool two;
};

// Rows of a V tile that no token of the item sees, to zeros (the whole warp; seen rows stay).
template <int D>
__device__ __forceinline__ void clear_unseen(uint32_t tile, const Seg& s, int k, int lane) {
  const int j0 = (k < s.head ? k : k + s.skip) * kTile;
  if ((j0 >= s.span.lo && j0 + kTile <= s.span.hi) || j0 + kTile <= s.span.sink) return;
  for (int i = lane; i < kTile * 8; i += 32) {  // 8 lanes a row of 128 bytes
    if (s.span.holds(j0 + (i >> 3))) continue;
    ptx::st_shared_v4(tile + i * 16, 0u, 0u, 0u, 0u);
    if (D == 128) ptx::st_shared_v4(tile + Smem<D>::kHalf + i * 16, 0u, 0u, 0u, 0u);
  }
  ptx::fence_proxy_async_smem();
  __syncwarp();
}

template <int D>
__device__ void run_mma(const Ctl& c, uint32_t sbase, const Record* recs, uint32_t tmem, int lane) {
  using S = Smem<D>;
  const uint32_t q0 = ptx::desc_lo(sbase + S::kOffQ, 16);
  const uint32_t k0 = ptx::desc_lo(sbase + S::kOffKV, 16);
  const uint32_t v0 = ptx::desc_lo(sbase + S::kOffKV, S::kHalf);
  // the column map (S0, S1, O0, O1 = 0, 128, 256, 384) needs all 512 columns from 0
  RA_BOUNDS(c.status, tmem == 0u && col_o(1) + 128u <= kTmemCols, 122);
  uint32_t kv = 0, pj[2] = {0, 0}, qj[2] = {0, 0}, u = 0;
  auto next = [&](Seg& s) {
    const Record* r = next_record(c, recs, u, kStatusTimeoutMma);
    if (r == nullptr) return false;
    s = {r->span, r->blk_head, r->blk_skip, r->k0, r->n, r->n1 > 0};
    release_record(c, u++, lane);
    return true;
  };
  Seg cur, nxt;
  if (!next(cur)) return;
  // Scores of an item's key tile: the queries arrive with its first tile, and their shared
  // memory is free for the next item's after its last.
  auto scores = [&](const Seg& s, int kt, int g, uint32_t ks) {
    if (kt == 0) {
      if (!RA_WAIT(kQFull + g, qj[g], kStatusTimeoutMma)) return false;
      ++qj[g];
    }
    issue_s<D>(q0, k0, tmem, g, ks);
    ptx::mma_commit_warp(c.bar(kSFull + g));
    if (kt == s.n - 1) ptx::mma_commit_warp(c.bar(kQEmpty + g));
    return true;
  };
  uint32_t ks = kv % kStages;
  if (!RA_WAIT(kKVFull + (int)ks, kv / kStages, kStatusTimeoutMma)) return;
  if (!scores(cur, 0, 0, ks)) return;
  if (cur.two && !scores(cur, 0, 1, ks)) return;
  ptx::mma_commit_warp(c.bar(kKVEmpty + (int)ks));
  ++kv;
  for (int kt = 0;;) {
    const bool last = kt == cur.n - 1;
    bool has_next = true;
    int nkt = kt + 1;
    nxt = cur;
    if (last) {
      has_next = next(nxt);
      nkt = 0;
    }
    const uint32_t vs = kv % kStages;
    if (!RA_WAIT(kKVFull + (int)vs, kv / kStages, kStatusTimeoutMma)) return;
    ++kv;
    clear_unseen<D>(sbase + S::kOffKV + vs * S::kTileBytes, cur, cur.k0 + kt, lane);
    if (!RA_WAIT(kPFull + 0, pj[0], kStatusTimeoutMma)) return;
    ++pj[0];
    ptx::tc_fence_after();
    issue_pv<D>(v0, tmem, 0, vs, kt > 0);
    if (last) ptx::mma_commit_warp(c.bar(kOFull + 0));
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
      issue_pv<D>(v0, tmem, 1, vs, kt > 0);
      if (last) ptx::mma_commit_warp(c.bar(kOFull + 1));
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

// The finished rows of an item.  They go out through shared memory, 128 bytes of a row at a time,
// so that 8 lanes write 128 consecutive bytes; parts go out as columns of 4 channels by rows.
template <int D>
__device__ __forceinline__ void store_rows(const PagedChunkParams& P, uint32_t tO, uint8_t* stage, float m, float l, float fix,
                                           int64_t out, int64_t lse_at, int part_row, int lane) {
  const float inv = l == 0.f ? 0.f : 1.0f / (l + fix);
#pragma unroll 1
  for (int cc = 0; cc < D / 64; ++cc) {
    uint32_t v[64];
    __syncwarp();
    ptx::tmem_ld32x2(tO + cc * 64, tO + cc * 64 + 32, v);
    if (part_row >= 0) {
      if (out < 0) continue;  // no row of this thread's
      float4* dst = reinterpret_cast<float4*>(P.part_o) + (int64_t)(part_row >> 7) * (D / 4) * kTile + (part_row & 127);
#pragma unroll
      for (int q = 0; q < 16; ++q)
        dst[(cc * 16 + q) * kTile] = make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                                                 __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]));
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
        const int64_t to = __shfl_sync(0xffffffffu, out, r);
        if (to >= 0) reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.o) + to)[cc * 8 + (lane & 7)] = x;
      }
    }
  }
  if (out < 0) return;
  if (part_row >= 0) P.part_ml[part_row] = make_float4(m, l, fix, 0.f);
  else if (P.lse != nullptr) P.lse[lse_at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D>
__device__ void run_softmax(const PagedChunkParams& P, const Ctl& c, uint8_t* stage, const Record* recs,
                            const volatile uint32_t* notes, uint32_t tmem, int g, int wq, int per_tile, int lane) {
  const int row = wq * 32 + lane;  // TMEM lane = query row of the tile
  const int token = row / P.group, in_group = row - token * P.group;
  const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
  const uint32_t tS = tmem + lane_off + col_s(g);
  const uint32_t tO = tmem + lane_off + col_o(g);
  RA_BOUNDS(c.status, wq >= 0 && wq < 4 && (tS & 0xFFFFu) + 128u <= kTmemCols && (tO & 0xFFFFu) + 128u <= kTmemCols, 123);
  const float sl2 = P.scale_log2;
  uint32_t sj = 0, oj = 0, tile = 0;

  for (uint32_t u = 0;; ++u) {
    const Record* rec = next_record(c, recs, u, kStatusTimeoutSoftmax);
    if (rec == nullptr) return;
    const int n = rec->n;
    if (g == 1 && rec->n1 == 0) {
      tile += n;
      release_record(c, u, lane);
      continue;
    }
    const bool valid = token < (g ? rec->n1 : rec->n0);
    const int at = rec->token + g * per_tile + token;
    const int my = rec->slot + g * per_tile + token;  // slot of the row's token
    RA_BOUNDS(c.status, !valid || (at < P.t.tokens && in_group < P.group), 124);

    float m = -INFINITY, l = 0.f, fix = 0.f;
    for (int kt = 0; kt < n; ++kt, ++tile) {
      const int j0 = rec->at(rec->k0 + kt) * kTile;
      // columns [c_lo, c_hi), and those below c_s, are seen (rows of no token: whatever)
      const int c_hi = valid ? min(kTile, my + 1 - j0) : kTile;
      const int c_lo = valid && P.window > 0 ? my - P.window + 1 - j0 : 0;
      const int c_s = min(P.sinks - j0, c_hi);

      bool ok = wait_bar(c, c.bar(kSFull + g), sj & 1u, kStatusTimeoutSoftmax);
      ++sj;
      if (!__all_sync(0xffffffffu, ok)) return;
      ptx::tc_fence_after();
      const uint32_t bad = notes[tile % kNotes];  // pieces whose page is none
      const bool full = c_hi >= kTile && (c_lo <= 0 || c_s >= kTile) && bad == 0u;
      const bool first = kt == 0;

      // The tile's weights into tensor memory, their sum into part, the rounding of the largest
      // into top_fix; m moves when the tile's largest score exceeds it by the slack.  Two copies
      // of the code: without a mask the loop over the columns stays free of branches.
      bool resc = false;
      float alpha = 1.0f, part_sum, top_fix;
      auto weights = [&](auto edge) {
        uint32_t raw[128];
        float mx4[4];
        ptx::tmem_ld128_max(tS, raw, mx4);
        float* s = reinterpret_cast<float*>(raw);
        uint32_t live = 15u;
        if (decltype(edge)::value) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t bits = (below(c_hi - 32 * q) & ~below(c_lo - 32 * q)) | below(c_s - 32 * q);
            if (bad) {  // (16 columns at a time: the smallest piece)
              const int half = P.piece >> 4;
              if ((bad >> (2 * q / half)) & 1u) bits &= 0xffff0000u;
              if ((bad >> ((2 * q + 1) / half)) & 1u) bits &= 0x0000ffffu;
            }
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
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
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
        const float2 a = ptx::add2(ptx::add2(acc[0], acc[1]), ptx::add2(acc[2], acc[3]));
        part_sum = a.x + a.y;
        // The PV product weighs each key by its bf16-rounded p while l sums the fp32 p.  `fix`
        // holds the rounding of every tile's largest p: O is divided by l + fix, so that when
        // one key dominates a row its rounding cancels; the LSE is that of l.
        const float p_top = ptx::ex2_approx(ptx::fma2(make_float2(mx, mx), sc2, neg).x);
        const float p_top_bf = __uint_as_float(ptx::pack_bf16x2(p_top, 0.f) << 16);
        top_fix = p_top_bf - p_top;
      };
      if (__all_sync(0xffffffffu, full)) weights(std::false_type());
      else weights(std::true_type());
      if (!first && __any_sync(0xffffffffu, resc)) {
        // O and l were accumulated against the old max: bring them to the new one (after the
        // scores are consumed, so their registers are free).
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
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
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(c.bar(kPFull + g));
    }
    bool ok = wait_bar(c, c.bar(kOFull + g), oj & 1u, kStatusTimeoutSoftmax);
    ++oj;
    if (!__all_sync(0xffffffffu, ok)) return;
    ptx::tc_fence_after();
    const int head = rec->head * P.group + in_group;
    const int part_row = rec->part < 0 ? -1 : (rec->part * 2 + g) * kTile + row;
    store_rows<D>(P, tO, stage, m, l, fix, valid ? at * P.os.token + head * P.os.head : -1,
                  (int64_t)at * P.heads_q + head, part_row, lane);
    ptx::tc_fence_before();
    release_record(c, u, lane);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tkv,
                       const PagedChunkParams P) {
  using S = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ctl = sgen + S::kOffBar;
  Ctl c{sbase + S::kOffBar, reinterpret_cast<volatile uint32_t*>(ctl + kOffAbort), P.t.status};
  uint32_t* notes = reinterpret_cast<uint32_t*>(ctl + kOffNotes);
  Record* recs = reinterpret_cast<Record*>(sgen + S::kOffRec);
  int64_t* prefix = reinterpret_cast<int64_t*>(sgen + S::kOffPrefix);
  const int per_tile = kTile / P.group;

  next_may_come();
  const Shares sh = shares_of(P, 2 * per_tile, prefix, reinterpret_cast<int64_t*>(sgen + S::kOffOut));
  // Shares that there are none of leave nothing to join.
  for (int s = (int)blockIdx.x + threadIdx.x * gridDim.x; s < P.rounds * (int)gridDim.x; s += kThreads * gridDim.x)
    if (sh.all == 0 || s >= sh.count) P.joins[s] = {0, 0, 0, 0};
  if (sh.all == 0 || (int)blockIdx.x >= min(sh.ctas, sh.count)) return;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kItemSlots; ++s) {
      ptx::mbar_init(c.bar(kItemFull + s), 1);
      ptx::mbar_init(c.bar(kItemEmpty + s), kItemConsumers);
    }
    for (int g = 0; g < 2; ++g) {
      ptx::mbar_init(c.bar(kQFull + g), 1);
      ptx::mbar_init(c.bar(kQEmpty + g), 1);
      ptx::mbar_init(c.bar(kSFull + g), 1);
      ptx::mbar_init(c.bar(kPFull + g), 4);
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
    ptx::tma_prefetch_desc(&tkv);
  }
  if (warp == 1) {
    ptx::tmem_alloc(sbase + S::kOffBar + kOffSlot, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(ctl + kOffSlot);

  ProducerState ps{0u, {0u, 0u}};
  if (warp < 4) {
    ptx::regs_release<kRegsOther>();
    if (warp == 0) {
      run_producer<D>(P, c, sbase, recs, notes, &tq, &tkv, ps, per_tile, lane);
      __syncwarp();
    } else if (warp == 1) {
      run_mma<D>(c, sbase, recs, tmem, lane);
      // Every MMA this warp issued must retire before TMEM is freed.
      ptx::mma_commit_warp(c.bar(kDone));
      drain_bar(c, c.bar(kDone), 0);
      __syncwarp();
    } else if (warp == 2) {
      run_records(P, c, recs, prefix, sh, per_tile, lane);
    }
  } else {
    ptx::regs_acquire<kRegsSoftmax>();
    run_softmax<D>(P, c, sgen + S::kOffOut + (warp - 4) * 32 * kStageRow, recs, notes, tmem, (warp - 4) >> 2, warp & 3,
                   per_tile, lane);
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

// ---------------------------------------------------------------- cut items --
// The items that shares begin and do not end: an item's first part is there, the others at the
// beginning of the shares up to the last.  A warp has 32 rows, a lane each, and kJoinCols columns of
// 4 channels of them, and folds the parts in order, kJoinParts at a time, with the running maximum.
// Small CTAs, many for a share: an item may be cut into a part for every CTA of the GPU, and then
// there are few such items (20 tokens over 60k of one head 43 us, with 8 CTAs of 16 warps a share 60,
// with 2 139; with 8 parts at a time 41, but 2048 tokens over 32k 656 us instead of 651).
constexpr int kJoinWarps = 4, kJoinCols = 2, kJoinParts = 4;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_chunk_join_kernel(const PagedChunkParams P, int shares) {
  after_previous();
  const int per_tile = kTile / P.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // A lane has the record of a round's share (most have nothing to join).
  static_assert(kMaxRounds <= 32, "a lane each");
  PagedJoin own{0, 0, 0, 0};
  if (lane < kMaxRounds && (int)blockIdx.x + lane * (int)gridDim.x < shares) own = P.joins[blockIdx.x + lane * gridDim.x];
  const int g = (int)blockIdx.y >> 2, in_tile = ((int)blockIdx.y & 3) * 32 + lane;  // this lane's row of both tiles
  const int token = in_tile / P.group;
  const int col = ((int)blockIdx.z * kJoinWarps + warp) * kJoinCols;
  for (uint32_t some = __ballot_sync(0xffffffffu, own.tokens != 0); some; some &= some - 1) {
    const int k = __ffs(some) - 1, s = (int)blockIdx.x + k * (int)gridDim.x;
    const PagedJoin rec{__shfl_sync(0xffffffffu, own.head, k), __shfl_sync(0xffffffffu, own.token, k),
                        __shfl_sync(0xffffffffu, own.tokens, k), __shfl_sync(0xffffffffu, own.last, k)};
    if (token >= per_tile || g * per_tile + token >= rec.tokens) continue;
    const int count = rec.last - s + 1;
    auto tile_of = [&](int i) { return (i == 0 ? 2 * s + 1 : 2 * (s + i)) * 2 + g; };
    const int at = rec.token + g * per_tile + token, head = rec.head * P.group + in_tile - token * P.group;
    const float4* parts = reinterpret_cast<const float4*>(P.part_o) + (int64_t)col * kTile + in_tile;
    float m = -INFINITY;
    float2 lf = make_float2(0.f, 0.f);  // the sum, its correction
    float4 x[kJoinCols];
#pragma unroll
    for (int q = 0; q < kJoinCols; ++q) x[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < count; i0 += kJoinParts) {
      float4 ml[kJoinParts], y[kJoinParts][kJoinCols];
#pragma unroll
      for (int i = 0; i < kJoinParts; ++i) {
        ml[i].x = -INFINITY;
        if (i0 + i < count) {
          const int tile = tile_of(i0 + i);
          ml[i] = P.part_ml[tile * kTile + in_tile];
#pragma unroll
          for (int q = 0; q < kJoinCols; ++q) y[i][q] = parts[((int64_t)tile * (D / 4) + q) * kTile];
        }
      }
      float top = m;
#pragma unroll
      for (int i = 0; i < kJoinParts; ++i) top = fmaxf(top, ml[i].x);
      const float ref = top == -INFINITY ? 0.f : top, alpha = exp2f(m - ref);
      m = top;
      lf.x *= alpha;
      lf.y *= alpha;
#pragma unroll
      for (int q = 0; q < kJoinCols; ++q) x[q].x *= alpha, x[q].y *= alpha, x[q].z *= alpha, x[q].w *= alpha;
#pragma unroll
      for (int i = 0; i < kJoinParts; ++i) {
        if (i0 + i >= count) break;
        const float f = exp2f(ml[i].x - ref);
        lf.x = fmaf(ml[i].y, f, lf.x);
        lf.y = fmaf(ml[i].z, f, lf.y);
#pragma unroll
        for (int q = 0; q < kJoinCols; ++q) {
          x[q].x = fmaf(y[i][q].x, f, x[q].x), x[q].y = fmaf(y[i][q].y, f, x[q].y);
          x[q].z = fmaf(y[i][q].z, f, x[q].z), x[q].w = fmaf(y[i][q].w, f, x[q].w);
        }
      }
    }
    const float l = lf.x, inv = l == 0.f ? 0.f : 1.0f / (l + lf.y);
    uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.o) + at * P.os.token + head * P.os.head + col * 4);
#pragma unroll
    for (int q = 0; q < kJoinCols; ++q)
      dst[q] = make_uint2(ptx::pack_bf16x2(x[q].x * inv, x[q].y * inv), ptx::pack_bf16x2(x[q].z * inv, x[q].w * inv));
    if (col == 0 && P.lse != nullptr)
      P.lse[(int64_t)at * P.heads_q + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

template <int D>
cudaError_t launch(const PagedChunkParams& prm, int grid, cudaStream_t stream, const char** why) {
  CUtensorMap tq, tkv;
  const int per_tile = kTile / prm.group;
  if (!encode_rows(&tkv, prm.t.cache, (int64_t)prm.t.pages * 2 * prm.t.heads_kv * prm.t.page_rows, D, prm.piece) ||
      !encode_packed(&tq, prm.q, prm.qs, prm.t.tokens, prm.heads_q, D, prm.group, per_tile)) {
    *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  static std::atomic<int> ready[kMaxDevices];
  constexpr uint32_t kMost = Smem<D>::kFixed + (kMaxChunkSequences + 1) * 8;
  static_assert(kMost <= 232448, "shared memory");
  cudaError_t e = prepare_once(paged_chunk_kernel<D>, ready, kThreads, 128 * kRegsOther + 256 * kRegsSoftmax, (int)kMost, why);
  if (e != cudaSuccess) return e;
  paged_chunk_kernel<D><<<grid, kThreads, Smem<D>::kFixed + (prm.t.batch + 1) * 8, stream>>>(tq, tkv, prm);
  e = cudaGetLastError();
  if (e != cudaSuccess) *why = "launch failed";
  return e;
}

}  // namespace

cudaError_t launch_paged_chunk(int head_dim, const PagedChunkParams& prm, int grid, cudaStream_t stream, const char** why) {
  return head_dim == 128 ? launch<128>(prm, grid, stream, why) : launch<64>(prm, grid, stream, why);
}

cudaError_t launch_paged_chunk_join(int head_dim, const PagedChunkParams& prm, int grid, cudaStream_t stream) {
  const dim3 blocks((unsigned)grid, 8, (unsigned)(head_dim / 4 / (kJoinWarps * kJoinCols)));
  const int shares = grid * prm.rounds;
  return head_dim == 128 ? launch_behind(paged_chunk_join_kernel<128>, blocks, kJoinWarps * 32, 0, stream, prm, shares)
                         : launch_behind(paged_chunk_join_kernel<64>, blocks, kJoinWarps * 32, 0, stream, prm, shares);
}

}  // namespace ra
