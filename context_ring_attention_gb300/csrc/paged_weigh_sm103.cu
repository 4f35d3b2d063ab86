// The attention weight that cached keys receive from chunks of new tokens, bf16, on the
// sm_100-family tensor cores (include/ra.h, ra_paged_weigh; paged_weigh.cu has the formula).
//
// An item is 256 keys of one sequence and key/value head, two tiles of 128, with the query tiles
// that see any of them: 128 / group tokens with the rows of all heads of the group.  The scores
// are made with the keys in the rows (S^T = K Q^T), so that a thread has one key and sums
// e^(score - LSE) over the columns in its registers: no exchange between threads, no product
// after it.  The keys lie in tensor memory, as the first operand, while the queries stream by.
//
// The LSE enters by the product too: the queries have 16 channels more, -LSE / scale in three
// bf16 terms (2^-24 of it) and zeros, the keys 1, 1, 1 and zeros; a first kernel makes them.  What a
// thread has left to do for a score is one multiplication, the exponential and the sum.
//
// Shares: all items laid in a row, each as long as its query tiles, cut into one share per CTA.
// An item that is cut leaves a sum per key and part, which a last kernel adds in order.
//
// Bound by the tensor cores and the exponentials alike (69% and 64% of the cycles busy, 55% of the
// issue slots).  Measured: 1000 tokens of 32 and 8 heads, D 128, over 32k 186 us (2.6e11 operations,
// 1.42 PFLOP/s), 4000 tokens 641 us (1.61).  With the LSE subtracted by the warps that sum, from
// shared memory, 219 (the product is shorter by its ninth part, the sums longer); with the second
// half of a warp's scores read behind the first's exponentials 192 (the products wait for it); with the
// extra channels made by a warp of this kernel 250, with every tile asked whether it needs a mask
// 189, with the warp-level instruction 3.5 ms.
//
// Roles (one CTA per SM, 20 warps): warp 0 TMA producer, warp 1 tcgen05 issuer, warp 2 the
// items' records, warps 4-19 sums: four for each key tile and half of the columns (two threads
// per key, whose sums meet in shared memory at an item's end).  With one thread per key, two
// warps per scheduler, neither unit was busy half of the time.
// TMEM: scores of the two key tiles 0-127 and 128-255, the keys 256-319 and 320-383, their extra
// channels 384-391.
//
// Every mbarrier wait is bounded as in paged_chunk_sm103.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "paged_sm103.cuh"

namespace ra {
namespace {

constexpr int kWarps = 20;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 128;
constexpr int kPair = 2 * kTile;  // keys of an item
constexpr int kKeySlots = 2;      // key tiles on their way to tensor memory
constexpr int kStages = 3;        // query tiles
constexpr int kItemSlots = 4;
constexpr int kMinUnits = 2;      // query tiles of a share
constexpr uint32_t kExtra = kTile * 32;  // bytes of a tile's 16 channels more: [2][128 rows][16 bytes], the second half zeros

struct alignas(16) Record {
  int32_t head, b, key0, part;    // part: where to leave the sums, or -1: the item is whole
  int32_t token0, count, length;  // of the sequence
  int32_t t0, n;                  // query tiles [t0, t0 + n); n 0: no more items
  int32_t extra;                  // place of the sequence's first tile among the tiles' extra channels
  int32_t pad[2];
  __device__ __forceinline__ int slot0() const { return length - count; }
};

template <int D>
struct Smem {
  static constexpr uint32_t kTileBytes = kTile * D * 2;
  static constexpr uint32_t kHalf = kTile * 128;
  static constexpr uint32_t kOffK = 0;
  static constexpr uint32_t kOffQ = kKeySlots * kTileBytes;
  static constexpr uint32_t kOffExtra = kOffQ + kStages * kTileBytes;
  static constexpr uint32_t kOffHalf = kOffExtra + kStages * kExtra;  // sums of the second halves, by item slot
  static constexpr uint32_t kOffRec = kOffHalf + kItemSlots * kPair * 4;
  static constexpr uint32_t kOffBar = kOffRec + kItemSlots * (uint32_t)sizeof(Record);
  static constexpr uint32_t kOffPrefix = kOffBar + 448;
  static constexpr uint32_t kFixed = kOffPrefix + 1024;  // + slack to align the base to 1 KiB
};

enum : int {
  kKFull = 0,
  kKEmpty = kKFull + kKeySlots,
  kQFull = kKEmpty + kKeySlots,
  kQEmpty = kQFull + kStages,
  kSFull = kQEmpty + kStages,  // one per key tile
  kSEmpty = kSFull + 2,
  kKReady = kSEmpty + 2,       // keys in tensor memory
  kHalfSum = kKReady + 2,  // key tile * kItemSlots + item slot
  kItemFull = kHalfSum + 2 * kItemSlots,
  kItemEmpty = kItemFull + kItemSlots,
  kDone = kItemEmpty + kItemSlots,
  kNumBars = kDone + 1
};
constexpr uint32_t kItemConsumers = 18;  // producer, MMA and 16 warps of sums
constexpr uint32_t kOffSlot = 8 * kNumBars, kOffAbort = kOffSlot + 4, kOffNotes = kOffSlot + 8;
static_assert(kOffNotes + 4 * 2 * kItemSlots <= 448, "barriers");

constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t col_s(int g) { return (uint32_t)g * 128u; }
__device__ __forceinline__ uint32_t col_k(int g) { return 256u + (uint32_t)g * 64u; }  // two channels a column
constexpr uint32_t kColOnes = 384;                                                     // 16 channels: 1, 1, 1, 0 ..

constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(kTile, kTile, false, false);  // K, Q both K-major
// An operand without a swizzle: groups of 8 rows of 16 bytes follow each other (128 bytes), the
// two halves of the 16 channels lie 2 KiB apart.
__device__ __forceinline__ uint64_t plain_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(2048u >> 4) << 16) | ((uint64_t)(128u >> 4) << 32) | ((uint64_t)1 << 46);
}
// D[tmem] += A[tmem] * B[smem], one step of 16; a converged warp executes it, one elected lane issues.
__device__ __forceinline__ void mma_extra_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.eq.b32 p, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc)
      : "memory");
}

// --------------------------------------------------------------------- shares --
// Whether some token of the call sees slot j of a sequence.
__device__ __forceinline__ bool seen_by_some(const PagedWeighChunkParams& P, int slot0, int count, int j) {
  return count > 0 && (P.window == 0 || j > slot0 - P.window || j < P.sinks);
}
// Query tiles that see one of the keys [key0, key0 + 256) of a sequence: [t0, t0 + n).
struct Tiles {
  int t0, n;
};
__device__ __forceinline__ Tiles tiles_of(const PagedWeighChunkParams& P, const PagedSeq& q, int per_tile, int i) {
  const int j0 = i * kPair, jl = min(j0 + kPair, q.length) - 1;
  const int tok0 = max(0, j0 - q.slot0());
  const int64_t far = P.window > 0 && j0 >= P.sinks ? (int64_t)jl + P.window - q.slot0() : q.count;
  const int tok1 = (int)max((int64_t)0, min((int64_t)q.count, far));
  if (tok1 <= tok0) return {0, 0};
  return {tok0 / per_tile, (tok1 + per_tile - 1) / per_tile - tok0 / per_tile};
}

struct Shares {
  int64_t all, per_head;
  int count;
  __device__ __forceinline__ int64_t begin(int s) const { return all * s / count; }
};

// Slots that no token sees keep what they had: copied by all warps of the launch.
__device__ void copy_unseen(const PagedWeighChunkParams& P) {
  if (P.weight_in == P.weight) return;
  constexpr int kSpan = 1024;
  const int lane = threadIdx.x & 31, me = (int)blockIdx.x * kWarps + (threadIdx.x >> 5), all = (int)gridDim.x * kWarps;
  for (int b0 = 0; b0 < P.t.batch; b0 += 32) {
    int lo = 0, hi = 0;
    if (b0 + lane < P.t.batch) {
      const PagedSeq q = paged_seq(P.t, b0 + lane);
      if (!paged_mine(P.t, q, P.group)) hi = 0;
      else if (q.count == 0) hi = q.length;
      else if (P.window > 0) lo = P.sinks, hi = q.slot0() - P.window + 1;
      hi = (int)min((int64_t)hi, P.weight_width);
    }
    for (uint32_t some = __ballot_sync(0xffffffffu, lo < hi); some; some &= some - 1) {
      const int src = __ffs(some) - 1, l = __shfl_sync(0xffffffffu, lo, src), h = __shfl_sync(0xffffffffu, hi, src);
      const int spans = (h - l + kSpan - 1) / kSpan;
      for (int64_t k = (me + all - (b0 + src) % all) % all; k < (int64_t)spans * P.t.heads_kv; k += all) {
        const int head = (int)(k / spans);
        const int64_t at = ((int64_t)(b0 + src) * P.t.heads_kv + head) * P.weight_width;
        const int s0 = l + (int)(k % spans) * kSpan;
        for (int j = s0 + lane; j < min(h, s0 + kSpan); j += 32)
          P.weight[at + j] = P.weight_in != nullptr ? P.weight_in[at + j] : 0.f;
      }
    }
  }
}

// The weight of slot j, whose sum over the rows is known.
__device__ __forceinline__ void put(const PagedWeighChunkParams& P, int b, int head, int j, int slot0, float sum) {
  if (j >= P.weight_width) return;  // (reported, as every sequence of more slots is)
  const int64_t at = ((int64_t)b * P.t.heads_kv + head) * P.weight_width + j;
  RA_BOUNDS(P.t.status, j >= 0 && at < (int64_t)P.t.batch * P.t.heads_kv * P.weight_width, 130);
  P.weight[at] = (P.weight_in != nullptr && j < slot0 ? P.weight_in[at] : 0.f) + sum;
}

// Warp 2: this CTA's share as records, a few ahead of the other roles.
__device__ void run_records(const PagedWeighChunkParams& P, const Ctl& c, Record* recs, const int64_t* prefix,
                            const Shares& sh, int per_tile, int lane) {
  uint32_t u = 0;
  const int s = (int)blockIdx.x;
  int64_t x = sh.begin(s);
  const int64_t x1 = sh.begin(s + 1);
  int head = (int)(x / sh.per_head), b = paged_find(prefix, P.t.batch, x - head * sh.per_head);
  PagedSeq q = paged_seq(P.t, b);
  int64_t item_x = 0;
  int items = (q.length + kPair - 1) / kPair;
  int i = warp_find(items, x - head * sh.per_head - prefix[b], item_x, [&](int k) { return tiles_of(P, q, per_tile, k).n; });
  item_x += head * sh.per_head + prefix[b];
  while (x < x1) {
    const Tiles t = tiles_of(P, q, per_tile, i);
    if (t.n > 0) {
      const int u0 = (int)(x - item_x), u1 = (int)min((int64_t)t.n, x1 - item_x);
      RA_BOUNDS(c.status, i < items && u0 >= 0 && u0 < u1 && head < P.t.heads_kv && q.token0 + q.count <= P.t.tokens, 131);
      const bool cut = u0 > 0 || u1 < t.n;
      const uint32_t slot = u % kItemSlots;
      if (!RA_WAIT(kItemEmpty + (int)slot, (u / kItemSlots) ^ 1u, kStatusTimeoutProducer)) return;
      if (lane == 0) {
        Record& r = recs[slot];
        r.head = head;
        r.b = b;
        r.key0 = i * kPair;
        r.part = cut ? 2 * s + (u0 > 0 ? 0 : 1) : -1;
        r.token0 = q.token0;
        r.count = q.count;
        r.length = q.length;
        r.t0 = t.t0 + u0;
        r.n = u1 - u0;
        r.extra = __ldcg(P.extra_at + b);
        if (cut && u0 == 0) P.joins[s] = {head, b, i * kPair, (int)(((item_x + t.n) * sh.count - 1) / sh.all)};
        ptx::mbar_arrive(c.bar(kItemFull + (int)slot));
      }
      __syncwarp();
      ++u;
      x = item_x + u1;
    }
    // to the next item
    item_x = x;
    ++i;
    if (i >= items && x < x1) {
      if (x - head * sh.per_head == sh.per_head) ++head;
      b = paged_find(prefix, P.t.batch, x - head * sh.per_head);
      q = paged_seq(P.t, b);
      items = (q.length + kPair - 1) / kPair;
      i = 0;
    }
  }
  const uint32_t slot = u % kItemSlots;
  if (!RA_WAIT(kItemEmpty + (int)slot, (u / kItemSlots) ^ 1u, kStatusTimeoutProducer)) return;
  if (lane == 0) {
    recs[slot].n = 0;
    ptx::mbar_arrive(c.bar(kItemFull + (int)slot));
  }
}

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
  uint32_t k_issued, q_issued;
};

template <int D>
__device__ void run_producer(const PagedWeighChunkParams& P, const Ctl& c, uint32_t sbase, const Record* recs, uint32_t* notes,
                             const CUtensorMap* tq, const CUtensorMap* tkv, ProducerState& st, int per_tile, int lane) {
  using S = Smem<D>;
  const int piece = P.piece, pieces = kTile / piece;
  const int rows_all = P.t.pages * 2 * P.t.heads_kv * P.t.page_rows;  // the first row that reads as zeros
  const uint32_t q_bytes = (uint32_t)(per_tile * P.group * D * 2);
  for (uint32_t u = 0;; ++u) {
    const Record* r = next_record(c, recs, u, kStatusTimeoutProducer);
    if (r == nullptr) return;
    // Lane p brings piece p of a key tile: its page's row of keys, or the row of zeros.
    auto load_keys = [&](int g) {
      const int j = r->key0 + g * kTile + lane * piece;
      const bool want = lane < pieces && j < r->length &&
                        (seen_by_some(P, r->slot0(), r->count, j) ||
                         seen_by_some(P, r->slot0(), r->count, min(j + piece, r->length) - 1));
      int row = rows_all;
      if (want) {
        const int page = paged_page(P.t, r->b, j / P.t.page_rows);
        if (page >= 0) row = (int)paged_row(P.t, page, 0, r->head, j % P.t.page_rows);
      }
      const uint32_t bad = __ballot_sync(0xffffffffu, want && row == rows_all);
      const uint32_t s = st.k_issued % kKeySlots, use = st.k_issued / kKeySlots;
      if (!RA_WAIT(kKEmpty + (int)s, use ^ 1u, kStatusTimeoutProducer)) return false;
      if (lane == 0) notes[2 * (u % kItemSlots) + g] = bad;
      __syncwarp();
      RA_BOUNDS(c.status, row >= 0 && (row == rows_all || row + piece <= rows_all), 132);
      const uint32_t dst = sbase + S::kOffK + s * S::kTileBytes + lane * piece * 128;
      ptx::mbar_arrive_expect_tx_warp(c.bar(kKFull + (int)s), S::kTileBytes);
      __syncwarp();
      if (lane < pieces) {
        ptx::tma_load_2d(dst, tkv, c.bar(kKFull + (int)s), 0, row);
        if (D == 128) ptx::tma_load_2d(dst + S::kHalf, tkv, c.bar(kKFull + (int)s), 64, row);
      }
      __syncwarp();
      ++st.k_issued;
      return true;
    };
    auto load_queries = [&](int t) {
      const uint32_t s = st.q_issued % kStages, use = st.q_issued / kStages;
      if (!RA_WAIT(kQEmpty + (int)s, use ^ 1u, kStatusTimeoutProducer)) return false;
      const uint32_t dst = sbase + S::kOffQ + s * S::kTileBytes;
      const int h = r->head * P.group, token = r->token0 + t * per_tile;
      RA_BOUNDS(c.status, token >= 0 && token < P.t.tokens && h + P.group <= P.heads_q, 133);
      ptx::mbar_arrive_expect_tx_warp(c.bar(kQFull + (int)s), q_bytes + kExtra / 2);
      tma_load_3d_warp(dst, tq, c.bar(kQFull + (int)s), 0, h, token);
      if (D == 128) tma_load_3d_warp(dst + S::kHalf, tq, c.bar(kQFull + (int)s), 64, h, token);
      const int at = min(r->extra + t, P.tiles - 1);
      RA_BOUNDS(c.status, r->extra >= 0 && r->extra + t < P.tiles, 136);
      ptx::bulk_load_warp(sbase + S::kOffExtra + s * kExtra, P.extra + ((int64_t)r->head * P.tiles + at) * kTile, kExtra / 2,
                          c.bar(kQFull + (int)s));
      ++st.q_issued;
      return true;
    };
    if (!load_keys(0) || !load_keys(1)) return;
    for (int t = 0; t < r->n; ++t)
      if (!load_queries(r->t0 + t)) return;
    release_record(c, u, lane);
  }
}

// ----------------------------------------------------------------------- MMA --
template <int D>
__device__ void run_mma(const Ctl& c, uint32_t sbase, const Record* recs, uint32_t tmem, int lane) {
  using S = Smem<D>;
  const uint32_t q0 = ptx::desc_lo(sbase + S::kOffQ, 16);
  const uint64_t extra0 = plain_desc(sbase + S::kOffExtra);
  RA_BOUNDS(c.status, tmem == 0u && kColOnes + 8u <= kTmemCols, 134);
  uint32_t tile = 0;
  for (uint32_t u = 0;; ++u) {
    const Record* r = next_record(c, recs, u, kStatusTimeoutMma);
    if (r == nullptr) return;
    const int n = r->n;
    release_record(c, u, lane);
    for (int t = 0; t < n; ++t, ++tile) {
      const uint32_t qs = tile % kStages;
      if (!RA_WAIT(kQFull + (int)qs, tile / kStages, kStatusTimeoutMma)) return;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (t == 0 && !RA_WAIT(kKReady + g, u, kStatusTimeoutMma)) return;
        if (!RA_WAIT(kSEmpty + g, tile ^ 1u, kStatusTimeoutMma)) return;
        ptx::tc_fence_after();
        const uint32_t b0 = q0 + qs * (S::kTileBytes >> 4);
#pragma unroll
        for (uint32_t kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * S::kHalf + (kk & 3u) * 32u) >> 4;
          ptx::mma_bf16_ts_lo_warp(tmem + col_s(g), tmem + col_k(g) + kk * 8u, b0 + off, kIdescS, kk > 0 ? 1u : 0u);
        }
        // (last: the scores' own sums are not cut at the size of the LSE)
        mma_extra_warp(tmem + col_s(g), tmem + kColOnes, extra0 + qs * (kExtra >> 4), kIdescS);
        ptx::mma_commit_warp(c.bar(kSFull + g));
      }
      ptx::mma_commit_warp(c.bar(kQEmpty + (int)qs));
    }
  }
}

// ---------------------------------------------------------------------- sums --
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : ~(~0u << n)); }
// 32 or 16 registers per thread -> 32 lanes by as many columns of tensor memory, waited.
__device__ __forceinline__ void tmem_st32_words(uint32_t taddr, const uint32_t (&r)[32]) { ptx::tmem_st32(taddr, r); }
__device__ __forceinline__ void tmem_st16_words(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ int clamped(int64_t x) { return (int)max((int64_t)-1, min((int64_t)(kTile + 1), x)); }

template <int D>
__device__ void run_sums(const PagedWeighChunkParams& P, const Ctl& c, uint32_t sbase, const Record* recs,
                         const volatile uint32_t* notes,
                         float* halves, uint32_t tmem, int g, int half, int wq, int per_tile, int lane) {
  const int row = wq * 32 + lane;  // TMEM lane = key of the tile
  const uint32_t tS = tmem + ((uint32_t)(wq * 32) << 16) + half * 64;
  RA_BOUNDS(c.status, wq >= 0 && wq < 4, 135);
  const float2 sc2 = make_float2(P.scale_log2, P.scale_log2);
  uint32_t tile = 0;
  for (uint32_t u = 0;; ++u) {
    const Record* r = next_record(c, recs, u, kStatusTimeoutSoftmax);
    if (r == nullptr) return;
    const int j = r->key0 + g * kTile + row, slot0 = r->slot0(), count = r->count, n = r->n, t0 = r->t0;
    const bool mine = j < r->length && seen_by_some(P, slot0, count, j);
    // The keys into tensor memory, from where the products take them: as operands from shared
    // memory both sides together cost more of its cycles than the product takes.  The products of
    // the item before are done (its last scores were waited for).
    {
      const int ks = g;  // (two places, two tiles an item)
      if (!RA_WAIT(kKFull + ks, u, kStatusTimeoutSoftmax)) return;
      uint32_t w[D / 4];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {  // 16 bytes at a time of this thread's half of the row
        const int ch = half * (D / 16) + i;
        const uint32_t at = sbase + Smem<D>::kOffK + ks * Smem<D>::kTileBytes + (ch >> 3) * Smem<D>::kHalf + row * 128 +
                            (((ch & 7) ^ (row & 7)) * 16);
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3]) : "r"(at) : "memory");
      }
      const uint32_t to = tmem + ((uint32_t)(wq * 32) << 16) + col_k(g) + half * (D / 4);
      if constexpr (D == 128) tmem_st32_words(to, w);
      else tmem_st16_words(to, w);
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(c.bar(kKReady + g));
        ptx::mbar_arrive(c.bar(kKEmpty + ks));
      }
    }
    float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    // Query tiles [full0, full1) are seen by every key of the warp that is asked for, in every row:
    // told once an item, as the sums are bound by the instructions of a tile.
    int full0, full1;
    {
      const int top = __reduce_max_sync(0xffffffffu, mine ? j : 0);
      const bool edge = mine && P.window > 0 && j >= P.sinks;
      const int low = __reduce_min_sync(0xffffffffu, edge ? j : INT32_MAX);
      full0 = top > slot0 ? (top - slot0 + per_tile - 1) / per_tile : 0;
      full1 = count / per_tile;
      if (low != INT32_MAX) full1 = (int)min((int64_t)full1, max((int64_t)0, (int64_t)low + P.window - slot0) / per_tile);
    }
    for (int t = 0; t < n; ++t, ++tile) {
      const bool ok = wait_bar(c, c.bar(kSFull + g), tile & 1u, kStatusTimeoutSoftmax);
      if (!__all_sync(0xffffffffu, ok)) return;
      ptx::tc_fence_after();
      uint32_t raw[64];
      ptx::tmem_ld32x2(tS + col_s(g), tS + col_s(g) + 32, raw);
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(c.bar(kSEmpty + g));  // (a warp's 32 arrivals would come one after the other)
      const float* s = reinterpret_cast<const float*>(raw);
      auto sums = [&](auto edge) {
        int c_lo = 0, c_hi = 0;
        if (decltype(edge)::value) {
          // rows [c_lo, c_hi) see the key (keys that nobody asks for: all)
          const int first = slot0 + (t0 + t) * per_tile;  // slot of the tile's first token
          c_hi = min(per_tile, count - (t0 + t) * per_tile) * P.group;
          if (mine) {
            c_lo = clamped(j - first) * P.group;
            if (P.window > 0 && j >= P.sinks) c_hi = min(c_hi, clamped((int64_t)j + P.window - first) * P.group);
          }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t bits = ~0u;
          if (decltype(edge)::value) {
            bits = below(c_hi - 64 * half - 32 * q) & ~below(c_lo - 64 * half - 32 * q);
            if (!__any_sync(0xffffffffu, bits != 0u)) continue;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {  // columns 32 q + 4 e .. of this half
            const int col = 32 * q + 4 * e;
            float2 x = ptx::mul2(make_float2(s[col], s[col + 1]), sc2);
            float2 y = ptx::mul2(make_float2(s[col + 2], s[col + 3]), sc2);
            x.x = ptx::ex2_approx(x.x);
            x.y = ptx::ex2_approx(x.y);
            y.x = ptx::ex2_approx(y.x);
            y.y = ptx::ex2_approx(y.y);
            if (decltype(edge)::value) {
              x.x = ((bits >> (4 * e)) & 1u) ? x.x : 0.f;
              x.y = ((bits >> (4 * e + 1)) & 1u) ? x.y : 0.f;
              y.x = ((bits >> (4 * e + 2)) & 1u) ? y.x : 0.f;
              y.y = ((bits >> (4 * e + 3)) & 1u) ? y.y : 0.f;
            }
            acc[(2 * e) & 3] = ptx::add2(acc[(2 * e) & 3], x);
            acc[(2 * e + 1) & 3] = ptx::add2(acc[(2 * e + 1) & 3], y);
          }
        }
      };
      if (t0 + t >= full0 && t0 + t < full1) sums(std::false_type());
      else sums(std::true_type());
    }
    const float2 a = ptx::add2(ptx::add2(acc[0], acc[1]), ptx::add2(acc[2], acc[3]));
    // (an item's place is written again four items on, when this item's record was given back)
    const uint32_t slot = u % kItemSlots;
    float* other = halves + slot * kPair + g * kTile + row;
    if (half == 1) {
      *other = a.x + a.y;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(c.bar(kHalfSum + g * kItemSlots + (int)slot));
    } else {
      if (!RA_WAIT(kHalfSum + g * kItemSlots + (int)slot, u / kItemSlots, kStatusTimeoutSoftmax)) return;
      const float sum = (a.x + a.y) + *other;
      const bool bad = (notes[2 * slot + g] >> (row / P.piece)) & 1u;
      if (mine) {
        // (a sum of weights is never negative: -1 stands for a key whose page is none)
        if (r->part >= 0) P.parts[(int64_t)r->part * kPair + g * kTile + row] = bad ? -1.f : sum;
        else if (!bad) put(P, r->b, r->head, j, slot0, sum);
      }
    }
    release_record(c, u, lane);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_weigh_chunk_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tkv,
                             const PagedWeighChunkParams P) {
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
  if (threadIdx.x == 0) P.joins[blockIdx.x] = {0, 0, 0, -1};  // nothing to join
  copy_unseen(P);
  paged_sums<kWarps>(P.t.batch, prefix, [&](int b) {
    const PagedSeq q = paged_seq(P.t, b);
    const bool mine = paged_mine(P.t, q, P.group);
    if (mine && q.length > P.weight_width) atomicOr(P.t.status, kPagedStatusRange);
    return warp_total(mine ? (q.length + kPair - 1) / kPair : 0, [&](int i) { return tiles_of(P, q, per_tile, i).n; });
  });
  Shares sh;
  sh.per_head = prefix[P.t.batch];
  sh.all = sh.per_head * P.t.heads_kv;
  sh.count = (int)max((int64_t)1, min((int64_t)gridDim.x, sh.all / kMinUnits));
  if (sh.all == 0 || (int)blockIdx.x >= sh.count) {
    after_previous();  // (every CTA: this kernel's end then tells that the other one's has come)
    return;
  }

  for (uint32_t at = threadIdx.x * 16; at < kStages * kExtra; at += kThreads * 16)
    ptx::st_shared_v4(sbase + S::kOffExtra + at, 0u, 0u, 0u, 0u);
  ptx::fence_proxy_async_smem();
  // Rows that a query tile's box never fills have no weight: they have to be finite.
  if (per_tile * P.group < kTile) {
    for (uint32_t at = threadIdx.x * 16; at < kStages * S::kTileBytes; at += kThreads * 16)
      ptx::st_shared_v4(sbase + S::kOffQ + at, 0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kKeySlots; ++s) ptx::mbar_init(c.bar(kKFull + s), 1), ptx::mbar_init(c.bar(kKEmpty + s), 8);
    for (int s = 0; s < kStages; ++s) ptx::mbar_init(c.bar(kQFull + s), 1), ptx::mbar_init(c.bar(kQEmpty + s), 1);
    for (int g = 0; g < 2; ++g) {
      ptx::mbar_init(c.bar(kSFull + g), 1);
      ptx::mbar_init(c.bar(kSEmpty + g), 8);
      ptx::mbar_init(c.bar(kKReady + g), 8);
    }
    for (int s = 0; s < 2 * kItemSlots; ++s) ptx::mbar_init(c.bar(kHalfSum + s), 4);
    for (int s = 0; s < kItemSlots; ++s) {
      ptx::mbar_init(c.bar(kItemFull + s), 1);
      ptx::mbar_init(c.bar(kItemEmpty + s), kItemConsumers);
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
  if (warp >= 4 && warp < 8) {  // the keys' extra channels
    const uint32_t ones[8] = {0x3f803f80u, 0x3f80u, 0u, 0u, 0u, 0u, 0u, 0u};
    tmem_st8(tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColOnes, ones);
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();

  after_previous();  // (the extra channels)
  ProducerState ps{0u, 0u};
  if (warp < 4) {
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
    const int w = (warp - 4) >> 2;
    run_sums<D>(P, c, sbase, recs, notes, reinterpret_cast<float*>(sgen + S::kOffHalf), tmem, w & 1, w >> 1, warp & 3, per_tile, lane);
  }

  if (warp == 0 && lane == 0 && *c.abort) {  // (every lane of warp 0 holds the same counts)
    // Let this CTA's own TMA loads land before its shared memory goes away.
    for (uint32_t s = 0; s < (uint32_t)kKeySlots; ++s)
      if (ps.k_issued > s) drain_bar(c, c.bar(kKFull + (int)s), ((ps.k_issued - 1 - s) / kKeySlots) & 1u);
    for (uint32_t s = 0; s < (uint32_t)kStages; ++s)
      if (ps.q_issued > s) drain_bar(c, c.bar(kQFull + (int)s), ((ps.q_issued - 1 - s) / kStages) & 1u);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------ extra channels --
// -LSE / scale of every query tile's rows as three bf16 terms; of rows of no token -inf, which
// leaves nothing of their weights at any scale.  A thread has a row; the tiles of the sequences follow each other.
__global__ void __launch_bounds__(kTile) paged_weigh_extra_kernel(const PagedWeighChunkParams P) {
  extern __shared__ int64_t prefix[];
  next_may_come();
  const int per_tile = kTile / P.group;
  for (int b = threadIdx.x; b < P.t.batch; b += kTile) {
    const PagedSeq q = paged_seq(P.t, b);
    prefix[b + 1] = paged_mine(P.t, q, P.group) ? (q.count + per_tile - 1) / per_tile : 0;
  }
  __syncthreads();
  if (threadIdx.x < 32) paged_scan(P.t.batch, prefix);
  __syncthreads();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int b = threadIdx.x; b < P.t.batch; b += kTile) P.extra_at[b] = (int32_t)min(prefix[b], (int64_t)P.tiles - 1);
  const int head = (int)blockIdx.y, row = threadIdx.x, tok = row / P.group;
  const float inv = -1.0f / P.scale;
  // (offsets that fall can make sequences share tokens: no more tiles than there is room for)
  const int tiles = (int)min(prefix[P.t.batch], (int64_t)P.tiles);
  for (int i = (int)blockIdx.x; i < tiles; i += (int)gridDim.x) {
    const int b = paged_find(prefix, P.t.batch, i);
    const PagedSeq q = paged_seq(P.t, b);
    const int token = (i - (int)prefix[b]) * per_tile + tok;
    float x = -INFINITY;
    if (tok < per_tile && token < q.count)
      x = inv * __ldg(P.lse + (int64_t)(q.token0 + token) * P.heads_q + head * P.group + row - tok * P.group);
    const uint32_t hi = ptx::pack_bf16x2(x, 0.f) & 0xffffu;
    const float r1 = x - __uint_as_float(hi << 16);  // (exact; NaN where x is not finite)
    const uint32_t mid = fabsf(r1) <= 3e38f ? ptx::pack_bf16x2(r1, 0.f) & 0xffffu : 0u;
    const float r2 = r1 - __uint_as_float(mid << 16);
    const uint32_t lo = fabsf(r2) <= 3e38f ? ptx::pack_bf16x2(r2, 0.f) & 0xffffu : 0u;
    P.extra[((int64_t)head * P.tiles + i) * kTile + row] = make_uint4(hi | (mid << 16), lo, 0u, 0u);
  }
}

// The item that share x begins and does not end: its first part there, the others at the
// beginning of the shares up to the last.
__global__ void __launch_bounds__(kPair) paged_weigh_join_kernel(const PagedWeighChunkParams P) {
  after_previous();
  const PagedWeighJoin rec = P.joins[blockIdx.x];
  if (rec.last < 0) return;
  const PagedSeq q = paged_seq(P.t, rec.b);
  const int j = rec.key0 + threadIdx.x;
  if (j >= q.length || !seen_by_some(P, q.slot0(), q.count, j)) return;
  float sum = P.parts[(int64_t)(2 * blockIdx.x + 1) * kPair + threadIdx.x];
  if (sum == -1.f) return;
#pragma unroll 4
  for (int s = (int)blockIdx.x + 1; s <= rec.last; ++s) sum += P.parts[(int64_t)(2 * s) * kPair + threadIdx.x];
  put(P, rec.b, rec.head, j, q.slot0(), sum);
}

template <int D>
cudaError_t launch(const PagedWeighChunkParams& prm, int grid, cudaStream_t stream, const char** why) {
  CUtensorMap tq, tkv;
  if (!encode_rows(&tkv, prm.t.cache, (int64_t)prm.t.pages * 2 * prm.t.heads_kv * prm.t.page_rows, D, prm.piece) ||
      !encode_packed(&tq, prm.q, prm.qs, prm.t.tokens, prm.heads_q, D, prm.group, kTile / prm.group)) {
    *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  static std::atomic<int> ready[kMaxDevices];
  constexpr uint32_t kMost = Smem<D>::kFixed + (kMaxChunkSequences + 1) * 8;
  static_assert(kMost <= 232448, "shared memory");
  cudaError_t e = prepare_once(paged_weigh_chunk_kernel<D>, ready, kThreads, 0, (int)kMost, why);
  if (e != cudaSuccess) return e;
  const dim3 extra((unsigned)std::min(prm.tiles, 1024), (unsigned)prm.t.heads_kv);
  paged_weigh_extra_kernel<<<extra, kTile, (prm.t.batch + 1) * 8, stream>>>(prm);
  e = cudaGetLastError();
  if (e != cudaSuccess) {
    *why = "launch failed";
    return e;
  }
  e = launch_behind(paged_weigh_chunk_kernel<D>, dim3((unsigned)grid), kThreads,
                    (size_t)Smem<D>::kFixed + (prm.t.batch + 1) * 8, stream, tq, tkv, prm);
  if (e != cudaSuccess) *why = "launch failed";
  return e;
}

}  // namespace

cudaError_t launch_paged_weigh_join(const PagedWeighChunkParams& prm, int grid, cudaStream_t stream) {
  return launch_behind(paged_weigh_join_kernel, dim3((unsigned)grid), kPair, 0, stream, prm);
}

cudaError_t launch_paged_weigh_chunk(int head_dim, const PagedWeighChunkParams& prm, int grid, cudaStream_t stream,
                                     const char** why) {
  return head_dim == 128 ? launch<128>(prm, grid, stream, why) : launch<64>(prm, grid, stream, why);
}

}  // namespace ra
