// Attention over the paged cache for few query rows per sequence, and in float32 for any.
//
// For the 16 query rows of an item (rows of a key/value head's group and of the new tokens) and
// the cached keys j that they see,
//   m = max_j s_j,  s_j = scale * q.k_j,  l = sum_j e^(s_j - m),  O = sum_j e^(s_j - m) v_j / l,
//   LSE = m + ln l,
// folded block by block of 16 keys with the running maximum and sum.
//
// Bound by HBM: the keys and values are read once for the rows of a group.  bf16 takes the
// warp-level tensor instruction m16n8k16 with the query rows as its 16 rows: for so few rows
// the 5th-generation one would spend its 128 rows on padding, and the products are far from
// the bound.  Each warp takes every fourth block of its CTA's share through a ring of its own
// (cp.async, 16 bytes a lane, rows swizzled for ldmatrix); rows that no query sees arrive as
// zeros, so that what a page holds there does not matter.  The warps' sums are joined in shared
// memory, the parts of an item that several CTAs share by a second kernel, both in a fixed order.
// The weights are rounded to bf16 for the second product, whose operands are bf16; O is divided by
// the sum of the exact ones.  (The chunk kernel, whose running maximum may be stale, corrects that sum by the
// rounding of each tile's largest weight; here the largest weight of a warp's keys is 1
// but for float32's rounding, which bf16 has.)  The exponentials are ex2.approx, off by 2^-22: nothing beside 2^-8.
//
// Measured (32 query and 8 key/value heads, D 128, bf16): one token of 16 sequences up to 32k
// (1.27 GB) 190 us, 6.7 TB/s; one token over 1M 598 us, 7.2 TB/s.  float32 has no such instruction
// to its precision: few rows are bound by the latency of a step of 32 keys, one token of 16
// sequences of 4k (0.32 GB) 78 us, 4.1 TB/s; many by the reads of shared memory, 500 tokens of 16
// heads over 4k 715 us, 22 TFLOP/s (a step's weights handed on by shuffles, not through shared
// memory: 773).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "paged_share.cuh"
#include "sm100_ptx.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;   // blocks of a warp's ring
// Blocks of a share at least: bf16 two a warp (512 tokens of one sequence 13 us, with four 14.5,
// as one item 16.5); float32, whose 32 keys at a time take 3 us, two times that (3 sequences of
// 300 tokens: 41 us with 16 blocks).
template <typename T>
constexpr int kMinUnits = sizeof(T) == 2 ? 8 : 4;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// 16 bytes from global to shared memory, asynchronously; zeros where !live.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
// The same, with an L2 policy.
__device__ __forceinline__ void copy16_hint(uint32_t dst, const void* src, bool live, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// A CTA's walk over its share: items and the units [u0, u1) of each.  Where no item is long and
// there are CTAs for all of them, shares are whole items instead (a unit is an item).
struct Walk {
  int64_t x, x1, all;
  int slots;
  bool whole;
  int b, tile;
  int64_t item_x;  // the item's first unit
  PagedSeq seq;
};
constexpr int kWholeUnits = 16;  // blocks of the longest item in that form
// Where this CTA's share begins; false where it has none.  Every thread of the CTA calls it.
template <typename T>
__device__ __forceinline__ bool walk_begin(const PagedAttendParams& P, int64_t* prefix, Walk& w) {
  __shared__ int longest;
  if (threadIdx.x == 0) longest = 0;
  paged_prefix<kRowsTile, kRowsBlock, kWarps>(P.t, P.group, P.window, P.sinks, prefix);
  w.all = prefix[P.t.batch];
  const int c = (int)blockIdx.x;
  if (w.all == 0) return false;
  // (a sequence of one item, as in a decoding step, is as long as it)
  int most = 0;
  for (int b = threadIdx.x; b < P.t.batch; b += kThreads) most = max(most, (int)min(prefix[b + 1] - prefix[b], (int64_t)1 << 30));
  if (most > 0) atomicMax(&longest, most);
  __syncthreads();
  w.whole = longest <= kWholeUnits && P.t.batch <= P.slots;
  if (w.whole) {
    __syncthreads();  // (all have read the units)
    for (int b = threadIdx.x; b < P.t.batch; b += kThreads) {
      const PagedSeq q = paged_seq(P.t, b);
      prefix[b + 1] = paged_mine(P.t, q, P.group) ? (q.count * P.group + kRowsTile - 1) / kRowsTile : 0;
    }
    __syncthreads();
    if (threadIdx.x < 32) paged_scan(P.t.batch, prefix);
    __syncthreads();
    w.all = prefix[P.t.batch];
    w.slots = (int)min((int64_t)P.slots, w.all);
  } else {
    w.slots = (int)max((int64_t)1, min((int64_t)P.slots, w.all / kMinUnits<T>));
  }
  if (c >= w.slots) return false;
  w.x = w.all * c / w.slots;
  w.x1 = w.all * (c + 1) / w.slots;
  w.b = paged_find(prefix, P.t.batch, w.x);
  w.seq = paged_seq(P.t, w.b);
  if (w.whole) {
    w.tile = (int)(w.x - prefix[w.b]);
    w.item_x = w.x;
  } else {
    w.tile = paged_find_item<kRowsTile, kRowsBlock>(w.seq, P.group, P.window, P.sinks, w.x - prefix[w.b], w.item_x);
    w.item_x += prefix[w.b];
  }
  return true;
}
// To the item at x (the share's current item is done).
__device__ __forceinline__ void walk_next(const PagedAttendParams& P, const int64_t* prefix, Walk& w) {
  w.item_x = w.x;
  ++w.tile;
  if (w.x < prefix[w.b + 1]) return;
  while (w.b + 1 < P.t.batch && prefix[w.b + 1] <= w.x) ++w.b;
  w.seq = paged_seq(P.t, w.b);
  w.tile = 0;
}

// The part of an item that is cut: its sums in scratch, and, where it begins, how to join it.
__device__ __forceinline__ int64_t part_at(const PagedAttendParams& P, const Walk& w, const PagedItem& it, int u0, int n) {
  const int64_t me = (int64_t)blockIdx.y * P.slots + blockIdx.x;
  if (u0 > 0) return me * 2;
  if (threadIdx.x == 0) {
    const int last = (int)(((w.item_x + n) * w.slots - 1) / w.all);
    P.joins[me] = make_int4(w.seq.token0 * P.group + it.row0, it.rows, last, 0);
  }
  return me * 2 + 1;
}

// Where this kernel runs beside a chunk kernel: its end, that of one CTA of it, has to come after
// the other's, so that what waits for this one finds both done.
__device__ __forceinline__ void end_after_others(const PagedAttendParams& P) {
  if (P.beside && blockIdx.x == 0 && blockIdx.y == 0) after_previous();
}

// Where row `row` (over the tokens' groups) of this head lies.
template <typename T>
__device__ __forceinline__ T* row_of(const PagedStrides& s, const void* base, int group, int head, int row) {
  const int token = row / group;
  return static_cast<T*>(const_cast<void*>(base)) + token * s.token + (int64_t)(head * group + row - token * group) * s.head;
}

// ------------------------------------------------------------------------ bf16 --
template <int D>
struct Bf16 {
  static constexpr int kRowBytes = D * 2;
  static constexpr int kChunks = D / 8;  // of 16 bytes in a row
  static constexpr int kBlockBytes = kRowsBlock * kRowBytes;
  static constexpr int kRing = kWarps * kStages * 2 * kBlockBytes;
  static constexpr int kJoinRow = D + 4;  // floats
  static_assert(kWarps * kRowsTile * (kJoinRow + 2) * 4 <= kRing, "the warps' sums lie in the ring");
};

template <int D>
__global__ void __launch_bounds__(kThreads) rows_bf16_kernel(const PagedAttendParams P) {
  using G = Bf16<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  int64_t* prefix = reinterpret_cast<int64_t*>(smem + G::kRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, head = (int)blockIdx.y;
  next_may_come();
  if (P.joins != nullptr && threadIdx.x == 0) P.joins[(int64_t)head * P.slots + blockIdx.x] = make_int4(0, 0, 0, 0);
  Walk w;
  if (!walk_begin<__nv_bfloat16>(P, prefix, w)) return end_after_others(P);

  const uint32_t ring = ptx::smem_addr(smem) + warp * kStages * 2 * G::kBlockBytes;
  const uint8_t* lane_src = static_cast<const uint8_t*>(P.t.cache) + lane / G::kChunks * G::kRowBytes + lane % G::kChunks * 16;
  const int64_t to_v = (int64_t)P.t.heads_kv * P.t.page_rows * G::kRowBytes;  // from a key's row to its value's
  const uint64_t once = ptx::l2_policy_evict_first();  // (a chunk kernel beside this one keeps its keys in the L2)
  const int quad = lane >> 2, two = (lane & 3) * 2;
  float* sums = reinterpret_cast<float*>(smem);
  float2* stats = reinterpret_cast<float2*>(sums + kWarps * kRowsTile * G::kJoinRow);

  for (;; walk_next(P, prefix, w)) {
    const PagedItem it = paged_item<kRowsTile>(w.seq, P.group, w.tile);
    const PagedSpan span = paged_span(P.window, P.sinks, it.s0, it.s1);
    const PagedBlocks<kRowsBlock> blocks(span);
    const int n = max(1, blocks.n);
    const int u0 = w.whole ? 0 : (int)(w.x - w.item_x), u1 = w.whole ? n : (int)min((int64_t)n, w.x1 - w.item_x);
    const int n_live = min(u1, blocks.n);
    const int mine = n_live > u0 + warp ? (n_live - u0 - warp + kWarps - 1) / kWarps : 0;  // blocks of this warp

    // The rows as the first operand: rows quad and quad + 8, channels two.. and two + 8..
    RA_BOUNDS(P.t.status, it.row0 >= 0 && it.rows > 0 && w.seq.token0 + w.seq.count <= P.t.tokens && u0 >= 0 && u0 < u1 && u1 <= n, 116);
    const int row_a = w.seq.token0 * P.group + it.row0 + quad;
    uint32_t q[D / 16][4];
    int slot[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool live = quad + 8 * i < it.rows;
      slot[i] = live ? w.seq.slot0() + (it.row0 + quad + 8 * i) / P.group : -1;
      const __nv_bfloat16* src = live ? row_of<const __nv_bfloat16>(P.qs, P.q, P.group, head, row_a + 8 * i) : nullptr;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          q[kk][i + 2 * e] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16 + e * 8 + two)) : 0u;
    }
    float o[D / 8][4];
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    // Block i of this warp into its ring, and its first slot.  A lane knows one of the next 32
    // blocks: what it takes to find them is done once for all.
    int known_j = 0, known_row = -1;  // first slot; row of the cache (-1: the page is none)
    bool known_full = false;          // some token sees every slot of the block
    uint32_t bad = 0u;                // stages whose page is none
    auto load = [&](int i) {
      if ((i & 31) == 0 && i < mine) {
        const int k = u0 + warp + (i + lane) * kWarps;
        known_row = -1;
        if (i + lane < mine) {
          known_j = blocks.at(k) * kRowsBlock;
          const int page = paged_page(P.t, w.b, known_j / P.t.page_rows);
          if (page >= 0) known_row = (int)paged_row(P.t, page, 0, head, known_j % P.t.page_rows);
          known_full = page >= 0 && ((known_j >= span.lo && known_j + kRowsBlock <= span.hi) || known_j + kRowsBlock <= span.sink);
        }
      }
      const int j0 = __shfl_sync(0xffffffffu, known_j, i & 31);
      if (i < mine) {
        const int row0 = __shfl_sync(0xffffffffu, known_row, i & 31), s = i % kStages;
        const bool full = __shfl_sync(0xffffffffu, known_full, i & 31);
        bad = row0 < 0 ? bad | (1u << s) : bad & ~(1u << s);
        RA_BOUNDS(P.t.status, row0 >= -1 && row0 + kRowsBlock <= (int64_t)P.t.pages * 2 * P.t.heads_kv * P.t.page_rows, 111);
        const uint8_t* src = lane_src + (int64_t)max(row0, 0) * G::kRowBytes;
        const uint32_t dst = ring + s * 2 * G::kBlockBytes;
        auto copies = [&](auto whole) {
#pragma unroll
          for (int x = 0; x < G::kChunks / 2; ++x) {
            constexpr int kStep = 32 / G::kChunks;  // rows
            const int r = x * kStep + lane / G::kChunks, ch = lane % G::kChunks;
            const bool live = decltype(whole)::value || (row0 >= 0 && span.holds(j0 + r));
            const uint32_t to = dst + r * G::kRowBytes + ((ch ^ (r & 7)) * 16);
            copy16_hint(to, src + x * kStep * G::kRowBytes, live, once);
            copy16_hint(to + G::kBlockBytes, src + to_v + x * kStep * G::kRowBytes, live, once);
          }
        };
        if (full) copies(std::true_type());
        else copies(std::false_type());
      }
      copies_commit();
      return j0;
    };
    int ahead[kStages - 1];  // first slots of the blocks under way
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) ahead[i] = load(i);
    for (int i = 0; i < mine; ++i) {
      copies_wait<kStages - 2>();
      __syncwarp();
      const int j0 = ahead[0];
#pragma unroll
      for (int e = 0; e + 1 < kStages - 1; ++e) ahead[e] = ahead[e + 1];
      ahead[kStages - 2] = load(i + kStages - 1);
      const int st = i % kStages;
      const uint32_t kb = ring + st * 2 * G::kBlockBytes, vb = kb + G::kBlockBytes;
      // Scores: rows x 16 keys, as two products of 8 keys.
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const int kr = (lane & 7) + ((lane >> 4) << 3);  // key of this lane's address; its half of 16 channels:
      const int kc = (lane >> 3) & 1;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t r[4];
        ldmatrix4(r, kb + kr * G::kRowBytes + (((2 * kk + kc) ^ (kr & 7)) * 16));
        mma16816(s[0], q[kk], r[0], r[1]);
        mma16816(s[1], q[kk], r[2], r[3]);
      }
      // Blocks that every row sees whole need no mask.
      const bool whole = !((bad >> st) & 1u) && j0 + kRowsBlock - 1 <= it.s0 &&
                         (P.window == 0 || j0 > it.s1 - P.window || j0 + kRowsBlock <= P.sinks);
      if (!whole) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (((bad >> st) & 1u) || !paged_sees(P.window, P.sinks, slot[e >> 1], j0 + c * 8 + two + (e & 1)))
              s[c][e] = -INFINITY;
      }
      uint32_t p[4];
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2) {  // rows quad, quad + 8
        float mx = fmaxf(fmaxf(s[0][2 * i2], s[0][2 * i2 + 1]), fmaxf(s[1][2 * i2], s[1][2 * i2 + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float m_new = fmaxf(m[i2], mx * P.scale_log2);
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = ptx::ex2_approx(m[i2] - ref);  // (0 from -inf)
        m[i2] = m_new;
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float a = ptx::ex2_approx(fmaf(s[c][2 * i2], P.scale_log2, -ref));
          const float e = ptx::ex2_approx(fmaf(s[c][2 * i2 + 1], P.scale_log2, -ref));
          sum += a + e;
          p[i2 + 2 * c] = ptx::pack_bf16x2(a, e);
        }
        l[i2] = l[i2] * alpha + sum;
        if (__any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            o[c][2 * i2] *= alpha;
            o[c][2 * i2 + 1] *= alpha;
          }
        }
      }
      // O += P V: 16 keys x 8 channels at a time.
      const int vr = (lane & 7) + (((lane >> 3) & 1) << 3), vc = lane >> 4;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        uint32_t r[4];
        ldmatrix4t(r, vb + vr * G::kRowBytes + (((2 * c + vc) ^ (vr & 7)) * 16));
        mma16816(o[2 * c], p, r[0], r[1]);
        mma16816(o[2 * c + 1], p, r[2], r[3]);
      }
      __syncwarp();
    }
    copies_wait<0>();
    __syncthreads();  // every warp is done with its ring

    // The warps' sums side by side, then joined.
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if ((lane & 3) == 0) stats[warp * kRowsTile + quad + 8 * i] = make_float2(m[i], l[i]);
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        *reinterpret_cast<float2*>(sums + (warp * kRowsTile + quad + 8 * i) * G::kJoinRow + c * 8 + two) =
            make_float2(o[c][2 * i], o[c][2 * i + 1]);
    }
    __syncthreads();
    const bool cut = u0 > 0 || u1 < n;
    const int64_t part = cut ? part_at(P, w, it, u0, n) : 0;
    for (int id = threadIdx.x; id < kRowsTile * G::kChunks; id += kThreads) {
      const int r = id / G::kChunks, ch = id % G::kChunks;
      float mr = -INFINITY, lr = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < kWarps; ++v) mr = fmaxf(mr, stats[v * kRowsTile + r].x);
      const float ref = mr == -INFINITY ? 0.f : mr;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float2 ml = stats[v * kRowsTile + r];
        const float f = ptx::ex2_approx(ml.x - ref);
        lr += ml.y * f;
        const float4* src = reinterpret_cast<const float4*>(sums + (v * kRowsTile + r) * G::kJoinRow + ch * 8);
        const float4 a = src[0], e = src[1];
        x[0] += a.x * f, x[1] += a.y * f, x[2] += a.z * f, x[3] += a.w * f;
        x[4] += e.x * f, x[5] += e.y * f, x[6] += e.z * f, x[7] += e.w * f;
      }
      if (cut) {
        float4* dst = reinterpret_cast<float4*>(P.part_o + (part * kRowsTile + r) * D + ch * 8);
        dst[0] = make_float4(x[0], x[1], x[2], x[3]);
        dst[1] = make_float4(x[4], x[5], x[6], x[7]);
        if (ch == 0) P.part_ml[part * kRowsTile + r] = make_float2(mr, lr);
      } else if (r < it.rows) {
        const int row = w.seq.token0 * P.group + it.row0 + r;
        const float inv = lr > 0.f ? 1.0f / lr : (lr == 0.f ? 0.f : lr);
        __nv_bfloat16* dst = row_of<__nv_bfloat16>(P.os, P.o, P.group, head, row) + ch * 8;
        uint4 y;
        y.x = ptx::pack_bf16x2(x[0] * inv, x[1] * inv);
        y.y = ptx::pack_bf16x2(x[2] * inv, x[3] * inv);
        y.z = ptx::pack_bf16x2(x[4] * inv, x[5] * inv);
        y.w = ptx::pack_bf16x2(x[6] * inv, x[7] * inv);
        *reinterpret_cast<uint4*>(dst) = y;
        if (ch == 0 && P.lse != nullptr) {
          const int token = row / P.group;
          P.lse[(int64_t)token * P.heads_q + head * P.group + row - token * P.group] =
              lr == 0.f ? -INFINITY : (mr + log2f(lr)) * kLn2;
        }
      }
    }
    __syncthreads();  // the ring is free for the next item
    w.x = w.item_x + (w.whole ? 1 : u1);
    if (w.x >= w.x1) return end_after_others(P);
  }
}

// --------------------------------------------------------------------- float32 --
// A CTA meets 32 keys (two blocks) at a time.  Items of more than 4 rows: a warp has 4 of the 16
// rows, a lane scores one key against them, and then holds D / 32 channels of their outputs.  Items
// of up to 4 (a token of a group of 4): a warp has 8 of the keys and all rows, 4 lanes share a key,
// and the warps' sums are joined at the end; with the other form, three warps without rows, one
// token of 16 sequences of 4k took 149 us, of 64k 230 (now 118).  Which slot and row of the
// cache a step's keys are is read two steps ahead (3 sequences of 300 tokens: 27 -> 23 us).
template <int D>
struct F32 {
  static constexpr int kRow = D + 4;  // floats; 8 lanes' 16-byte reads of a column fall into different banks
  static constexpr int kKeys = 2 * kRowsBlock;
  static constexpr int kStage = 2 * kKeys * kRow * 4;
  static constexpr int kQ = kRowsTile * D * 4;
  static constexpr int kP = kWarps * kKeys * 16;  // a step's weights of 4 rows
  static constexpr int kBytes = 2 * kStage + kQ + kP;
};
// D / 32 channels that follow each other.
__device__ __forceinline__ void load_channels(float (&x)[4], const float* p) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load_channels(float (&x)[2], const float* p) {
  const float2 v = *reinterpret_cast<const float2*>(p);
  x[0] = v.x, x[1] = v.y;
}
__device__ __forceinline__ void store_channels(float* p, const float (&x)[4], float f) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
}
__device__ __forceinline__ void store_channels(float* p, const float (&x)[2], float f) {
  *reinterpret_cast<float2*>(p) = make_float2(x[0] * f, x[1] * f);
}

template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 4 : 2) rows_f32_kernel(const PagedAttendParams P) {
  using G = F32<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  float* qs = reinterpret_cast<float*>(smem + 2 * G::kStage);
  int64_t* prefix = reinterpret_cast<int64_t*>(smem + G::kBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, head = (int)blockIdx.y;
  float4* ps = reinterpret_cast<float4*>(smem + 2 * G::kStage + G::kQ) + warp * G::kKeys;  // of this warp's keys
  next_may_come();
  if (P.joins != nullptr && threadIdx.x == 0) P.joins[(int64_t)head * P.slots + blockIdx.x] = make_int4(0, 0, 0, 0);
  Walk w;
  if (!walk_begin<float>(P, prefix, w)) return;
  const float* cache = static_cast<const float*>(P.t.cache);
  constexpr int kPer = kRowsTile / kWarps, kCh = D / 32, kFew = 4;
  static_assert(kPer == 4 && kFew == kWarps && kWarps * 8 == G::kKeys, "4 rows a float4; a warp for 8 keys, and for a row in the end");

  for (;; walk_next(P, prefix, w)) {
    const PagedItem it = paged_item<kRowsTile>(w.seq, P.group, w.tile);
    const PagedSpan span = paged_span(P.window, P.sinks, it.s0, it.s1);
    const PagedBlocks<kRowsBlock> blocks(span);
    const int n = max(1, blocks.n);
    const int u0 = w.whole ? 0 : (int)(w.x - w.item_x), u1 = w.whole ? n : (int)min((int64_t)n, w.x1 - w.item_x);
    const int n_live = min(u1, blocks.n);
    const int steps = n_live > u0 ? (n_live - u0 + 1) / 2 : 0;
    RA_BOUNDS(P.t.status, it.row0 >= 0 && it.rows > 0 && w.seq.token0 + w.seq.count <= P.t.tokens && u0 >= 0 && u0 < u1 && u1 <= n, 117);
    const int row0 = w.seq.token0 * P.group + it.row0;
    for (int id = threadIdx.x; id < kRowsTile * (D / 4); id += kThreads) {
      const int r = id / (D / 4), ch = id % (D / 4);
      reinterpret_cast<float4*>(qs)[id] = r < it.rows
          ? __ldg(reinterpret_cast<const float4*>(row_of<const float>(P.qs, P.q, P.group, head, row0 + r)) + ch)
          : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // Slot and row of the cache of this lane's key of a step; row -1: past the share's end, a slot
    // that no token sees, or a page that is none.  Read a step ahead.
    auto find = [&](int step, int& j, int& row) {
      const int k = u0 + 2 * step + (lane >> 4);
      j = k < n_live ? blocks.at(k) * kRowsBlock + (lane & 15) : 0;
      row = -1;
      if (k < n_live && span.holds(j)) {
        const int page = paged_page(P.t, w.b, j / P.t.page_rows);
        if (page >= 0) row = (int)paged_row(P.t, page, 0, head, j % P.t.page_rows);
      }
      RA_BOUNDS(P.t.status, row >= -1 && row < (int64_t)P.t.pages * 2 * P.t.heads_kv * P.t.page_rows, 125);
    };
    auto load = [&](int step, int row) {
      if (step < steps) {
        const uint32_t dst = ptx::smem_addr(smem + (step & 1) * G::kStage);
        constexpr int kCh4 = D / 4;  // 16-byte pieces of a row
#pragma unroll
        for (int x = 0; x < G::kKeys * kCh4 / kThreads; ++x) {
          const int id = threadIdx.x + x * kThreads, i = id / kCh4, ch = id % kCh4;
          const int from = __shfl_sync(0xffffffffu, row, i);
          const float* src = cache + (int64_t)max(from, 0) * D + ch * 4;
          const uint32_t to = dst + (i * G::kRow + ch * 4) * 4;
          copy16(to, src, from >= 0);
          copy16(to + G::kKeys * G::kRow * 4, src + (int64_t)P.t.heads_kv * P.t.page_rows * D, from >= 0);
        }
      }
      copies_commit();
    };
    int j, row, j_next, row_next;
    find(0, j, row);
    load(0, row);
    find(1, j_next, row_next);
    const bool cut = u0 > 0 || u1 < n;
    const int64_t part = cut ? part_at(P, w, it, u0, n) : 0;
    // Row `at` of the item, of which this lane has kCh channels.
    auto put = [&](int at, float m, float l, const float (&acc)[kCh]) {
      if (cut) {
        store_channels(P.part_o + (part * kRowsTile + at) * D + lane * kCh, acc, 1.0f);
        if (lane == 0) P.part_ml[part * kRowsTile + at] = make_float2(m, l);
      } else if (at < it.rows) {
        const int row = row0 + at;
        const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);
        store_channels(row_of<float>(P.os, P.o, P.group, head, row) + lane * kCh, acc, inv);
        if (lane == 0 && P.lse != nullptr) {
          const int token = row / P.group;
          P.lse[(int64_t)token * P.heads_q + head * P.group + row - token * P.group] =
              l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
      }
    };
    if (it.rows <= kFew) {
      int order = lane >> 2;  // keys 4 apart beside each other: 4 lanes' pieces of them fall into different banks
      order = (order >> 1) + 4 * (order & 1);
      const int key = warp * 8 + order, r = lane & 3, slot = r < it.rows ? w.seq.slot0() + (it.row0 + r) / P.group : -1;
      float m = -INFINITY, l = 0.f, acc[kFew][kCh];  // m, l: of row r
#pragma unroll
      for (int e = 0; e < kFew; ++e)
#pragma unroll
        for (int c = 0; c < kCh; ++c) acc[e][c] = 0.f;
      for (int step = 0; step < steps; ++step) {
        load(step + 1, row_next);
        int j_after, row_after;
        find(step + 2, j_after, row_after);
        copies_wait<1>();
        __syncthreads();
        const float* ks = reinterpret_cast<const float*>(smem + (step & 1) * G::kStage);
        const float* vs = ks + G::kKeys * G::kRow;
        float s[kFew] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {  // a fourth of the channels each
          const float4 k4 = *reinterpret_cast<const float4*>(ks + key * G::kRow + c * 16 + r * 4);
#pragma unroll
          for (int e = 0; e < kFew; ++e) {
            const float4 q4 = *reinterpret_cast<const float4*>(qs + e * D + c * 16 + r * 4);
            s[e] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, s[e]))));
          }
        }
#pragma unroll
        for (int e = 0; e < kFew; ++e) {
          s[e] += __shfl_xor_sync(0xffffffffu, s[e], 1);
          s[e] += __shfl_xor_sync(0xffffffffu, s[e], 2);
        }
        const int j_key = __shfl_sync(0xffffffffu, j, key), row_key = __shfl_sync(0xffffffffu, row, key);
        const float own = r < 2 ? (r == 0 ? s[0] : s[1]) : (r == 2 ? s[2] : s[3]);
        const float x = row_key >= 0 && paged_sees(P.window, P.sinks, slot, j_key) ? own : -INFINITY;
        float mx = x;
#pragma unroll
        for (int o = 16; o > 2; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float m_new = fmaxf(m, mx * P.scale_log2);
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = exp2f(m - ref), p = exp2f(fmaf(x, P.scale_log2, -ref));
        m = m_new;
        l = l * alpha + p;
        if (__any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll
          for (int e = 0; e < kFew; ++e) {
            const float f = __shfl_sync(0xffffffffu, alpha, e);
#pragma unroll
            for (int c = 0; c < kCh; ++c) acc[e][c] *= f;
          }
        }
        reinterpret_cast<float*>(ps)[order * 4 + r] = p;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v[kCh];
          load_channels(v, vs + (warp * 8 + i) * G::kRow + lane * kCh);
          const float4 p4 = ps[i];
#pragma unroll
          for (int c = 0; c < kCh; ++c) {
            acc[0][c] = fmaf(p4.x, v[c], acc[0][c]);
            acc[1][c] = fmaf(p4.y, v[c], acc[1][c]);
            acc[2][c] = fmaf(p4.z, v[c], acc[2][c]);
            acc[3][c] = fmaf(p4.w, v[c], acc[3][c]);
          }
        }
        j = j_next, row = row_next;
        j_next = j_after, row_next = row_after;
        __syncthreads();
      }
      copies_wait<0>();
      // The warps' sums side by side, then a row each joined by a warp.
      float* sums = reinterpret_cast<float*>(smem);
      float2* stats = reinterpret_cast<float2*>(sums + kWarps * kFew * D);
#pragma unroll
      for (int o = 16; o > 2; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      __syncthreads();
      if (lane < kFew) stats[warp * kFew + lane] = make_float2(m, l);
#pragma unroll
      for (int e = 0; e < kFew; ++e) store_channels(sums + (warp * kFew + e) * D + lane * kCh, acc[e], 1.0f);
      __syncthreads();
      float top = -INFINITY, all = 0.f, out[kCh] = {};
#pragma unroll
      for (int v = 0; v < kWarps; ++v) top = fmaxf(top, stats[v * kFew + warp].x);
      const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float2 ml = stats[v * kFew + warp];
        const float f = exp2f(ml.x - base);
        all = fmaf(ml.y, f, all);
        float x[kCh];
        load_channels(x, sums + (v * kFew + warp) * D + lane * kCh);
#pragma unroll
        for (int c = 0; c < kCh; ++c) out[c] = fmaf(x[c], f, out[c]);
      }
      put(warp, top, all, out);
    } else {
      int slot[kPer];
      float m[kPer], l[kPer], acc[kPer][kCh];
#pragma unroll
      for (int r = 0; r < kPer; ++r) {
        const int own = warp * kPer + r;
        slot[r] = own < it.rows ? w.seq.slot0() + (it.row0 + own) / P.group : -1;
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < kCh; ++c) acc[r][c] = 0.f;
      }
      for (int step = 0; step < steps; ++step) {
        load(step + 1, row_next);
        int j_after, row_after;
        find(step + 2, j_after, row_after);
        copies_wait<1>();
        __syncthreads();
        const float* ks = reinterpret_cast<const float*>(smem + (step & 1) * G::kStage);
        const float* vs = ks + G::kKeys * G::kRow;
        float s[kPer];
#pragma unroll
        for (int r = 0; r < kPer; ++r) s[r] = 0.f;
#pragma unroll 8
        for (int c = 0; c < D / 4; ++c) {
          const float4 k4 = *reinterpret_cast<const float4*>(ks + lane * G::kRow + c * 4);
#pragma unroll
          for (int r = 0; r < kPer; ++r) {
            const float4 q4 = *reinterpret_cast<const float4*>(qs + (warp * kPer + r) * D + c * 4);
            s[r] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, s[r]))));
          }
        }
        float p[kPer];
#pragma unroll
        for (int r = 0; r < kPer; ++r) {
          const float x = row >= 0 && paged_sees(P.window, P.sinks, slot[r], j) ? s[r] : -INFINITY;
          float mx = x;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const float m_new = fmaxf(m[r], mx * P.scale_log2);
          const float ref = m_new == -INFINITY ? 0.f : m_new;
          const float alpha = exp2f(m[r] - ref);
          m[r] = m_new;
          p[r] = exp2f(fmaf(x, P.scale_log2, -ref));
          l[r] = l[r] * alpha + p[r];
#pragma unroll
          for (int c = 0; c < kCh; ++c) acc[r][c] *= alpha;
        }
        ps[lane] = make_float4(p[0], p[1], p[2], p[3]);
        __syncwarp();
#pragma unroll 8
        for (int i = 0; i < G::kKeys; ++i) {
          float v[kCh];
          load_channels(v, vs + i * G::kRow + lane * kCh);
          const float4 p4 = ps[i];
#pragma unroll
          for (int c = 0; c < kCh; ++c) {
            acc[0][c] = fmaf(p4.x, v[c], acc[0][c]);
            acc[1][c] = fmaf(p4.y, v[c], acc[1][c]);
            acc[2][c] = fmaf(p4.z, v[c], acc[2][c]);
            acc[3][c] = fmaf(p4.w, v[c], acc[3][c]);
          }
        }
        j = j_next, row = row_next;
        j_next = j_after, row_next = row_after;
        __syncthreads();
      }
#pragma unroll
      for (int r = 0; r < kPer; ++r) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
        put(warp * kPer + r, m[r], l[r], acc[r]);
      }
    }
    __syncthreads();
    w.x = w.item_x + (w.whole ? 1 : u1);
    if (w.x >= w.x1) return;
  }
}

// ---------------------------------------------------------------- cut items --
// The item that slot x's share begins and does not end: its first part there, the others at the
// beginning of the slots up to the last.  A row has kJoinSplit warps, each of which folds its parts,
// every kJoinSplit-th, with the running maximum, 8 at a time; the warps' sums are added in order.
constexpr int kJoinParts = 8, kJoinThreads = 512;
template <typename T, int D, int kJoinSplit>
__global__ void __launch_bounds__(kJoinThreads) rows_join_kernel(const PagedAttendParams P) {
  constexpr int kJoinRows = kJoinThreads / 32 / kJoinSplit;  // of a CTA
  __shared__ float4 sums[kJoinRows * kJoinSplit][D / 4];
  __shared__ float2 stats[kJoinRows * kJoinSplit];
  const int head = (int)blockIdx.y;
  const int64_t me = (int64_t)head * P.slots + blockIdx.x;
  after_previous();
  const int4 rec = P.joins[me];
  if (rec.y <= (int)blockIdx.z * kJoinRows) return;
  const int count = rec.z - (int)blockIdx.x + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ch = lane % (D / 4);
  const int r = (int)blockIdx.z * kJoinRows + warp / kJoinSplit, first = warp % kJoinSplit;
  auto part = [&](int i) { return (i == 0 ? me * 2 + 1 : (me + i) * 2) * kRowsTile + r; };
  float m = -INFINITY, l = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r < rec.y) {
    for (int i0 = first; i0 < count; i0 += kJoinSplit * kJoinParts) {
      float2 ml[kJoinParts];
      float4 y[kJoinParts];
#pragma unroll
      for (int e = 0; e < kJoinParts; ++e) {
        const int i = i0 + e * kJoinSplit;
        ml[e] = make_float2(-INFINITY, 0.f);
        y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < count) {
          ml[e] = P.part_ml[part(i)];
          y[e] = *reinterpret_cast<const float4*>(P.part_o + part(i) * D + ch * 4);
        }
      }
      float top = m;
#pragma unroll
      for (int e = 0; e < kJoinParts; ++e) top = fmaxf(top, ml[e].x);
      const float ref = top == -INFINITY ? 0.f : top, alpha = exp2f(m - ref);
      m = top;
      l *= alpha;
      x.x *= alpha, x.y *= alpha, x.z *= alpha, x.w *= alpha;
#pragma unroll
      for (int e = 0; e < kJoinParts; ++e) {
        const float f = exp2f(ml[e].x - ref);
        l = fmaf(ml[e].y, f, l);
        x.x = fmaf(y[e].x, f, x.x), x.y = fmaf(y[e].y, f, x.y), x.z = fmaf(y[e].z, f, x.z), x.w = fmaf(y[e].w, f, x.w);
      }
    }
  }
  if (lane < D / 4) sums[warp][ch] = x;
  if (lane == 0) stats[warp] = make_float2(m, l);
  __syncthreads();
  if (first != 0 || r >= rec.y || lane >= D / 4) return;
  m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < kJoinSplit; ++e) m = fmaxf(m, stats[warp + e].x);
  const float ref = m == -INFINITY ? 0.f : m;
  x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int e = 0; e < kJoinSplit; ++e) {
    const float f = exp2f(stats[warp + e].x - ref);
    const float4 y = sums[warp + e][ch];
    l = fmaf(stats[warp + e].y, f, l);
    x.x = fmaf(y.x, f, x.x), x.y = fmaf(y.y, f, x.y), x.z = fmaf(y.z, f, x.z), x.w = fmaf(y.w, f, x.w);
  }
  const int row = rec.x + r;
  const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);
  T* dst = row_of<T>(P.os, P.o, P.group, head, row) + ch * 4;
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(ptx::pack_bf16x2(x.x * inv, x.y * inv), ptx::pack_bf16x2(x.z * inv, x.w * inv));
  } else {
    *reinterpret_cast<float4*>(dst) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
  }
  if (ch == 0 && P.lse != nullptr) {
    const int token = row / P.group;
    P.lse[(int64_t)token * P.heads_q + head * P.group + row - token * P.group] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

template <typename Kernel>
cudaError_t raise_smem(Kernel kernel, std::atomic<int>* ready, int bytes) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool cached = dev >= 0 && dev < kMaxDevices;
  if (cached && ready[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && cached) ready[dev].store(1, std::memory_order_release);
  return e;
}

template <typename T, int D>
cudaError_t launch(const PagedAttendParams& prm, bool beside, cudaStream_t stream) {
  const dim3 grid((unsigned)prm.slots, (unsigned)prm.t.heads_kv);
  const int prefix = (prm.t.batch + 1) * 8, most = (kMaxSequences + 1) * 8;
  static std::atomic<int> ready[kMaxDevices];
  if constexpr (sizeof(T) == 2) {
    const cudaError_t e = raise_smem(rows_bf16_kernel<D>, ready, Bf16<D>::kRing + most);
    if (e != cudaSuccess) return e;
    if (beside) return launch_behind(rows_bf16_kernel<D>, grid, kThreads, Bf16<D>::kRing + prefix, stream, prm);
    rows_bf16_kernel<D><<<grid, kThreads, Bf16<D>::kRing + prefix, stream>>>(prm);
  } else {
    const cudaError_t e = raise_smem(rows_f32_kernel<D>, ready, F32<D>::kBytes + most);
    if (e != cudaSuccess) return e;
    rows_f32_kernel<D><<<grid, kThreads, F32<D>::kBytes + prefix, stream>>>(prm);
  }
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t launch_join(const PagedAttendParams& prm, cudaStream_t stream) {
  if (prm.slots == 1) return cudaSuccess;
  // Of many shares a head an item may be cut into as many parts: one token over 60k of one head, 304
  // parts, 27 us, with a warp a row 50.  With few shares more CTAs only cost their start: one of 512
  // tokens and 31 single ones 195 us, with a warp a row 189.
  const dim3 grid((unsigned)prm.slots, (unsigned)prm.t.heads_kv);
  if (prm.slots <= 128) return launch_behind(rows_join_kernel<T, D, 1>, grid, kJoinThreads, 0, stream, prm);
  return launch_behind(rows_join_kernel<T, D, 4>, dim3(grid.x, grid.y, 4), kJoinThreads, 0, stream, prm);
}

}  // namespace

cudaError_t launch_paged_rows(int dtype, int head_dim, const PagedAttendParams& prm, bool beside, cudaStream_t stream) {
  if (dtype == RA_DTYPE_BF16)
    return head_dim == 128 ? launch<__nv_bfloat16, 128>(prm, beside, stream) : launch<__nv_bfloat16, 64>(prm, beside, stream);
  return head_dim == 128 ? launch<float, 128>(prm, beside, stream) : launch<float, 64>(prm, beside, stream);
}

cudaError_t launch_paged_rows_join(int dtype, int head_dim, const PagedAttendParams& prm, cudaStream_t stream) {
  if (dtype == RA_DTYPE_BF16)
    return head_dim == 128 ? launch_join<__nv_bfloat16, 128>(prm, stream) : launch_join<__nv_bfloat16, 64>(prm, stream);
  return head_dim == 128 ? launch_join<float, 128>(prm, stream) : launch_join<float, 64>(prm, stream);
}

}  // namespace ra
