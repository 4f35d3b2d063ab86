// The attention weight that cached keys receive from a packed batch of new tokens
// (include/ra.h, ra_paged_weigh): for every slot j of a sequence and key/value head,
//   weight_j = (weight_in_j, of slots before the call's tokens) + sum_i e^(scale * q_i.k_j - LSE_i)
// over the query rows i of the head's group that see j.  Given the rows' LSE no softmax is
// left: the sums run down the columns, each column belongs to one warp, and no order varies.
//
// Bound by HBM for few rows: the keys are read once.  bf16: the blocks of 16 keys of all
// sequences are laid in a row and shared out among the warps in equal runs; a warp streams its
// run through a ring of its own (cp.async, 16 bytes a lane) and scores the keys against 16 query
// rows at a time by m16n8k16, the rows of a sequence of up to 16 staying in registers.
// float32: keys in shared memory, a lane one of them, 16 query rows at a time; bound by the reads
// of shared memory (5 for 16 products of 4 channels).
//
// Measured (32 query and 8 key/value heads, D 128): one token of 16 sequences up to 8k (163 MB of
// keys) 35 us, with a CTA a chunk of keys and no ring 93; one token over 1M 334 us, 6.4 TB/s;
// float32, one token of 16 sequences of 4k (0.16 GB) 55 us, 500 tokens over 4k 380.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "paged_share.cuh"
#include "sm100_ptx.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kKeys = 32;  // float32: a lane each
constexpr float kLog2e = 1.4426950408889634f;

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
// 16 or 4 bytes from global to shared memory, asynchronously; zeros where !live.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Sums of the sequences' blocks of kB slots (as paged_prefix, of lengths).
template <int kB>
__device__ void slot_prefix(const PagedTable& t, int group, int64_t* prefix) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    int64_t before = 0;
    for (int b0 = 0; b0 < t.batch; b0 += 32) {
      int64_t x = 0;
      if (b0 + lane < t.batch) {
        const PagedSeq q = paged_seq(t, b0 + lane);
        if (paged_mine(t, q, group)) x = (q.length + kB - 1) / kB;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b0 + lane < t.batch) prefix[b0 + lane + 1] = before + x;
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) prefix[0] = 0;
  }
  __syncthreads();
}

// What both kernels know of a sequence for one head.
template <typename T>
struct Rows {
  const PagedWeighParams& P;
  PagedSeq seq;
  int head;
  // Tiles of 16 rows that see one of the slots [j0, j0 + n): behind a key's own slot all tokens
  // of the call do, up to the window (sinks: to the end).
  __device__ __forceinline__ void tiles(int j0, int n, int& tile0, int& tile1) const {
    const int jl = min(j0 + n, seq.length) - 1;
    const int tok0 = max(0, j0 - seq.slot0());
    const int64_t far = P.window > 0 && j0 >= P.sinks ? (int64_t)jl + P.window - seq.slot0() : seq.count;
    const int tok1 = (int)max((int64_t)0, min((int64_t)seq.count, far));
    tile0 = tok0 * P.group / 16;
    tile1 = tok1 > tok0 ? (tok1 * P.group + 15) / 16 : 0;
  }
  // Slots that no token of the call sees keep what they had; their pages are not looked up.
  __device__ __forceinline__ bool seen(int j) const {
    return seq.count > 0 && (P.window == 0 || j > seq.slot0() - P.window || j < P.sinks);
  }
  __device__ __forceinline__ const T* row_ptr(int r) const {
    const int row = seq.token0 * P.group + r, token = row / P.group;
    return static_cast<const T*>(P.q) + token * P.qs.token + (int64_t)(head * P.group + row - token * P.group) * P.qs.head;
  }
  __device__ __forceinline__ float lse_of(int r) const {
    const int row = seq.token0 * P.group + r, token = row / P.group;
    return __ldg(P.lse + (int64_t)token * P.heads_q + head * P.group + row - token * P.group);
  }
};

constexpr int kStages = 2;  // steps of a warp's ring: three leave room for 8 warps an SM, not 12 (1M tokens 389 us, 336)
constexpr int kStepKeys = 32;  // two blocks of 16 (one at a time: 1M tokens 416 us)

template <int D>
__global__ void __launch_bounds__(kThreads) weigh_bf16_kernel(const PagedWeighParams P) {
  constexpr int kRowBytes = D * 2, kChunks = D / 8, kBlockBytes = kStepKeys * kRowBytes;
  constexpr int kStageBytes = kBlockBytes + kStepKeys * 4;  // keys, and what they had before
  extern __shared__ __align__(128) uint8_t smem_bytes[];
  uint8_t* smem = smem_bytes;
  int64_t* prefix = reinterpret_cast<int64_t*>(smem + kWarps * kStages * kStageBytes);
  next_may_come();
  // Where this kernel runs beside a chunk kernel: its end, that of one CTA of it, comes after the other's.
  auto end_after_others = [&] {
    if (P.beside && blockIdx.x == 0 && blockIdx.y == 0) after_previous();
  };
  slot_prefix<kStepKeys>(P.t, P.group, prefix);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, head = (int)blockIdx.y;
  const int quad = lane >> 2, two = (lane & 3) * 2;
  const int64_t all = prefix[P.t.batch], me = (int64_t)blockIdx.x * kWarps + warp, runs = (int64_t)gridDim.x * kWarps;
  const int64_t x0 = all * me / runs;
  const int n = (int)(all * (me + 1) / runs - x0);
  if (n <= 0) return end_after_others();
  const uint32_t ring = ptx::smem_addr(smem) + warp * kStages * kStageBytes;
  int b_first = 0;  // sequence of the run's first block
  for (int end = P.t.batch; end - b_first > 1;) {
    const int mid = (b_first + end) >> 1;
    (prefix[mid] <= x0 ? b_first : end) = mid;
  }
  while (prefix[b_first + 1] <= x0) ++b_first;

  // Step i of the run into the ring; a lane knows one of the next 32: what it takes to find them is
  // done once for all.
  int known_b = b_first, known_j = 0, known_row[2] = {-2, -2};  // rows of the cache; -1: the page is none, -2: nobody sees it
  const uint8_t* lane_src = static_cast<const uint8_t*>(P.t.cache) + lane / kChunks * kRowBytes + lane % kChunks * 16;
  uint32_t bad = 0u;  // blocks of the stages whose page is none
  auto load = [&](int i) {
    if ((i & 31) == 0 && i < n) {
      int b = __shfl_sync(0xffffffffu, known_b, 31);  // (the last step known so far)
      if (i == 0) b = b_first;
      const int64_t x = min(x0 + i + lane, x0 + n - 1);
      while (prefix[b + 1] <= x) ++b;
      known_b = b;
      known_j = (int)(x - prefix[b]) * kStepKeys;
      const Rows<__nv_bfloat16> rows{P, paged_seq(P.t, b), head};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = known_j + e * kRowsBlock;
        known_row[e] = -2;
        // (of a block the first slot or the last one is seen, or none)
        if (j < rows.seq.length && (rows.seen(j) || rows.seen(min(j + kRowsBlock, rows.seq.length) - 1))) {
          const int page = paged_page(P.t, b, j / P.t.page_rows);
          known_row[e] = page < 0 ? -1 : (int)paged_row(P.t, page, 0, head, j % P.t.page_rows);
        }
      }
    }
    if (i < n) {
      const int b = __shfl_sync(0xffffffffu, known_b, i & 31), j0 = __shfl_sync(0xffffffffu, known_j, i & 31);
      const int s = i % kStages;
      const uint32_t dst = ring + s * kStageBytes;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row0 = __shfl_sync(0xffffffffu, known_row[e], i & 31);
        const uint32_t bit = 1u << (2 * s + e);
        bad = row0 == -1 ? bad | bit : bad & ~bit;
        RA_BOUNDS(P.t.status, row0 >= -2 && row0 + kRowsBlock <= (int64_t)P.t.pages * 2 * P.t.heads_kv * P.t.page_rows, 115);
        const uint8_t* src = lane_src + (int64_t)max(row0, 0) * kRowBytes;
#pragma unroll
        for (int x = 0; x < kChunks / 2; ++x) {
          constexpr int kStep = 32 / kChunks;  // rows
          const int r = x * kStep + lane / kChunks, ch = lane % kChunks;
          copy16(dst + (e * kRowsBlock + r) * kRowBytes + ((ch ^ (r & 7)) * 16), src + x * kStep * kRowBytes, row0 >= 0);
        }
      }
      {
        const int j = j0 + lane;
        const bool had = P.weight_in != nullptr && j < P.weight_width && j < paged_seq(P.t, b).slot0();
        const int64_t at = ((int64_t)b * P.t.heads_kv + head) * P.weight_width + j;
        copy4(dst + kBlockBytes + lane * 4, had ? P.weight_in + at : P.weight, had);
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load(i);

  int b = b_first, held = -1;  // held: the tile of sequence b that is in registers
  Rows<__nv_bfloat16> rows{P, paged_seq(P.t, b), head};
  uint32_t q[D / 16][4];
  float lse2[2] = {0.f, 0.f};
  int slot[2] = {-1, -1};
  for (int i = 0; i < n; ++i) {
    copies_wait<kStages - 2>();
    __syncwarp();
    load(i + kStages - 1);
    const int st = i % kStages;
    if (prefix[b + 1] <= x0 + i) {
      while (prefix[b + 1] <= x0 + i) ++b;
      rows.seq = paged_seq(P.t, b);
      held = -1;
    }
    const int j0 = (int)(x0 + i - prefix[b]) * kStepKeys;
    const int rows_n = rows.seq.count * P.group;
    int tile0, tile1;
    rows.tiles(j0, kStepKeys, tile0, tile1);
    const uint32_t kb = ring + st * kStageBytes;
    float sum[4][2] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};  // keys two, two + 1 of each 8
    for (int t = tile0; t < tile1; ++t) {
      if (t != held) {
        // The rows as the first operand: rows quad and quad + 8, channels two.. and two + 8..
        held = t;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = t * 16 + quad + 8 * e;
          const bool live = r < rows_n;
          slot[e] = live ? rows.seq.slot0() + r / P.group : -1;
          lse2[e] = live ? rows.lse_of(r) * kLog2e : INFINITY;  // (rows of no token: no weight)
          const __nv_bfloat16* src = live ? rows.row_ptr(r) : nullptr;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int f = 0; f < 2; ++f)
              q[kk][e + 2 * f] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16 + f * 8 + two)) : 0u;
        }
      }
      float s[4][4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[c][e] = 0.f;
      const int kr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t r[4];
          ldmatrix4(r, kb + (e * kRowsBlock + kr) * kRowBytes + (((2 * kk + kc) ^ (kr & 7)) * 16));
          mma16816(s[2 * e], q[kk], r[0], r[1]);
          mma16816(s[2 * e + 1], q[kk], r[2], r[3]);
        }
      // Keys that every row of the tile sees need no mask.
      const int s0 = rows.seq.slot0() + t * 16 / P.group;
      const int s1 = rows.seq.slot0() + (min(t * 16 + 16, rows_n) - 1) / P.group;
      const bool whole = j0 + kStepKeys - 1 <= s0 && (P.window == 0 || j0 > s1 - P.window || j0 + kStepKeys <= P.sinks);
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p = ptx::ex2_approx(fmaf(s[c][e], P.scale_log2, -lse2[e >> 1]));
          if (!whole && !paged_sees(P.window, P.sinks, slot[e >> 1], j0 + 8 * c + two + (e & 1))) p = 0.f;
          sum[c][e & 1] += p;
        }
    }
    // Down the columns; then lane l has slot j0 + l.
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) sum[c][e] += __shfl_xor_sync(0xffffffffu, sum[c][e], o);
    // (lanes 4 n + i hold the keys 8 c + 2 i, + 1 in sum[c])
    float mine = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = __shfl_sync(0xffffffffu, sum[c][e], (lane & 7) >> 1);
        if ((lane >> 3) == c && (lane & 1) == e) mine = x;
      }
    const int j = j0 + lane;
    if (j < rows.seq.length && !(((bad >> (2 * st + (lane >> 4))) & 1u) && rows.seen(j))) {
      if (j < P.weight_width) {
        const float had = *reinterpret_cast<const float*>(smem + (kb - ptx::smem_addr(smem)) + kBlockBytes + lane * 4);
        const int64_t at = ((int64_t)b * P.t.heads_kv + head) * P.weight_width + j;
        RA_BOUNDS(P.t.status, j >= 0 && at < (int64_t)P.t.batch * P.t.heads_kv * P.weight_width, 112);
        P.weight[at] = had + mine;
      } else {
        atomicOr(P.t.status, kPagedStatusRange);
      }
    }
    __syncwarp();
  }
  end_after_others();
}

// A lane has a key, in shared memory; a warp has a tile of 16 query rows in shared memory of its
// own, where all lanes read a row's value at once: a key's value enters as many products as there
// are rows.  kFew: each of the CTA's kTeam warps has 32 keys and goes through all tiles.  Otherwise
// the CTA has 32 keys and its warps take the tiles in turn; their sums are added in order.
template <int D, bool kFew, int kTeam>
struct F32 {
  static constexpr int kOwn = kFew ? kTeam * kKeys : kKeys;  // keys of the CTA
  static constexpr int kRow = D + 4;  // floats; 8 lanes' 16-byte reads of a column fall into different banks
  static constexpr int kKeyBytes = kOwn * kRow * 4;
  static constexpr int kWarpBytes = 16 * D * 4 + 2 * 16 * 4;
  static constexpr int kBytes = kKeyBytes + kTeam * kWarpBytes + (kFew ? 0 : kTeam * kKeys * 4);
};

template <int D, bool kFew, int kTeam>
__global__ void __launch_bounds__(kTeam * 32) weigh_f32_kernel(const PagedWeighParams P) {
  using G = F32<D, kFew, kTeam>;
  extern __shared__ __align__(128) uint8_t smem_bytes[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, head = (int)blockIdx.y;
  float* keys = reinterpret_cast<float*>(smem_bytes) + (kFew ? warp * kKeys * G::kRow : 0);
  float* qs = reinterpret_cast<float*>(smem_bytes + G::kKeyBytes + warp * G::kWarpBytes);
  float* lse2 = qs + 16 * D;
  int* slots = reinterpret_cast<int*>(lse2 + 16);
  float* sums = reinterpret_cast<float*>(smem_bytes + G::kKeyBytes + kTeam * G::kWarpBytes);
  int64_t* prefix = reinterpret_cast<int64_t*>(smem_bytes + G::kBytes);
  slot_prefix<G::kOwn>(P.t, P.group, prefix);
  const int64_t chunks = prefix[P.t.batch];
  const float* cache = static_cast<const float*>(P.t.cache);
  int b = 0;
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    while (prefix[b + 1] <= c) ++b;
    const Rows<float> rows{P, paged_seq(P.t, b), head};
    const int first = (int)(c - prefix[b]) * G::kOwn + (kFew ? warp * kKeys : 0), j = first + lane;
    const bool look = j < rows.seq.length && rows.seen(j);
    const int page = look ? paged_page(P.t, b, j / P.t.page_rows) : -1;
    const int row = page >= 0 ? (int)paged_row(P.t, page, 0, head, j % P.t.page_rows) : -1;
    RA_BOUNDS(P.t.status, row >= -1 && row < (int64_t)P.t.pages * 2 * P.t.heads_kv * P.t.page_rows, 114);
    // Keys and sums of the chunk before are done with.
    if constexpr (kFew) __syncwarp(); else __syncthreads();
    constexpr int kPieces = D / 4, kBring = kFew ? 32 : kTeam * 32;
#pragma unroll 8
    for (int x = 0; x < kKeys * kPieces / kBring; ++x) {
      const int id = (kFew ? lane : (int)threadIdx.x) + x * kBring, i = id / kPieces, ch = id % kPieces;
      const int from = __shfl_sync(0xffffffffu, row, i);
      copy16(ptx::smem_addr(keys + i * G::kRow + ch * 4), cache + (int64_t)max(from, 0) * D + ch * 4, from >= 0);
    }
    copies_commit();
    const int rows_n = rows.seq.count * P.group;
    int tile0, tile1;
    rows.tiles(first, kKeys, tile0, tile1);
    float sum = 0.f;
    bool there = false;  // the keys are
    auto await = [&] {
      if (there) return;
      copies_wait<0>();
      if constexpr (kFew) __syncwarp(); else __syncthreads();
      there = true;
    };
    for (int t = tile0 + (kFew ? 0 : warp); t < tile1; t += kFew ? 1 : kTeam) {
      const int n = min(16, rows_n - t * 16);
      __syncwarp();
      for (int id = lane; id < n * kPieces; id += 32)
        reinterpret_cast<float4*>(qs)[id] = __ldg(reinterpret_cast<const float4*>(rows.row_ptr(t * 16 + id / kPieces)) + id % kPieces);
      if (lane < n) {
        lse2[lane] = rows.lse_of(t * 16 + lane) * kLog2e;
        slots[lane] = rows.seq.slot0() + (t * 16 + lane) / P.group;
      }
      __syncwarp();
      await();
      const float* k = keys + lane * G::kRow;
      auto add = [&](auto most, int r0) {  // rows r0 .. r0 + most
        constexpr int kN = decltype(most)::value;
        float s[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) s[i] = 0.f;
#pragma unroll 4
        for (int x = 0; x < kPieces; ++x) {
          const float4 kk = *reinterpret_cast<const float4*>(k + x * 4);
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const float4 q = *reinterpret_cast<const float4*>(qs + (r0 + i) * D + x * 4);
            s[i] = fmaf(q.x, kk.x, fmaf(q.y, kk.y, fmaf(q.z, kk.z, fmaf(q.w, kk.w, s[i]))));
          }
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          if (r0 + i >= n) break;
          const float p = exp2f(fmaf(s[i], P.scale_log2, -lse2[r0 + i]));
          sum += paged_sees(P.window, P.sinks, slots[r0 + i], j) ? p : 0.f;
        }
      };
      if (n > 8) {
        add(std::integral_constant<int, 16>(), 0);
      } else {
        for (int r0 = 0; r0 < n; r0 += 4) add(std::integral_constant<int, 4>(), r0);
      }
    }
    await();
    if constexpr (!kFew) {
      sums[warp * kKeys + lane] = sum;
      __syncthreads();
    }
    if ((kFew || warp == 0) && j < rows.seq.length && (page >= 0 || !look)) {
      if (j < P.weight_width) {
        const int64_t at = ((int64_t)b * P.t.heads_kv + head) * P.weight_width + j;
        RA_BOUNDS(P.t.status, at < (int64_t)P.t.batch * P.t.heads_kv * P.weight_width, 113);
        if constexpr (!kFew) {
          sum = 0.f;
#pragma unroll
          for (int i = 0; i < kTeam; ++i) sum += sums[i * kKeys + lane];
        }
        P.weight[at] = (P.weight_in != nullptr && j < rows.seq.slot0() ? P.weight_in[at] : 0.f) + sum;
      } else {
        atomicOr(P.t.status, kPagedStatusRange);
      }
    }
  }
}

// CTAs per head: as many as the GPU holds at once, each with work at the sizes given.
unsigned slots_of(const PagedWeighParams& prm, int sm_count, int per_sm, int own) {
  const int64_t most = (int64_t)std::min(prm.t.batch, 1 << 20) * ((prm.t.width * prm.t.page_rows + own - 1) / own);
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>(most, (int64_t)sm_count * per_sm / prm.t.heads_kv));
}

template <typename Kernel>
cudaError_t launch(Kernel kernel, std::atomic<int>* ready, const PagedWeighParams& prm, unsigned slots, int threads,
                   int bytes, cudaStream_t stream) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool cached = dev >= 0 && dev < kMaxDevices;
  if (!cached || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes + (kMaxSequences + 1) * 8);
    if (e != cudaSuccess) return e;
    if (cached) ready[dev].store(1, std::memory_order_release);
  }
  const dim3 grid(slots, (unsigned)prm.t.heads_kv);
  const int all = bytes + (prm.t.batch + 1) * 8;
  if (prm.beside) return launch_behind(kernel, grid, threads, all, stream, prm);
  kernel<<<grid, threads, all, stream>>>(prm);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_bf16(const PagedWeighParams& prm, int sm_count, cudaStream_t stream) {
  static std::atomic<int> ready[kMaxDevices];
  return launch(weigh_bf16_kernel<D>, ready, prm, slots_of(prm, sm_count, 3, kWarps * kStepKeys), kThreads,
                kWarps * kStages * (kStepKeys * D * 2 + kStepKeys * 4), stream);
}
template <int D, bool kFew, int kTeam>
cudaError_t launch_f32(const PagedWeighParams& prm, int sm_count, cudaStream_t stream) {
  using G = F32<D, kFew, kTeam>;
  static std::atomic<int> ready[kMaxDevices];
  constexpr int kPerSm = kTeam == 16 ? 1 : (kFew ? 4 : 8) / (D / 64);
  return launch(weigh_f32_kernel<D, kFew, kTeam>, ready, prm, slots_of(prm, sm_count, kPerSm, G::kOwn), kTeam * 32, G::kBytes,
                stream);
}
template <int D>
cudaError_t launch_f32(const PagedWeighParams& prm, int sm_count, cudaStream_t stream) {
  // By the mean rows of a sequence and head.  16 sequences of 4k, D 128, few and not: 4 rows 54
  // and 65 us, 16 rows 102 and 132, 32 rows 170 and 158, 64 rows 310 and 231 (D 64: 26 and 47,
  // 47 and 88, 78 and 108, 138 and 147).
  const int64_t rows = (int64_t)prm.t.tokens * prm.group;
  if (rows <= 32 * (int64_t)prm.t.batch) return launch_f32<D, true, kWarps>(prm, sm_count, stream);
  // Many rows and few keys: more warps of a CTA.  400 tokens of 8 heads over 700 slots of one 162 us
  // (with 4 warps 302), 2048 tokens of one head 105 (195); but 500 tokens over 4k of 8 heads, D 64, 205
  // (172), and 64 rows of a sequence 404 (231).
  const int64_t ctas = (int64_t)prm.t.batch * ((prm.t.width * prm.t.page_rows + kKeys - 1) / kKeys) * prm.t.heads_kv;
  if (rows >= 256 * (int64_t)prm.t.batch && ctas < 4 * (int64_t)sm_count) return launch_f32<D, false, 16>(prm, sm_count, stream);
  return launch_f32<D, false, kWarps>(prm, sm_count, stream);
}

}  // namespace

cudaError_t launch_paged_weigh_rows(int dtype, int head_dim, const PagedWeighParams& prm, int sm_count,
                                    cudaStream_t stream) {
  if (dtype == RA_DTYPE_BF16)
    return head_dim == 128 ? launch_bf16<128>(prm, sm_count, stream) : launch_bf16<64>(prm, sm_count, stream);
  return head_dim == 128 ? launch_f32<128>(prm, sm_count, stream) : launch_f32<64>(prm, sm_count, stream);
}

}  // namespace ra
