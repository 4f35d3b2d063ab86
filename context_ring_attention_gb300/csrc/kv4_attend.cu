// Attention of a few new tokens per sequence over the 4-bit cache.
//
// For the query rows of one key/value head (rows of its group's heads and of the new
// tokens, 8 to a tile) and the cached keys j that they see, with codes n, scales ks, vs
// and minima kl, vl of every group g of 32 channels,
//   s_j = sum_g [ ks_jg * sum_{c in g} q_c n_jc + kl_jg * sum_{c in g} q_c ],
//   O   = sum_j p_j [ vs_jg * (n_jc - 8) + (vl_jg + 8 vs_jg) ] / sum_j p_j,  p_j = e^(s_j - m).
// The codes enter the products as exact integers and the parameters are applied per group
// in fp32: to the 4 sums of a score, and to p before it is rounded for the second product;
// the minima's share of O is a plain fp32 sum per group.  The values' codes are centred
// (by a second product with the constant -8 and the same rounded p), which keeps the
// rounding of p from being multiplied by the offset of the group.
//
// Bound by HBM at 20 * d bytes per 16 tokens and head.  The products are so few (8 query
// rows) that the warp-level tensor instruction serves: m16n8k16 with the codes as the
// 16-row operand -- keys x channels for the scores, channels x keys for the output -- and
// the query rows as its 8 columns, so that nothing is computed for absent rows beyond 8.
// What had to be made cheap is turning codes into operands (the first form, which made
// bf16 n - 8 by a shift, a logical and a subtraction a pair, ran at 2.9 TB/s, bound by
// those).  bf16 numbers whose top 8 bits are zero are the integers 0..255 times 2^-133,
// subnormal below 128 and linear across the border, and the instruction takes them as they
// are: a word of 8 codes yields 4 operand registers by one shift and 4 logicals, the codes
// of the bytes' high nibbles standing for 16 n.  The other operands carry the powers of two
// that bring the products back: the queries 2^E (E from the row's largest), the weights p
// 2^kShift.  Scales of value groups from 2^-52 to 2^58 keep full precision that way.
// The instruction aligns a product by its operands' exponents, which for n are those of 128
// (for 16 n those of 128 too, or n's own from 8 on): measured, a product n * q is off by up to
// 2^-18 of q, 16 n * q by 2^-22, which bf16 results do not see.  fp32 takes all codes as 16 n, by
// two shifts more a word (84 us became 86 for the figure below).
// Scores come out with keys in rows and are turned for the second product by an 8x8
// transpose in registers.
//
// Split: a CTA of 4 warps takes a share of the 16-token blocks that a tile sees, each warp
// a quarter; m, l and O are joined across warps in shared memory, and across CTAs by a
// second kernel in a fixed order.  A warp works on two blocks at a time: with one at a time
// and four CTAs an SM (128 registers) its chains of dependent instructions, from the scores
// to the weights, were what it waited for; two blocks (three CTAs an SM) took one sequence of
// 1M tokens from 276 to 257 us (before the form for few rows) and 16 new tokens of 64k from 180
// to 136.  Two blocks in 128 registers: 276 us; two pairs a warp in shared memory for three: 260.
//
// Measured (32 query and 8 key/value heads, d = 128, bf16, one new token): 1M tokens 235 us,
// 1.34 GB of cache at 5.7 TB/s (0.84 of a plain copy's rate); 64k tokens 26.7 us; 32 sequences
// of 2k to 32k under a window of 8192 tokens 70 us.  What bounds it is the latency of
// dependent instructions with 11 warps an SM (55% of the issue slots, HBM 65%, the largest
// stall a fixed wait): some 300 instructions a block and warp, more than half of them for
// turning codes and weights into operands.  Every tile of 8 query rows reads and unpacks the
// cache for itself: 2 new tokens over 1M take 258 us, 16 over 64k (8 tiles) 136, 4 over 8
// sequences of up to 32k (2 tiles) 100.  fp32 takes three terms per query and weight and three times the products:
// 4 sequences of 64k tokens 86 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kv4_internal.h"
#include "sm100_ptx.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;
constexpr int kTile = 8;  // query rows of a tile
constexpr int kMinBlocks = 16;  // of a share: four a warp
constexpr int kSnap = 8;
constexpr int kPairs = 3;  // pairs of cache blocks a warp holds or has under way
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleSlack = 8.0f;  // log2 units: keep a stale maximum while p <= 2^8

// D = A (16 x 16, row) * B (16 x 8, col) + D, bf16 in, fp32 sums.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// The same with zeros for D on the way in.
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
}
// Transpose of an 8 x 8 matrix of 16-bit elements held two to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Pairs of codes as bf16 operands: n * 2^-133 from bits 0-3 and 16-19 of x, 16 n * 2^-133
// from bits 4-7 and 20-23.
__device__ __forceinline__ uint32_t codes_lo(uint32_t x) { return x & 0x000f000fu; }
__device__ __forceinline__ uint32_t codes_hi(uint32_t x) { return x & 0x00f000f0u; }
// The first of the two by the number of terms: the second form, brought there, where there are 3.
template <int kTerms>
__device__ __forceinline__ uint32_t codes_first(uint32_t word, int at) {
  if (kTerms == 1) return codes_lo(word >> at);
  return codes_hi(at == 0 ? word << 4 : word >> (at - 4));
}
constexpr uint32_t kMinus8Lo = 0x80088008u, kMinus8Hi = 0x80808080u;  // the code -8 in both forms
constexpr int kShift = 60;  // log2 of the factor that every p carries into the products
// The part of it that the exponential's argument brings: all, without another instruction, for
// bf16; none for fp32, where an argument near 60 would lose 2^-19.
template <int kTerms>
constexpr int kInExponent = kTerms == 1 ? kShift : 0;
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126..127
__device__ __forceinline__ float scale_of(uint32_t par) { return __uint_as_float(par << 16); }
__device__ __forceinline__ float low_of(uint32_t par) { return __uint_as_float(par & 0xffff0000u); }

// Token of a block that row i of the score product stands for.
__device__ __forceinline__ int token_of(int i) {
  const int j = i & 7;
  return (i & 8) + ((j & 1) ? 4 + ((j >> 1) ^ 1) : j >> 1);
}

// 16 bytes from global to shared memory, asynchronously.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// kN 32-bit words from shared memory, in the widest loads.
template <int kN>
__device__ __forceinline__ void load_words(const uint8_t* src, uint32_t (&w)[kN]) {
  if constexpr (kN == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(src);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if constexpr (kN == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(src);
    w[0] = x.x, w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(src);
  }
}

// x as kTerms bf16 terms (packed in pairs with y): 1 rounds, 3 keep 24 bits.
template <int kTerms>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&out)[kTerms]) {
#pragma unroll
  for (int n = 0; n < kTerms; ++n) {
    out[n] = ptx::pack_bf16x2(x, y);
    if (n + 1 < kTerms) {
      x -= __uint_as_float(out[n] << 16);
      y -= __uint_as_float(out[n] & 0xffff0000u);
    }
  }
}

template <typename T>
__device__ __forceinline__ float to_f(T x) {
  return (float)x;
}

// The blocks of a sequence that some row of its queries sees: the sinks' [0, first), then
// from `from` on; n of them in all.
struct Blocks {
  int32_t first, from, n;
};
__device__ __forceinline__ Blocks blocks_of(const Kv4AttendParams& P, int32_t len) {
  Blocks b;
  const int32_t end = (len + kKvBlockRows - 1) / kKvBlockRows;
  int64_t lo = 0;
  if (P.window > 0) lo = (int64_t)len - P.rows - P.window + 1;
  if (lo < 0) lo = 0;
  b.from = (int32_t)(lo / kKvBlockRows);
  const int32_t sink_rows = P.sinks < lo ? P.sinks : (int32_t)lo;
  b.first = (sink_rows + kKvBlockRows - 1) / kKvBlockRows;
  if (b.first > b.from) b.first = b.from;
  b.n = b.first + (end - b.from);
  return b;
}

// Tokens of sequence b that the cache holds; a length out of range counts as none.
__device__ __forceinline__ int32_t length_of(const Kv4AttendParams& P, int b, bool& bad) {
  const int32_t len = __ldg(P.length + b);
  bad = len < 0 || len > P.t.width * P.t.page_rows;
  return bad ? 0 : len;
}

// The share of a slot: n blocks of the sequences one after the other, from block `off` of
// sequence b on.  (A sequence without blocks stands in the row with one, so that its rows are
// written.)
struct Share {
  int32_t b, off, n;
};
// N blocks in all make up to `slots` equal shares of kMinBlocks or more; a border that would
// fall within kSnap blocks of a sequence's end is put there.  Every CTA finds its own from the
// lengths.
template <bool kInRow>
__device__ __forceinline__ Share share_of(const Kv4AttendParams& P, int slot) {
  bool bad;
  auto blocks = [&](int b) { return b < P.t.batch ? max(1, blocks_of(P, length_of(P, b, bad)).n) : 0; };
  if (!kInRow && P.slots == P.t.batch) return {slot, 0, blocks(slot)};
  auto border = [&](int32_t total, int i) {
    const int32_t shares = kInRow ? max(1, min(P.slots, total / kMinBlocks)) : P.slots;
    return i >= shares ? total : (int32_t)((int64_t)total * i / shares);
  };
  if (!kInRow) {  // one sequence; every slot has a part, if of no blocks
    const int32_t total = blocks(0), from = border(total, slot);
    return {0, from, border(total, slot + 1) - from};
  }
  __shared__ int32_t sums[kWarps], ends[kWarps];
  __shared__ int32_t found[2][3];  // of either border: sequence, block of it, place
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t mine = blocks(threadIdx.x);
  int32_t total = mine;  // (the host keeps the sum within 31 bits)
  for (int b = threadIdx.x + kWarps * 32; b < P.t.batch; b += kWarps * 32) total += blocks(b);
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0) sums[warp] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += sums[w];
  const int32_t at[2] = {border(total, slot), border(total, slot + 1)};
  if (at[0] == at[1]) return {0, 0, 0};
  if (threadIdx.x == 0) found[1][2] = total;  // (where at[1] is the end of all)
  int32_t base = 0;
  for (int b0 = 0; b0 < P.t.batch && base <= at[1]; b0 += kWarps * 32) {  // (uniform)
    const int b = b0 + threadIdx.x;
    const int32_t n = b0 == 0 ? mine : blocks(b);
    int32_t end = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t x = __shfl_up_sync(0xffffffffu, end, d);
      if (lane >= d) end += x;
    }
    __syncthreads();  // (the last chunk's ends are read no more; found[1] has its default)
    if (lane == 31) ends[warp] = end;
    __syncthreads();
    end += base;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) end += ends[w];
      base += ends[w];
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int32_t off = at[x] - (end - n);
      if (off < 0 || off >= n) continue;
      const bool down = off <= kSnap, up = !down && n - off <= kSnap;
      found[x][0] = up ? b + 1 : b;
      found[x][1] = down || up ? 0 : off;
      found[x][2] = down ? end - n : up ? end : at[x];
    }
  }
  __syncthreads();
  return {found[0][0], found[0][1], found[1][2] - found[0][2]};
}

// kInRow: the sequences' blocks are shared in a row, so that a CTA may have parts of several;
// otherwise it has (a share of) one.  (As one kernel a single sequence of 1M tokens took 4%
// longer, and one of 8k 12 us for 10.)
// kHalf: up to 4 query rows, one new token of a group of up to 4 heads.  The products have 8
// columns: the first 4 are then the rows over the first of the warp's two blocks, the others
// the same rows over the second, each with a maximum and sums of its own, joined at the end as
// the warps' are.  Scores, exponentials and weights take half the instructions (one sequence of
// 1M tokens 258 us with 4 empty columns, 234 so; 32 under a window of 8192 79 and 71).
template <typename T, int D, bool kInRow, bool kHalf>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 ? (kHalf ? D == 64 ? 4 : 3 : 3) : 1) kv4_attend_kernel(const Kv4AttendParams P) {
  using F = Kv4Block<D>;
  constexpr int G = F::kGroups;
  constexpr int kTerms = sizeof(T) == 2 ? 1 : 3, kIn = kInExponent<kTerms>;
  constexpr int kSets = kHalf ? 1 : 2;  // sets of scores: of either block, or of both
  constexpr int kRows = kHalf ? kTile / 2 : kTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  const int rq = kHalf ? r & 3 : r;  // query row of the fragments' column r
  const bool second = kHalf && c >= 2;  // this lane's columns are of the second block
  // One sequence: the shares of a head next to each other (1M tokens 2% faster than with the
  // heads of a share next to each other); several: the heads, whose blocks lie in the same
  // pages (64 sequences of up to 2k 6% faster).
  const bool one = !kInRow && P.t.batch == 1;
  const int cta = one ? blockIdx.x : blockIdx.y, ht = one ? blockIdx.y : blockIdx.x;
  const int tile = ht % P.tiles, h = ht / P.tiles;
  const int n_rows = P.group * P.rows;  // query rows of the head: row = group head * rows + token
  const int row0 = tile * kTile;

  cudaTriggerProgrammaticLaunchCompletion();
  if (!kInRow && row0 + r < n_rows) {  // the queries are on their way while the length is asked for
    const T* qrow = static_cast<const T*>(P.q) +
                    (((int64_t)(one ? 0 : cta) * P.heads_q + (int64_t)h * P.group) * P.rows + row0 + r) * D;
    asm volatile("prefetch.global.L1 [%0];" ::"l"(qrow + c * (D / 4)));
  }
  const Share share = share_of<kInRow>(P, cta);
  int32_t off = share.off, rest = share.n;
  for (int b = share.b; !kInRow || rest > 0; ++b) {
  RA_BOUNDS(P.t.status, b >= 0 && b < P.t.batch && h < P.t.heads_kv && share.off >= 0 && share.n >= 0, 95);
  bool bad_length;
  const int32_t len = length_of(P, b, bad_length);
  if (bad_length && threadIdx.x == 0) atomicOr(P.t.status, kKv4StatusRange);
  const Blocks blk = blocks_of(P, len);
  const int32_t x_lo = min(off, blk.n), x_hi = min(off + rest, blk.n);
  // the sequence begins and ends in this share
  const bool begins = kInRow ? off == 0 : P.slots == P.t.batch || cta == 0;
  const bool ends = kInRow ? off + rest >= blk.n : P.slots == P.t.batch || cta == P.slots - 1;
  rest -= max(1, blk.n) - off;
  off = 0;

  // Query fragments: lane (r, c) holds row r's channels 32g + 8c .. + 7 of every group, in
  // the pairs (0,4), (1,5), (2,6), (3,7) that a word of codes yields, times 2^E; the pairs
  // that meet 16 n (fp32: all) are divided by 16.  E puts the row's largest channel at 2^119..2^120.
  uint32_t qf[G][4][kTerms];
  uint32_t qsum[4]; // sum of group c's channels of row r, in the scores' unit 2^(E - 133)
  float back[2];    // that unit's inverse for rows 2c and 2c + 1, times the score scale (log2 units)
  {
    const bool live = row0 + rq < n_rows;
    const T* qrow = static_cast<const T*>(P.q) + (((int64_t)b * P.heads_q + (int64_t)h * P.group) * P.rows + row0 + rq) * D;
    float x[G][8];
    float top = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[g][i] = live ? to_f(qrow[32 * g + 8 * c + i]) : 0.f;
        top = fmaxf(top, fabsf(x[g][i]));
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // exponent of the largest channel (-126 for zeros and below); E in two factors
    const int exp_top = max((int)(__float_as_uint(top) >> 23) - 127, -126);
    const int e_row = 119 - exp_top;  // -9 .. 245
    const float f0 = two_to(e_row / 2), f1 = two_to(e_row - e_row / 2);
    float sums[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[g][i] = x[g][i] * f0 * f1;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = (i & 1) || kTerms > 1 ? 0.0625f : 1.f;
        split_pair<kTerms>(x[g][i] * f, x[g][i + 4] * f, qf[g][i]);
        sum += x[g][i] * two_to(-100) + x[g][i + 4] * two_to(-100);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sums[g] = sum * two_to(-33);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int up = 133 - __shfl_sync(0xffffffffu, e_row, 8 * c + 4 * e);  // -112 .. 142
      back[e] = P.scale_log2 * two_to(up / 2) * two_to(up - up / 2);
    }
    // (0, sum of group c) in four bf16 terms; lanes beyond the groups stand for none
    float mine_sum = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) mine_sum = c == g ? sums[g] : mine_sum;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      qsum[n] = ptx::pack_bf16x2(0.f, mine_sum);
      mine_sum -= __uint_as_float(qsum[n] & 0xffff0000u);
    }
  }
  extern __shared__ __align__(16) uint8_t ring[];
  // The fragments wait in shared memory, the same for all warps: registers are what bounds
  // the warps of an SM.
  constexpr int kFrags = G * kTerms * (kHalf ? 2 : 1);
  uint32_t* const qsm = reinterpret_cast<uint32_t*>(ring + kWarps * kPairs * 2 * F::kBytes);
  if (warp == 0) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int n = 0; n < kTerms; ++n) {
        const uint4 f = make_uint4(qf[g][0][n], qf[g][1][n], qf[g][2][n], qf[g][3][n]), none = make_uint4(0u, 0u, 0u, 0u);
        uint4* at = reinterpret_cast<uint4*>(qsm + ((g * kTerms + n) * 32 + lane) * 4);
        if (!kHalf) {
          at[0] = f;
        } else {  // for the first block in columns 0-3, for the second in 4-7
          at[0] = r < 4 ? f : none;
          at[G * kTerms * 32] = r < 4 ? none : f;
        }
      }
    }
    *reinterpret_cast<uint4*>(qsm + kFrags * 32 * 4 + lane * 4) = make_uint4(qsum[0], qsum[1], qsum[2], qsum[3]);
  }
  __syncthreads();
  // Positions of rows 2c and 2c + 1 (of the query), and the tokens of this lane's keys.
  int32_t qpos[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) qpos[e] = len - P.rows + (row0 + ((2 * c + e) & (kRows - 1))) % P.rows;
  const int tok0 = token_of(r), tok1 = token_of(r + 8);
  const int vt[4] = {token_of(2 * c), token_of(2 * c + 1), token_of(2 * c + 8), token_of(2 * c + 9)};

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[G][2][4];  // channels 32g + 4r + {0,1} and {2,3} of rows 2c, 2c + 1 (the odd ones, in fp32 all, times 16)
  float pm[G][2];    // sum of p * (middle of the group's range)
#pragma unroll
  for (int g = 0; g < G; ++g) {
    pm[g][0] = pm[g][1] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[g][i][e] = 0.f;
  }

  // Each warp brings its blocks, two at a time, through slots of its own in shared memory:
  // the next pairs are under way while it works on one.
  uint8_t* const mine = ring + warp * (kPairs * 2 * F::kBytes);
  const uint32_t mine_at = ptx::smem_addr(mine);
  uint32_t bad = 0;  // blocks of the slots that are not there: the page is out of range, or past the end
  // A warp's blocks follow each other: their place is looked up in the page table at the
  // first of each page, at the warp's first and behind the sinks.
  const int32_t w_lo = x_lo + (int32_t)((int64_t)(x_hi - x_lo) * warp / kWarps);
  const int32_t w_hi = x_lo + (int32_t)((int64_t)(x_hi - x_lo) * (warp + 1) / kWarps);
  auto block_at = [&](int32_t x) { return x < blk.first ? x : blk.from + (x - blk.first); };
  const int32_t bpp = P.t.blocks_per_page;
  const int32_t* table = P.t.page_table + (int64_t)b * P.t.width;
  const int64_t page_bytes = (int64_t)P.t.heads_kv * bpp * F::kBytes;
  const uint8_t* of_head = P.t.cache + (int64_t)h * bpp * F::kBytes + lane * 16;
  const uint8_t* src = nullptr;  // the next block to fetch, or nullptr: its page is out of range
  int32_t left = 0;              // blocks from there to the page's end or the sinks'
  int32_t fx = w_lo;
  auto fetch_one = [&](int at) {
    bad |= 1u << at;
    if (fx >= w_hi) return;
    if (left == 0) {
      const int32_t block = block_at(fx);
      const int32_t page_at = block / bpp, in_page = block - page_at * bpp;
      RA_BOUNDS(P.t.status, block >= 0 && page_at < P.t.width, 96);
      const int32_t page = __ldg(table + page_at);
      src = of_head + page * page_bytes + (int64_t)in_page * F::kBytes;
      left = bpp - in_page;
      if (fx < blk.first) left = min(left, blk.first - fx);
      if (page < 0 || page >= P.t.pages) {
        src = nullptr;
        if (lane == 0) atomicOr(P.t.status, kKv4StatusRange);
      }
    }
    if (src != nullptr) {
      bad &= ~(1u << at);
      RA_BOUNDS(P.t.status, in_pool<D>(P.t, src - lane * 16) && at >= 0 && at < 2 * kPairs, 97);
      const uint32_t dst = mine_at + at * F::kBytes + lane * 16;
#pragma unroll
      for (int i = 0; i * 512 < F::kBytes; ++i)
        if (i * 512 + 512 <= F::kBytes || lane * 16 + i * 512 < F::kBytes) copy16(dst + i * 512, src + i * 512);
      src += F::kBytes;
    }
    --left;
    ++fx;
  };
  auto fetch = [&](int slot) {
    fetch_one(2 * slot);
    fetch_one(2 * slot + 1);
    copies_commit();  // (an empty group where there is nothing to fetch)
  };
  // Blocks that every row sees whole need no mask: they end at the first query or before,
  // and begin within the last query's window or lie in the sinks.
  const int32_t whole_to = (len - P.rows + 1) >> 4;  // block + 1 <= this (arithmetic shift: may be negative)
  const int32_t whole_from = P.window == 0 ? 0 : (max(len - P.window, 0) + 15) >> 4;
  const int32_t whole_sinks = P.sinks >> 4;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) fetch(i);

  int slot = 0;
  for (int32_t x = w_lo; x < w_hi; x += 2, slot = slot == kPairs - 1 ? 0 : slot + 1) {
    copies_wait<kPairs - 1>();
    __syncwarp();  // every lane's copies have landed
    const uint8_t* base[2] = {mine + (2 * slot) * F::kBytes, mine + (2 * slot + 1) * F::kBytes};
    const uint32_t gone = (bad >> (2 * slot)) & 3u;
    auto own = [&](int n) { return kHalf ? (second ? base[1] : base[0]) : base[n]; };  // the block of score set n

    // Scores: s[n][0], s[n][1] of key tok0 of block n for rows 2c, 2c + 1; s[n][2], s[n][3]
    // of key tok1.  The minima's part first, as products of their own: a parameter word is
    // (scale, low) of key and group c, met by (0, sum of q) in bf16 terms.
    float s[kSets][4];
    uint32_t kp0[kSets][G], kp1[kSets][G];
    {
      uint32_t qw[4];
      load_words<4>(reinterpret_cast<const uint8_t*>(qsm + kFrags * 32 * 4 + lane * 4), qw);
      const uint32_t b01[2] = {qw[0], qw[1]}, b23[2] = {qw[2], qw[3]};
      float low[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        uint32_t lw[2];
        lw[0] = *reinterpret_cast<const uint32_t*>(base[n] + F::kOffKPar + tok0 * F::kParBytes + (c & (G - 1)) * 4);
        lw[1] = *reinterpret_cast<const uint32_t*>(base[n] + F::kOffKPar + tok1 * F::kParBytes + (c & (G - 1)) * 4);
        const uint32_t a[4] = {lw[0], lw[1], lw[0], lw[1]};
        mma16816_first(low[n], a, b23);
        mma16816(low[n], a, b01);
      }
#pragma unroll
      for (int n = 0; n < kSets; ++n) {
        // (the minima's products of the two blocks are apart, since what is not seen may be NaN)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = kHalf ? (second ? low[1][e] : low[0][e]) : low[n][e];
        load_words<G>(own(n) + F::kOffKPar + tok0 * F::kParBytes, kp0[n]);
        load_words<G>(own(n) + F::kOffKPar + tok1 * F::kParBytes, kp1[n]);
      }
    }
    {
      uint32_t k0[2][G], k1[2][G];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        load_words<G>(base[n] + F::kOffK + tok0 * F::kCodeBytes + c * (4 * G), k0[n]);
        load_words<G>(base[n] + F::kOffK + tok1 * F::kCodeBytes + c * (4 * G), k1[n]);
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float acc[kSets][4];
        uint32_t qg[kHalf ? 2 : 1][kTerms][4];
#pragma unroll
        for (int y = 0; y < (kHalf ? 2 : 1); ++y)
#pragma unroll
          for (int t = 0; t < kTerms; ++t)
            load_words<4>(reinterpret_cast<const uint8_t*>(qsm + (((y * G + g) * kTerms + t) * 32 + lane) * 4), qg[y][t]);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {  // nibbles (i, i + 4) and (i + 1, i + 5) of the words
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t a[4] = {codes_first<kTerms>(k0[n][g], 4 * i), codes_first<kTerms>(k1[n][g], 4 * i),
                                   codes_hi(k0[n][g] >> (4 * i)), codes_hi(k1[n][g] >> (4 * i))};
            const int set = kHalf ? 0 : n, y = kHalf ? n : 0;
#pragma unroll
            for (int t = kTerms - 1; t >= 0; --t) {
              const uint32_t q2[2] = {qg[y][t][i], qg[y][t][i + 1]};
              if (i == 0 && t == kTerms - 1 && y == 0) mma16816_first(acc[set], a, q2);
              else mma16816(acc[set], a, q2);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < kSets; ++n) {
          const float s0 = scale_of(kp0[n][g]), s1 = scale_of(kp1[n][g]);
          s[n][0] = fmaf(s0, acc[n][0], s[n][0]);
          s[n][1] = fmaf(s0, acc[n][1], s[n][1]);
          s[n][2] = fmaf(s1, acc[n][2], s[n][2]);
          s[n][3] = fmaf(s1, acc[n][3], s[n][3]);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < kSets; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] *= back[e & 1];

    const int32_t first_block = block_at(x), second_block = block_at(x + 1);
    uint32_t seen = 0xffu;  // bit 4n + e
    const bool whole = gone == 0u && first_block < whole_to && second_block < whole_to &&
                       (first_block >= whole_from || first_block < whole_sinks) &&
                       (second_block >= whole_from || second_block < whole_sinks);
    if (!whole) {
#pragma unroll
      for (int n = 0; n < kSets; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool last = kHalf ? second : n == 1;
          const int32_t j = (last ? second_block : first_block) * kKvBlockRows + (e < 2 ? tok0 : tok1), i = qpos[e & 1];
          if (((gone >> (last ? 1 : 0)) & 1u) || !(j <= i && (P.window == 0 || j > i - P.window || j < P.sinks))) {
            seen &= ~(1u << (4 * n + e));
            s[n][e] = -INFINITY;
          }
        }
    }

    // Running maximum, the same in all lanes of a row: moved only when a score exceeds it
    // by the slack.
    float mx[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[e] = fmaxf(s[0][e], s[0][e + 2]);
      if (!kHalf) mx[e] = fmaxf(mx[e], fmaxf(s[kSets - 1][e], s[kSets - 1][e + 2]));
    }
    if (__any_sync(0xffffffffu, mx[0] > m[0] + kRescaleSlack || mx[1] > m[1] + kRescaleSlack)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], d));
        mx[e] = fmaxf(mx[e], m[e]);
        const float alpha = m[e] == -INFINITY ? 0.f : ptx::ex2_approx(m[e] - mx[e]);
        m[e] = mx[e];
        l[e] *= alpha;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          pm[g][e] *= alpha;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            o[g][i][e] *= alpha;
            o[g][i][e + 2] *= alpha;
          }
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float ref = m[e] == -INFINITY ? 0.f : m[e] - (float)kIn;
#pragma unroll
      for (int n = 0; n < kSets; ++n)
#pragma unroll
        for (int i = e; i < 4; i += 2) {
          s[n][i] = ptx::ex2_approx(s[n][i] - ref);  // p from here on
          l[e] += s[n][i];
        }
    }

    // O: per group, p times the value's scale as the 16 x 8 operand (keys x rows), the
    // codes of two keys a register as the 16 x 16 one (channels x keys).
    auto values = [&](auto masked) {
      constexpr uint32_t kFirst8 = kTerms == 1 ? kMinus8Lo : kMinus8Hi;
      const uint32_t minus8[4] = {kFirst8, kMinus8Hi, kFirst8, kMinus8Hi};
      constexpr int kWith = kHalf ? 2 : 1;  // blocks of a score set
#pragma unroll
      for (int n = 0; n < kSets; ++n) {
        asm volatile("" ::: "memory");  // (one set's words are held at a time)
        uint32_t vp0[G], vp1[G], vw[kWith][4][G / 2];
        load_words<G>(own(n) + F::kOffVPar + tok0 * F::kParBytes, vp0);
        load_words<G>(own(n) + F::kOffVPar + tok1 * F::kParBytes, vp1);
#pragma unroll
        for (int y = 0; y < kWith; ++y)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            load_words<G / 2>(base[kHalf ? y : n] + F::kOffV + vt[i] * F::kCodeBytes + r * (2 * G), vw[y][i]);
        // pw: the products' weights, which carry 2^kShift; p: the middles' without it, so that
        // their sums stay as far below float32's largest number as the values do
        const float other = two_to(kIn ? -kIn : kShift);
        float p[4], pw[4];
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float2 x = {s[n][i], s[n][i + 1]};
          const float2 y = ptx::mul2(x, make_float2(other, other));
          p[i] = kIn ? y.x : x.x, p[i + 1] = kIn ? y.y : x.y;
          pw[i] = kIn ? x.x : y.x, pw[i + 1] = kIn ? x.y : y.y;
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float s0 = scale_of(vp0[g]), s1 = scale_of(vp1[g]);
          const float m0 = fmaf(8.f, s0, low_of(vp0[g])), m1 = fmaf(8.f, s1, low_of(vp1[g]));
          float w[4] = {pw[0] * s0, pw[1] * s0, pw[2] * s1, pw[3] * s1};
          if (decltype(masked)::value) {  // what stands in places that are not seen may be anything
            const float mid[4] = {m0, m0, m1, m1};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (!((seen >> (4 * n + e)) & 1u)) w[e] = 0.f;
              else pm[g][e & 1] = fmaf(p[e], mid[e], pm[g][e & 1]);
            }
          } else {
            pm[g][0] = fmaf(p[0], m0, fmaf(p[2], m1, pm[g][0]));
            pm[g][1] = fmaf(p[1], m0, fmaf(p[3], m1, pm[g][1]));
          }
          uint32_t w0[kTerms], w1[kTerms], b2[kTerms][2];
          split_pair<kTerms>(w[0], w[1], w0);
          split_pair<kTerms>(w[2], w[3], w1);
#pragma unroll
          for (int t = 0; t < kTerms; ++t) {
            b2[t][0] = transpose8(w0[t]);
            b2[t][1] = transpose8(w1[t]);
          }
#pragma unroll
          for (int y = 0; y < kWith; ++y) {
            const uint32_t sel = (g & 1) ? 0x7632u : 0x5410u;
            const uint32_t a01 = __byte_perm(vw[y][0][g / 2], vw[y][1][g / 2], sel);
            const uint32_t a23 = __byte_perm(vw[y][2][g / 2], vw[y][3][g / 2], sel);
            uint32_t a[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t x01 = a01 >> (8 * i), x23 = a23 >> (8 * i);
              a[i][0] = codes_first<kTerms>(a01, 8 * i);
              a[i][1] = codes_hi(x01);
              a[i][2] = codes_first<kTerms>(a23, 8 * i);
              a[i][3] = codes_hi(x23);
            }
            // columns 0-3 are the first block's weights, 4-7 the second's
            const uint32_t mine_only = kHalf ? ((r < 4) == (y == 0) ? ~0u : 0u) : ~0u;
#pragma unroll
            for (int t = kTerms - 1; t >= 0; --t) {
              const uint32_t by[2] = {b2[t][0] & mine_only, b2[t][1] & mine_only};
              mma16816(o[g][0], a[0], by);
              mma16816(o[g][1], a[1], by);
            }
          }
#pragma unroll
          for (int t = kTerms - 1; t >= 0; --t) {
            mma16816(o[g][0], minus8, b2[t]);
            mma16816(o[g][1], minus8, b2[t]);
          }
        }
      }
    };
    if (whole) values(std::false_type());
    else values(std::true_type());
    __syncwarp();  // every lane is done with the slot
    fetch(slot);
  }

  // Rows' sums over the lanes that held different keys.
#pragma unroll
  for (int d = 4; d <= 16; d <<= 1) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
#pragma unroll
      for (int g = 0; g < G; ++g) pm[g][e] += __shfl_xor_sync(0xffffffffu, pm[g][e], d);
    }
  }

  // Join the warps, in the rings' memory.
  copies_wait<0>();
  __syncthreads();
  using Row = float[D + 4];
  static_assert(kWarps * kTile * (D + 4 + 2) * 4 <= kWarps * kPairs * 2 * F::kBytes, "join area");
  auto sm_o = reinterpret_cast<Row(*)[kTile]>(ring);
  auto sm_m = reinterpret_cast<float(*)[kTile]>(ring + sizeof(Row) * kTile * kWarps);
  auto sm_l = sm_m + kWarps;
  constexpr int kTo = (kTerms == 1 ? 133 : 129) - kShift;
  if (r == 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sm_m[warp][2 * c + e] = m[e];
      sm_l[warp][2 * c + e] = l[e] * two_to(-kIn);
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      // 2^-kShift brings p back, and another 2^133 (2^129 for 16 n) the codes
      *reinterpret_cast<float4*>(&sm_o[warp][2 * c + e][32 * g + 4 * r]) =
          make_float4(fmaf(o[g][0][e], two_to(kTo), pm[g][e]), fmaf(o[g][0][e + 2], two_to(129 - kShift), pm[g][e]),
                      fmaf(o[g][1][e], two_to(kTo), pm[g][e]), fmaf(o[g][1][e + 2], two_to(129 - kShift), pm[g][e]));
  __syncthreads();
  for (int at = threadIdx.x; at < kRows * D; at += kWarps * 32) {
    const int row = at / D, ch = at % D;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
      for (int col = row; col < kTile; col += kRows) mx = fmaxf(mx, sm_m[w][col]);
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
      for (int y = 0; y < kTile / kRows; ++y) {
        const int col = row + y * kRows;
        const float f = sm_m[w][col] == -INFINITY ? 0.f : ptx::ex2_approx(sm_m[w][col] - mx);
        // (a warp that saw nothing of this row holds zeros, one that saw only NaN a sum of NaN:
        // a row is empty when its sum is 0)
        sum = fmaf(f, sm_l[w][col], sum);
        acc = fmaf(f, sm_o[w][col][ch], acc);
      }
    if (!(begins && ends)) {
      const int64_t part = ((int64_t)ht * P.slots + cta) * 2 + begins;
      RA_BOUNDS(P.t.status, P.part_o != nullptr && part >= 0 && part < (int64_t)P.t.heads_kv * P.tiles * P.slots * 2, 98);
      P.part_o[(part * kTile + row) * D + ch] = acc;
      if (ch == 0) P.part_ml[part * kTile + row] = make_float2(mx, sum);
    } else if (row0 + row < n_rows) {
      const int64_t out = ((int64_t)b * P.heads_q + (int64_t)h * P.group) * P.rows + row0 + row;
      RA_BOUNDS(P.t.status, out >= 0 && out < (int64_t)P.t.batch * P.heads_q * P.rows, 99);
      static_cast<T*>(P.o)[out * D + ch] = (T)(sum == 0.f ? 0.f : acc / sum);
      if (ch == 0 && P.lse != nullptr) P.lse[out] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
    }
  }
  if (!kInRow) break;
  if (ht == 0 && threadIdx.x == 0) {
    if (begins) P.shares[b].x = cta;
    if (ends) P.shares[b].y = cta;
  }
  __syncthreads();  // (the next sequence's fragments and blocks come into the same memory)
  }
}

// Joins the parts of a row, in a fixed order: one CTA a row.  The parts' weights
// 2^(m_s - m) come first, then D/4 lanes read a part's row, each warp every eighth part
// (or every sixteenth half-warp) and the warps' sums are added.  A loop over the parts by
// one thread a channel took 15 us for 64 of them; this takes 3.
constexpr int kJoinWarps = 8;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) kv4_join_kernel(const Kv4AttendParams P) {
  constexpr int kLanes = D / 4;                        // lanes of a part's row
  constexpr int kParts = kJoinWarps * 32 / kLanes;     // parts read at a time
  __shared__ float weight[kMaxSlots];
  __shared__ float red[2][kJoinWarps];
  __shared__ float4 sums[kParts][kLanes];
  cudaGridDependencySynchronize();  // (the parts and their places are written)
  const int unit = blockIdx.x, row = blockIdx.y;  // unit = (b * heads_kv + h) * tiles + tile
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = unit % P.tiles, bh = unit / P.tiles, b = bh / P.t.heads_kv;
  if (tile * kTile + row >= P.group * P.rows) return;
  const int2 share = P.t.batch == 1 ? make_int2(0, P.slots - 1) : P.shares[b];  // (first slot, last slot)
  RA_BOUNDS(P.t.status, b < P.t.batch && share.x >= 0 && share.x <= share.y && share.y < P.slots, 100);
  const int n = share.y - share.x + 1;
  if (n == 1) return;  // (that CTA wrote the row)
  // a slot has two parts: of a sequence that it has the beginning of the second
  const int64_t part0 = ((int64_t)(unit - b * P.t.heads_kv * P.tiles) * P.slots + share.x) * 2;
  auto part_at = [&](int s) { return part0 + (s == 0 ? 1 : 2 * s); };
  const float2* ml = P.part_ml + row;

  float mx = -INFINITY;
  for (int s = threadIdx.x; s < n; s += kJoinWarps * 32) mx = fmaxf(mx, ml[part_at(s) * kTile].x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  if (lane == 0) red[0][warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) mx = fmaxf(mx, red[0][w]);
  float sum = 0.f;
  for (int s = threadIdx.x; s < n; s += kJoinWarps * 32) {
    const float2 x = ml[part_at(s) * kTile];
    const float f = x.x == -INFINITY ? 0.f : ptx::ex2_approx(x.x - mx);
    weight[s] = f;
    sum = fmaf(f, x.y, sum);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) red[1][warp] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) sum += red[1][w];

  const int part = threadIdx.x / kLanes, at = threadIdx.x % kLanes;
  const float4* po = reinterpret_cast<const float4*>(P.part_o + row * D) + at;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = part; s < n; s += kParts) {
    const float f = weight[s];
    const float4 x = po[part_at(s) * (kTile * kLanes)];
    acc.x = fmaf(f, x.x, acc.x);
    acc.y = fmaf(f, x.y, acc.y);
    acc.z = fmaf(f, x.z, acc.z);
    acc.w = fmaf(f, x.w, acc.w);
  }
  sums[part][at] = acc;
  __syncthreads();
  const int64_t out = (int64_t)bh * P.group * P.rows + tile * kTile + row;
  RA_BOUNDS(P.t.status, out >= 0 && out < (int64_t)P.t.batch * P.heads_q * P.rows, 101);
  if (threadIdx.x < D) {
    float y = 0.f;
#pragma unroll
    for (int x = 0; x < kParts; ++x) y += reinterpret_cast<const float*>(sums[x])[threadIdx.x];
    static_cast<T*>(P.o)[out * D + threadIdx.x] = (T)(sum == 0.f ? 0.f : y / sum);
  }
  if (threadIdx.x == 0 && P.lse != nullptr) P.lse[out] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

template <typename T, int D, bool kInRow, bool kHalf>
cudaError_t attend_as(const Kv4AttendParams& prm, cudaStream_t st) {
  constexpr int kTerms = sizeof(T) == 2 ? 1 : 3;
  constexpr int kSmem = kWarps * kPairs * 2 * Kv4Block<D>::kBytes + 32 * 16 * ((D / 32) * kTerms * (kHalf ? 2 : 1) + 1);
  static std::atomic<int> ready[kMaxDevices];
  const char* why = "";
  cudaError_t e = prepare_once(kv4_attend_kernel<T, D, kInRow, kHalf>, ready, kWarps * 32, 0, kSmem, &why);
  if (e != cudaSuccess) return e;
  const unsigned heads = (unsigned)(prm.t.heads_kv * prm.tiles), slots = (unsigned)prm.slots;
  const dim3 grid = prm.t.batch == 1 ? dim3(slots, heads) : dim3(heads, slots);
  kv4_attend_kernel<T, D, kInRow, kHalf><<<grid, kWarps * 32, kSmem, st>>>(prm);
  e = cudaGetLastError();
  if (e != cudaSuccess || (!kInRow && prm.slots == prm.t.batch)) return e;
  // The join's CTAs may be placed while the last of the others still run; they wait for
  // the whole grid's results.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)prm.t.batch * prm.t.heads_kv * prm.tiles), kTile);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv4_join_kernel<T, D>, prm);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_attend(int dtype, int head_dim, const Kv4AttendParams& prm, cudaStream_t stream) {
  auto rows = [&](auto type, auto d, auto in_row) {
    using T = decltype(type);
    constexpr int D = decltype(d)::value;
    constexpr bool kInRow = decltype(in_row)::value;
    return prm.group * prm.rows <= kTile / 2 ? attend_as<T, D, kInRow, true>(prm, stream)
                                             : attend_as<T, D, kInRow, false>(prm, stream);
  };
  auto in_row = [&](auto type, auto d) {
    return prm.in_row != 0 ? rows(type, d, std::true_type()) : rows(type, d, std::false_type());
  };
  auto dim = [&](auto type) {
    return head_dim == 128 ? in_row(type, std::integral_constant<int, 128>())
                           : in_row(type, std::integral_constant<int, 64>());
  };
  return dtype == RA_DTYPE_BF16 ? dim(__nv_bfloat16()) : dim(float());
}

}  // namespace ra
