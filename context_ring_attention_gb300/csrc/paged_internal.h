// The paged key/value cache (include/ra.h, ra_paged_*): its layout, the sequences of a packed
// batch, which keys a run of tokens sees, and the launchers.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ra_internal.h"
#include "rope_internal.h"

namespace ra {

constexpr uint32_t kPagedStatusRange = 1u << 5;  // a page, offset, length or slot out of range
constexpr int kMaxSequences = 4096;              // of a call: their shares are summed in shared memory

// What the calls share: the cache [pages, 2, heads_kv, page_rows, d] and its sequences.
struct PagedTable {
  void* cache;
  const int32_t* page_table;  // [batch, width]
  const int32_t* offset;      // [batch + 1]
  const int32_t* length;      // [batch]
  int64_t width;
  int32_t pages, page_rows, batch, heads_kv, tokens;
  uint32_t* status;
  int32_t few;  // sequences of a launch: kAllRows, or those with up to / more than kFewRows query rows a head
};
enum : int32_t { kAllRows = 0, kFewOnly = 1, kManyOnly = 2 };
constexpr int kFewRows = 16;

struct PagedStrides {  // elements
  int64_t token, head;
};

struct PagedAppendParams {
  PagedTable t;
  RopeTable rope;  // speed nullptr: keys as they are
  int32_t d, heads_q;  // heads_q 0: no queries
  bool wide;
  const int32_t* position;  // [tokens] or nullptr: the slot
  const void *q, *k, *v;
  void* q_out;
  PagedStrides qs, ks, vs, qos;
};

struct PagedAttendParams {
  PagedTable t;
  int32_t heads_q, group, slots;  // slots: CTAs per key/value head at most
  int32_t window, sinks;          // window 0: the whole prefix
  float scale_log2;
  const void* q;
  void* o;
  PagedStrides qs, os;
  float* lse;        // [tokens, heads_q] or nullptr
  int32_t beside;    // a chunk kernel may still run: this one ends after it
  float* part_o;     // [head, slot, 2, kRowsTile, d]
  float2* part_ml;   // [head, slot, 2, kRowsTile]: running maximum (log2 units) and sum
  int4* joins;       // [head, slot]: first query row, rows, last slot of an item cut here (rows 0: none)
};

// An item that share x of the chunk kernel begins and does not end (tokens 0: none).
struct alignas(16) PagedJoin {
  int32_t head, token, tokens, last;  // last: the share that ends it
};

struct PagedChunkParams {
  PagedTable t;
  int32_t heads_q, group;
  int32_t window, sinks;
  int32_t piece;      // rows that are brought at a time: the largest power of two in 16..128 that divides a page
  int32_t rounds;     // shares of a CTA at most
  int32_t row_bytes;
  float scale_log2;
  const void* q;
  void* o;
  PagedStrides qs, os;
  float* lse;        // [tokens, heads_q] or nullptr
  float* part_o;     // [share, 2, tile, d / 4, 128, 4]
  float4* part_ml;   // [share, 2, tile, 128]: running maximum (log2 units), sum, its correction
  PagedJoin* joins;  // [share]
};

struct PagedWeighParams {
  PagedTable t;
  int32_t heads_q, group;
  int32_t window, sinks;
  float scale_log2;
  const void* q;
  PagedStrides qs;
  const float* lse;        // [tokens, heads_q]
  const float* weight_in;  // [batch, heads_kv, weight_width] or nullptr
  float* weight;
  int64_t weight_width;
  int32_t beside;          // as in PagedAttendParams (bf16)
};

// An item that share x of the chunk kernel begins and does not end (last < 0: none).
struct alignas(16) PagedWeighJoin {
  int32_t head, b, key0, last;  // last: the share that ends it
};

struct PagedWeighChunkParams {
  PagedTable t;
  int32_t heads_q, group;
  int32_t window, sinks;
  int32_t piece;  // as in PagedChunkParams
  float scale, scale_log2;
  const void* q;
  PagedStrides qs;
  const float* lse;
  const float* weight_in;
  float* weight;
  int64_t weight_width;
  float* parts;           // [share, 2, 256]
  uint4* extra;           // [head, tiles, 128]: the rows' LSE as bf16 channels
  int32_t* extra_at;      // [batch]: the sequences' first tiles
  int32_t tiles;          // tokens / (128 / group) + batch at most
  PagedWeighJoin* joins;  // [share]
};

struct PagedEvictParams {
  PagedTable t;  // (offset nullptr, tokens 0)
  int32_t d;
  const int32_t* new_table;  // [batch, new_width]
  int64_t new_width;
  const float* weight_in;    // [batch, heads_kv, weight_width]
  float* weight;             // or nullptr
  int64_t weight_width;
  int32_t keep, first, recent;
  int32_t* kept;        // [batch, heads_kv, keep]
  int32_t* new_length;  // [batch]
};

cudaError_t launch_paged_append(int dtype, const PagedAppendParams& prm, int sm_count, cudaStream_t stream);
// beside: the kernel starts while the chunk kernel before it in the stream runs.
cudaError_t launch_paged_rows(int dtype, int head_dim, const PagedAttendParams& prm, bool beside, cudaStream_t stream);
cudaError_t launch_paged_rows_join(int dtype, int head_dim, const PagedAttendParams& prm, cudaStream_t stream);
cudaError_t launch_paged_chunk(int head_dim, const PagedChunkParams& prm, int grid, cudaStream_t stream, const char** why);
cudaError_t launch_paged_chunk_join(int head_dim, const PagedChunkParams& prm, int grid, cudaStream_t stream);
cudaError_t launch_paged_weigh_rows(int dtype, int head_dim, const PagedWeighParams& prm, int sm_count,
                                    cudaStream_t stream);
cudaError_t launch_paged_weigh_chunk(int head_dim, const PagedWeighChunkParams& prm, int grid, cudaStream_t stream,
                                     const char** why);
cudaError_t launch_paged_weigh_join(const PagedWeighChunkParams& prm, int grid, cudaStream_t stream);
cudaError_t launch_paged_evict(int dtype, const PagedEvictParams& prm, int sm_count, cudaStream_t stream);

constexpr int kMaxChunkSequences = 2048;  // of a call of the chunk kernels (shared memory)
constexpr int kMaxRounds = 8;
constexpr int64_t kRoundBytes = int64_t(44) << 20;  // of keys and values that a round walks, a third of the L2

// Tensor maps of the chunk kernels (paged_maps.cu): rows of d bf16 in boxes of 64 channels by
// `box` rows; a packed tensor [tokens, heads, d] in boxes of 64 channels, `group` heads and
// `box` tokens.  128-byte swizzle; beyond the end zeros.
bool encode_rows(void* map, const void* base, int64_t rows, int d, int box);
bool encode_packed(void* map, const void* base, const PagedStrides& s, int64_t tokens, int64_t heads, int d, int group,
                   int box);

constexpr int kRowsTile = 16;   // query rows of an item of the row kernels
constexpr int kRowsBlock = 16;  // keys of a block

#ifdef __CUDACC__
// A kernel of a call behind another one's: its CTAs come to the SMs while the other kernel ends,
// and wait there (after_previous) until all of it is done and can be read.  The other kernel lets
// them come by next_may_come.
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = dim3((unsigned)threads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  config.attrs = &attr;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, args...);
}
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void next_may_come() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A sequence of the batch.  Offsets that do not rise within 0..tokens, or a length that is
// negative, smaller than the new tokens' count or beyond the page table: reported, and the
// sequence has no tokens and no keys.
struct PagedSeq {
  int token0, count, length;
  __device__ __forceinline__ int slot0() const { return length - count; }
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedTable& t, int b) {
  const int a = t.offset != nullptr ? __ldg(t.offset + b) : 0, e = t.offset != nullptr ? __ldg(t.offset + b + 1) : 0;
  const int n = __ldg(t.length + b);
  if (a < 0 || e < a || e > t.tokens || n < e - a || n > t.width * t.page_rows) {
    atomicOr(t.status, kPagedStatusRange);
    return {0, 0, 0};
  }
  return {a, e - a, n};
}

// Whether a launch takes a sequence.
__device__ __forceinline__ bool paged_mine(const PagedTable& t, const PagedSeq& q, int group) {
  return t.few == kAllRows || (q.count * group <= kFewRows) == (t.few == kFewOnly);
}

// Page of a sequence's entry; -1, and a report, where the table names none.
__device__ __forceinline__ int paged_page(const PagedTable& t, int b, int entry) {
  const int page = __ldg(t.page_table + b * t.width + entry);
  if (page >= 0 && page < t.pages) return page;
  atomicOr(t.status, kPagedStatusRange);
  return -1;
}

// Row of the cache, as [rows, d], that holds a page's row (which: 0 keys, 1 values).
__device__ __forceinline__ int64_t paged_row(const PagedTable& t, int page, int which, int head, int r) {
  return (((int64_t)page * 2 + which) * t.heads_kv + head) * t.page_rows + r;
}

// The slots that some token of the slots [s0, s1] sees: [0, sink) and [lo, hi), sink <= lo.
struct PagedSpan {
  int sink, lo, hi;
  __device__ __forceinline__ bool holds(int j) const { return j < hi && (j >= lo || j < sink); }
};
__device__ __forceinline__ PagedSpan paged_span(int window, int sinks, int s0, int s1) {
  PagedSpan sp;
  sp.hi = s1 + 1 > 0 ? s1 + 1 : 0;
  sp.lo = window > 0 ? max(0, s0 - window + 1) : 0;
  sp.sink = min(min(sinks, sp.lo), sp.hi);
  return sp;
}
// The blocks of kB slots that a span touches, in order: the k-th is block at(k).
template <int kB>
struct PagedBlocks {
  int head, skip, n;  // blocks of the sinks, then block head + skip on
  __device__ __forceinline__ explicit PagedBlocks(const PagedSpan& sp) {
    const int last = (sp.hi + kB - 1) / kB;
    int first = sp.lo / kB;
    head = (sp.sink + kB - 1) / kB;
    if (sp.sink > 0 && head >= first) head = first = 0;  // the sinks' blocks reach the window's
    skip = first - head;
    n = last - skip;
  }
  __device__ __forceinline__ int at(int k) const { return k < head ? k : k + skip; }
};
// Whether token slot s sees slot j.
__device__ __forceinline__ bool paged_sees(int window, int sinks, int s, int j) {
  return j <= s && (window == 0 || j > s - window || j < sinks);
}
#endif

}  // namespace ra
