// C ABI of the paged key/value cache (include/ra.h, ra_paged_*): argument checks, handles and
// the choice of kernels.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>
#include <vector>

#include "api_internal.h"
#include "paged_internal.h"

struct ra_paged_s {
  ra_paged_problem prob;
  int device = -1;
  int sm_count = 0;
  uint32_t* d_status = nullptr;
  // Stream of the handle's own allocation and free (see ra_plan_s::mem_stream).
  cudaStream_t mem_stream = nullptr;
  std::vector<ra::StreamMark> marks;
};

namespace {

ra_status fail(ra_status s, const char* fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  ra::set_last_error(msg);
  return s;
}
ra_status ok() {
  ra::set_last_error("");
  return RA_OK;
}

constexpr int64_t kMaxPositions = int64_t(1) << 30;  // of a sequence: slot arithmetic stays in 32 bits
constexpr int kMaxSlots = 512;                       // CTAs of a key/value head
// Of a sequence in the chunk kernels, so that an item, 2^18 tiles at most, ends well within their wait budget.
constexpr int64_t kMaxChunkSlots = int64_t(1) << 25, kMaxChunkTiles = int64_t(1) << 18;

ra_status validate(const ra_paged_problem* p) {
  if (p->pages < 1 || p->heads_q < 1 || p->heads_kv < 1 || p->head_dim < 1)
    return fail(RA_ERR_INVALID_ARG, "pages, heads and head_dim must be >= 1");
  if (p->page_rows < 16 || p->page_rows > 65536 || p->page_rows % 16)
    return fail(RA_ERR_INVALID_ARG, "page_rows must be a multiple of 16 in 16..65536 (got %d)", p->page_rows);
  if (p->heads_q % p->heads_kv) return fail(RA_ERR_INVALID_ARG, "heads_q %% heads_kv != 0");
  if (p->dtype != RA_DTYPE_F32 && p->dtype != RA_DTYPE_BF16) return fail(RA_ERR_INVALID_ARG, "unknown dtype %d", p->dtype);
  if (p->window < 0 || p->sinks < 0) return fail(RA_ERR_INVALID_ARG, "window and sinks must be >= 0");
  // (LSE / scale and the scores stay finite)
  if (!(p->scale == 0.f || (p->scale >= 0x1p-100f && p->scale <= 0x1p100f)))
    return fail(RA_ERR_INVALID_ARG, "scale must be 0 or in 2^-100..2^100");
  if (p->head_dim != 64 && p->head_dim != 128)
    return fail(RA_ERR_UNSUPPORTED, "the paged cache needs head_dim 64 or 128 (got %d)", p->head_dim);
  if (p->heads_kv > 65535) return fail(RA_ERR_UNSUPPORTED, "more than 65535 key/value heads");
  if (p->pages > INT32_MAX / 2 / p->page_rows / p->heads_kv)
    return fail(RA_ERR_UNSUPPORTED, "a cache of more than 2^31-1 rows");
  return RA_OK;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
int64_t elem_bytes(const ra_paged_problem& pb) { return pb.dtype == RA_DTYPE_BF16 ? 2 : 4; }

// The checks that every launch shares; n16 tensors need 16-byte alignment, n4 tables 4.
ra_status check_call(const ra_paged_s* kv, int64_t batch, int64_t tokens, int64_t width, const void* const* t16, int n16,
                     const void* const* t4, int n4, cudaStream_t st) {
  for (int i = 0; i < n16; ++i)
    if (!aligned(t16[i], 16)) return fail(RA_ERR_INVALID_ARG, "pointer %p is not 16-byte aligned", t16[i]);
  for (int i = 0; i < n4; ++i)
    if (!aligned(t4[i], 4)) return fail(RA_ERR_INVALID_ARG, "pointer %p is not 4-byte aligned", t4[i]);
  const ra_paged_problem& pb = kv->prob;
  if (batch < 1 || tokens < 1 || width < 1) return fail(RA_ERR_INVALID_ARG, "batch, tokens and table_width must be >= 1");
  if (width > kMaxPositions / pb.page_rows) return fail(RA_ERR_UNSUPPORTED, "table_width * page_rows above 2^30");
  if (batch > ra::kMaxSequences) return fail(RA_ERR_UNSUPPORTED, "more than %d sequences", ra::kMaxSequences);
  if (tokens > (int64_t(1) << 30) / (pb.heads_q + 2 * (int64_t)pb.heads_kv))
    return fail(RA_ERR_UNSUPPORTED, "tokens * (heads_q + 2 heads_kv) above 2^30");
  if (kv->device < 0) return fail(RA_ERR_NO_DEVICE, "the handle was created without a CUDA device");
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess || cur != kv->device)
    return fail(RA_ERR_INVALID_ARG, "current device %d differs from the handle's device %d", cur, kv->device);
  const ra_status s = ra::check_on_current_device(t16, n16, st);
  return s != RA_OK ? s : ra::check_on_current_device(t4, n4, st);
}

// Strides (token, head) of a packed tensor: rows at 16-byte boundaries, and in a tensor that is
// written no two rows in one place.
ra_status strides_of(const ra_paged_s* kv, const char* what, const int64_t* s, int64_t tokens, int64_t heads, bool written,
                     ra::PagedStrides* out) {
  if (s == nullptr) return fail(RA_ERR_INVALID_ARG, "%s: null strides", what);
  *out = {s[0], s[1]};
  const int64_t d = kv->prob.head_dim, e = elem_bytes(kv->prob), most = int64_t(1) << 38;
  if (s[0] < 0 || s[1] < 0 || s[0] > most || s[1] > most)
    return fail(RA_ERR_INVALID_ARG, "%s: a stride is negative or beyond 2^38 elements", what);
  if (s[0] * e % 16 || s[1] * e % 16) return fail(RA_ERR_INVALID_ARG, "%s: strides are not multiples of 16 bytes", what);
  if (!written) return RA_OK;
  const bool heads_inside = s[1] <= s[0];
  const int64_t in = heads_inside ? s[1] : s[0], in_n = heads_inside ? heads : tokens;
  const int64_t far = heads_inside ? s[0] : s[1], far_n = heads_inside ? tokens : heads;
  if ((in_n > 1 && in < d) || (far_n > 1 && far < (in_n - 1) * in + d))
    return fail(RA_ERR_INVALID_ARG, "%s: rows overlap in memory", what);
  return RA_OK;
}

ra::PagedTable table_of(const ra_paged_s* kv, const void* cache, int64_t batch, int64_t tokens, const int32_t* page_table,
                        int64_t width, const int32_t* offset, const int32_t* length) {
  ra::PagedTable t{};
  t.cache = const_cast<void*>(cache);
  t.page_table = page_table;
  t.offset = offset;
  t.length = length;
  t.width = width;
  t.pages = (int32_t)kv->prob.pages;
  t.page_rows = kv->prob.page_rows;
  t.batch = (int32_t)batch;
  t.heads_kv = kv->prob.heads_kv;
  t.tokens = (int32_t)tokens;
  t.status = kv->d_status;
  return t;
}

ra_status launched(ra_paged_s* kv, cudaError_t e, const char* what, cudaStream_t st) {
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  const ra_status s = ra::mark_use(&kv->marks, st);
  return s != RA_OK ? s : ok();
}

// CTAs per key/value head of the row kernels: as many as the GPU holds at once (two an SM, float32
// of 64 channels four: one token of 16 sequences of 4k 56 us with two, 46 with four), and no more than the largest number of shares or items that these sizes can make.  Beside a chunk
// kernel three times as many: it leaves them only some of the SMs, and more as it ends.
int row_slots(const ra_paged_s* kv, int64_t batch, int64_t tokens, int64_t width, bool beside) {
  const ra_paged_problem& pb = kv->prob;
  const int64_t tiles = tokens * (pb.heads_q / pb.heads_kv) / ra::kRowsTile + std::min(batch, tokens);
  int64_t blocks = width * pb.page_rows / ra::kRowsBlock;
  if (pb.window > 0 && pb.window < kMaxPositions && pb.sinks < kMaxPositions)
    blocks = std::min(blocks, (pb.window + ra::kRowsTile + pb.sinks) / ra::kRowsBlock + 3);
  const int64_t shares = tiles * blocks / (pb.dtype == RA_DTYPE_BF16 ? 8 : 4);  // as the kernels cut them (tiles below 2^30, blocks up to 2^26)
  const int64_t sms = kv->sm_count > 0 ? kv->sm_count : 148;
  const int64_t per_sm = beside ? 6 : pb.dtype == RA_DTYPE_F32 && pb.head_dim == 64 ? 4 : 2;
  return (int)std::max<int64_t>(1, std::min({std::max(shares, tiles), per_sm * sms / pb.heads_kv, (int64_t)kMaxSlots}));
}

// Shares of a CTA of the chunk kernel at most: where more than one item reads a sequence's keys,
// and these may be more than a round's (paged_chunk_sm103.cu).
int chunk_rounds(const ra_paged_s* kv, int64_t batch, int64_t tokens, int64_t width) {
  const ra_paged_problem& pb = kv->prob;
  if (tokens <= 2 * (128 / (pb.heads_q / pb.heads_kv))) return 1;
  const int64_t bytes = std::min(batch, tokens) * width * pb.page_rows * pb.heads_kv * 4 / 1024 * pb.head_dim;  // KiB
  return (int)std::max<int64_t>(1, std::min<int64_t>(ra::kMaxRounds, bytes / (ra::kRoundBytes >> 10)));
}

// Which kernels a call takes.  A sequence with up to 16 query rows a head belongs to the row
// kernels, which read its keys at the rate of HBM; one with more to the chunk kernels, whose query
// tiles have 128 rows.  The counts are on the device: where a call may have sequences of both
// kinds it launches both, each leaving out the other's sequences.  A batch whose largest sequence can
// have 128 rows at most (if every sequence has a token) takes the row kernels alone, which walk a
// sequence's keys once for 16 rows: the second kernel and its join cost 10 us, more than the walks where
// the keys are few.  Attention and weights in us, 32 and 8 heads, D 128, row kernels alone and both:
//   2 sequences of 20 rows over 1k 12 and 8, 23 and 13; over 8k 26 and 19, 34 and 19; over 32k 86 and 53, 77 and 41;
//   2 of 64 rows over 1k 18 and 13, 24 and 14; over 8k 36 and 36, 35 and 20; over 32k 162 and 108, 77 and 45;
//   5 of 20 rows over 1k 18 and 10, 27 and 14; over 8k 45 and 35, 61 and 30; over 32k 199 and 121, 140 and 80.
// The rule does not see the keys' number, and is the wrong one over long prefixes.
struct Route {
  bool rows, chunks;
};
Route route_of(const ra_paged_s* kv, int64_t batch, int64_t tokens, int64_t width) {
  const ra_paged_problem& pb = kv->prob;
  const int64_t group = pb.heads_q / pb.heads_kv;
  if (pb.dtype != RA_DTYPE_BF16 || group > 128 || batch > ra::kMaxChunkSequences || width * pb.page_rows > kMaxChunkSlots ||
      tokens / (128 / group) > kMaxChunkTiles)
    return {true, false};
  if (batch == 1) return {tokens * group <= ra::kFewRows, tokens * group > ra::kFewRows};
  return {true, (tokens - batch + 1) * group > 128};
}

int64_t chunk_scratch(const ra_paged_s* kv, int64_t shares) {
  const int64_t rows = shares * 2 * 2 * 128;
  return rows * (kv->prob.head_dim * 4 + 16) + shares * 16;
}
// Scratch of the weights' chunk kernel: 16 bytes a row of every query tile, a sum per key for two
// parts of every share, the joins, the sequences' first tiles.
int64_t weigh_tiles(const ra_paged_s* kv, int64_t batch, int64_t tokens) {
  return tokens / (128 / (kv->prob.heads_q / kv->prob.heads_kv)) + batch;
}
int64_t weigh_scratch(const ra_paged_s* kv, int64_t batch, int64_t tokens, int64_t grid) {
  return kv->prob.heads_kv * weigh_tiles(kv, batch, tokens) * 128 * 16 + grid * (2 * 256 * 4 + 16) + (batch + 3) / 4 * 16;
}
// The largest power of two in 16..128 that divides a page.
int piece_of(const ra_paged_problem& pb) {
  int piece = 16;
  while (piece < 128 && pb.page_rows % (2 * piece) == 0) piece *= 2;
  return piece;
}
int chunk_grid(const ra_paged_s* kv) { return kv->sm_count > 0 ? kv->sm_count : 148; }

int64_t rows_scratch(const ra_paged_s* kv, int slots) {
  if (slots == 1) return 0;
  const int64_t parts = (int64_t)kv->prob.heads_kv * slots * 2;
  return parts * ra::kRowsTile * (kv->prob.head_dim + 2) * 4 + (int64_t)kv->prob.heads_kv * slots * 16;
}

ra_status check_sizes(const ra_paged_s* kv, int64_t batch, int64_t tokens, int64_t width) {
  if (batch < 1 || tokens < 1 || width < 1) return fail(RA_ERR_INVALID_ARG, "batch, tokens and table_width must be >= 1");
  const ra_paged_problem& pb = kv->prob;
  if (width > kMaxPositions / pb.page_rows) return fail(RA_ERR_UNSUPPORTED, "table_width * page_rows above 2^30");
  if (batch > ra::kMaxSequences) return fail(RA_ERR_UNSUPPORTED, "more than %d sequences", ra::kMaxSequences);
  if (tokens > (int64_t(1) << 30) / (pb.heads_q + 2 * (int64_t)pb.heads_kv))
    return fail(RA_ERR_UNSUPPORTED, "tokens * (heads_q + 2 heads_kv) above 2^30");
  return RA_OK;
}

}  // namespace

extern "C" {

ra_status ra_paged_plan(const ra_paged_problem* prob, ra_paged_t* out) {
  if (prob == nullptr || out == nullptr) return fail(RA_ERR_INVALID_ARG, "null argument");
  *out = nullptr;
  ra_status s = validate(prob);
  if (s != RA_OK) return s;
  ra_paged_s* kv = new (std::nothrow) ra_paged_s();
  if (kv == nullptr) return fail(RA_ERR_UNSUPPORTED, "out of host memory");
  kv->prob = *prob;
  if (kv->prob.scale == 0.f) kv->prob.scale = 1.0f / std::sqrt((float)prob->head_dim);
  int dev = -1, count = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && cudaGetDeviceCount(&count) == cudaSuccess && count > 0) {
    kv->device = dev;
    cudaDeviceGetAttribute(&kv->sm_count, cudaDevAttrMultiProcessorCount, dev);
    cudaError_t e = cudaStreamCreateWithFlags(&kv->mem_stream, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaMallocAsync(reinterpret_cast<void**>(&kv->d_status), 256, kv->mem_stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(kv->d_status, 0, 256, kv->mem_stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(kv->mem_stream);
    if (e != cudaSuccess) {
      const ra_status f = fail(RA_ERR_CUDA, "cache handle: %s", cudaGetErrorString(e));
      ra_paged_destroy(kv);
      return f;
    }
  } else {
    cudaGetLastError();  // host-only handle
  }
  *out = kv;
  return ok();
}

ra_status ra_paged_destroy(ra_paged_t kv) {
  if (kv == nullptr) return RA_OK;
  if (kv->device >= 0) {
    int cur = -1;
    cudaGetDevice(&cur);
    if (cur != kv->device) cudaSetDevice(kv->device);
    if (kv->mem_stream != nullptr) {
      for (const ra::StreamMark& m : kv->marks) cudaStreamWaitEvent(kv->mem_stream, m.done, 0);
      if (kv->d_status != nullptr) cudaFreeAsync(kv->d_status, kv->mem_stream);
      cudaStreamDestroy(kv->mem_stream);  // released once its queued free has run
    }
    for (const ra::StreamMark& m : kv->marks) cudaEventDestroy(m.done);
    cudaGetLastError();
    if (cur >= 0 && cur != kv->device) cudaSetDevice(cur);
  }
  delete kv;
  return RA_OK;
}

ra_status ra_paged_append(ra_paged_t kv, ra_rope_t rope, void* cache, int64_t batch, int64_t tokens, const void* k,
                          const int64_t* k_strides, const void* v, const int64_t* v_strides, const void* q,
                          const int64_t* q_strides, void* q_out, const int64_t* q_out_strides,
                          const int32_t* page_table, int64_t table_width, const int32_t* offset, const int32_t* length,
                          const int32_t* position, void* stream) {
  if (kv == nullptr) return fail(RA_ERR_INVALID_ARG, "null handle");
  if (cache == nullptr || k == nullptr || v == nullptr || page_table == nullptr || offset == nullptr || length == nullptr)
    return fail(RA_ERR_INVALID_ARG, "null pointer");
  if ((q == nullptr) != (q_out == nullptr)) return fail(RA_ERR_INVALID_ARG, "q and q_out go together");
  const ra_paged_problem& pb = kv->prob;
  if (rope == nullptr && q != nullptr) return fail(RA_ERR_INVALID_ARG, "queries are rotated: a rotation is needed");
  if (rope == nullptr && position != nullptr) return fail(RA_ERR_INVALID_ARG, "positions without a rotation");
  if (rope != nullptr && (rope->prob.dtype != pb.dtype || rope->prob.head_dim != pb.head_dim))
    return fail(RA_ERR_INVALID_ARG, "the rotation's dtype and head_dim differ from the cache's");
  if (rope != nullptr && rope->device != kv->device)
    return fail(RA_ERR_INVALID_ARG, "the rotation belongs to device %d, the cache to %d", rope->device, kv->device);
  ra::PagedAppendParams prm{};
  ra_status s = strides_of(kv, "k", k_strides, tokens, pb.heads_kv, false, &prm.ks);
  if (s == RA_OK) s = strides_of(kv, "v", v_strides, tokens, pb.heads_kv, false, &prm.vs);
  if (s == RA_OK && q != nullptr) s = strides_of(kv, "q", q_strides, tokens, pb.heads_q, false, &prm.qs);
  if (s == RA_OK && q != nullptr) s = strides_of(kv, "q_out", q_out_strides, tokens, pb.heads_q, true, &prm.qos);
  if (s != RA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const void* t16[] = {cache, k, v, q, q_out};
  const void* t4[] = {page_table, offset, length, position};
  s = check_call(kv, batch, tokens, table_width, t16, 5, t4, 4, st);
  if (s != RA_OK) return s;
  prm.t = table_of(kv, cache, batch, tokens, page_table, table_width, offset, length);
  prm.d = pb.head_dim;
  prm.heads_q = q != nullptr ? pb.heads_q : 0;
  prm.rope = {nullptr, 1.0f, pb.head_dim, 0};
  if (rope != nullptr) {
    const ra_rope_problem& rp = rope->prob;
    prm.rope = {rope->d_speed, rp.amplitude == 0.0 ? 1.0f : (float)rp.amplitude, rp.rotary_dim, rp.interleaved};
  }
  prm.wide = ra::rope_wide(pb.dtype, pb.head_dim, prm.rope.rot);
  prm.position = position;
  prm.q = q;
  prm.k = k;
  prm.v = v;
  prm.q_out = q_out;
  const cudaError_t e = ra::launch_paged_append(pb.dtype, prm, kv->sm_count, st);
  if (e == cudaSuccess && rope != nullptr) s = ra::mark_use(&rope->marks, st);
  return s != RA_OK ? s : launched(kv, e, "cache append launch", st);
}

ra_status ra_paged_attend_scratch_size(ra_paged_t kv, int64_t batch, int64_t tokens, int64_t table_width, int64_t* bytes) {
  if (kv == nullptr || bytes == nullptr) return fail(RA_ERR_INVALID_ARG, "null argument");
  const ra_status s = check_sizes(kv, batch, tokens, table_width);
  if (s != RA_OK) return s;
  const Route route = route_of(kv, batch, tokens, table_width);
  *bytes = 0;
  if (route.chunks) *bytes += chunk_scratch(kv, (int64_t)chunk_grid(kv) * chunk_rounds(kv, batch, tokens, table_width));
  if (route.rows) *bytes += rows_scratch(kv, row_slots(kv, batch, tokens, table_width, route.chunks));
  return ok();
}

ra_status ra_paged_attend(ra_paged_t kv, const void* cache, int64_t batch, int64_t tokens, const void* q,
                          const int64_t* q_strides, const int32_t* page_table, int64_t table_width,
                          const int32_t* offset, const int32_t* length, void* o, const int64_t* o_strides, float* lse,
                          float* scratch, void* stream) {
  if (kv == nullptr) return fail(RA_ERR_INVALID_ARG, "null handle");
  if (cache == nullptr || q == nullptr || page_table == nullptr || offset == nullptr || length == nullptr || o == nullptr)
    return fail(RA_ERR_INVALID_ARG, "null pointer");
  const ra_paged_problem& pb = kv->prob;
  ra_status s = check_sizes(kv, batch, tokens, table_width);
  if (s != RA_OK) return s;
  ra::PagedAttendParams prm{};
  s = strides_of(kv, "q", q_strides, tokens, pb.heads_q, false, &prm.qs);
  if (s == RA_OK) s = strides_of(kv, "o", o_strides, tokens, pb.heads_q, true, &prm.os);
  if (s != RA_OK) return s;
  if ((tokens > 1 && prm.qs.token == 0) || (pb.heads_q > 1 && prm.qs.head == 0))
    return fail(RA_ERR_INVALID_ARG, "q: rows lie in one place");
  const Route route = route_of(kv, batch, tokens, table_width);
  const int slots = route.rows ? row_slots(kv, batch, tokens, table_width, route.chunks) : 1;
  const bool parts = route.chunks || slots > 1;
  if (parts && scratch == nullptr)
    return fail(RA_ERR_INVALID_ARG, "null scratch (ra_paged_attend_scratch_size bytes are needed)");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const void* t16[] = {cache, q, o, parts ? scratch : nullptr};
  const void* t4[] = {page_table, offset, length, lse};
  s = check_call(kv, batch, tokens, table_width, t16, 4, t4, 4, st);
  if (s != RA_OK) return s;
  prm.t = table_of(kv, cache, batch, tokens, page_table, table_width, offset, length);
  const int grid = chunk_grid(kv);
  ra::PagedChunkParams c{};
  if (route.chunks) {
    c.t = prm.t;
    c.t.few = route.rows ? ra::kManyOnly : ra::kAllRows;
    c.heads_q = pb.heads_q;
    c.group = pb.heads_q / pb.heads_kv;
    c.window = (int32_t)std::min(pb.window, kMaxPositions);
    c.sinks = pb.window > 0 ? (int32_t)std::min(pb.sinks, kMaxPositions) : 0;
    c.piece = piece_of(pb);
    c.rounds = chunk_rounds(kv, batch, tokens, table_width);
    c.row_bytes = pb.head_dim * 2;
    c.scale_log2 = pb.scale * 1.4426950408889634f;
    c.q = q;
    c.o = o;
    c.qs = prm.qs;
    c.os = prm.os;
    c.lse = lse;
    const int64_t shares = (int64_t)grid * c.rounds, n = shares * 2 * 2 * 128;
    c.part_o = scratch;
    c.part_ml = reinterpret_cast<float4*>(scratch + n * pb.head_dim);
    c.joins = reinterpret_cast<ra::PagedJoin*>(c.part_ml + n);
    scratch += chunk_scratch(kv, shares) / 4;
  }
  if (route.rows) {
    if (route.chunks) prm.t.few = ra::kFewOnly;
    prm.beside = route.chunks;
    prm.heads_q = pb.heads_q;
    prm.group = pb.heads_q / pb.heads_kv;
    prm.slots = slots;
    prm.window = (int32_t)std::min(pb.window, kMaxPositions);
    prm.sinks = pb.window > 0 ? (int32_t)std::min(pb.sinks, kMaxPositions) : 0;
    prm.scale_log2 = pb.scale * 1.4426950408889634f;
    prm.q = q;
    prm.o = o;
    prm.lse = lse;
    if (slots > 1) {
      const int64_t n = (int64_t)pb.heads_kv * slots * 2;
      prm.part_o = scratch;
      prm.part_ml = reinterpret_cast<float2*>(scratch + n * ra::kRowsTile * pb.head_dim);
      prm.joins = reinterpret_cast<int4*>(prm.part_ml + n * ra::kRowsTile);
    }
  }
  const char* why = "";
  cudaError_t e = cudaSuccess;
  if (route.chunks) e = ra::launch_paged_chunk(pb.head_dim, c, grid, st, &why);
  if (e == cudaSuccess && route.rows) e = ra::launch_paged_rows(pb.dtype, pb.head_dim, prm, route.chunks, st);
  if (e == cudaSuccess && route.chunks) e = ra::launch_paged_chunk_join(pb.head_dim, c, grid, st);
  if (e == cudaSuccess && route.rows) e = ra::launch_paged_rows_join(pb.dtype, pb.head_dim, prm, st);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "cache attention launch: %s %s", cudaGetErrorString(e), why);
  return launched(kv, e, "cache attention launch", st);
}

ra_status ra_paged_weigh_scratch_size(ra_paged_t kv, int64_t batch, int64_t tokens, int64_t table_width, int64_t* bytes) {
  if (kv == nullptr || bytes == nullptr) return fail(RA_ERR_INVALID_ARG, "null argument");
  const ra_status s = check_sizes(kv, batch, tokens, table_width);
  if (s != RA_OK) return s;
  *bytes = route_of(kv, batch, tokens, table_width).chunks ? weigh_scratch(kv, batch, tokens, chunk_grid(kv)) : 0;
  return ok();
}

ra_status ra_paged_weigh(ra_paged_t kv, const void* cache, int64_t batch, int64_t tokens, const void* q,
                         const int64_t* q_strides, const float* lse, const int32_t* page_table, int64_t table_width,
                         const int32_t* offset, const int32_t* length, const float* weight_in, float* weight,
                         int64_t weight_width, float* scratch, void* stream) {
  if (kv == nullptr) return fail(RA_ERR_INVALID_ARG, "null handle");
  if (cache == nullptr || q == nullptr || lse == nullptr || page_table == nullptr || offset == nullptr ||
      length == nullptr || weight == nullptr)
    return fail(RA_ERR_INVALID_ARG, "null pointer");
  if (weight_width < 1 || weight_width > kMaxPositions)
    return fail(RA_ERR_INVALID_ARG, "weight_width must be in 1..2^30");
  const ra_paged_problem& pb = kv->prob;
  ra_status s = check_sizes(kv, batch, tokens, table_width);
  if (s != RA_OK) return s;
  ra::PagedWeighParams prm{};
  s = strides_of(kv, "q", q_strides, tokens, pb.heads_q, false, &prm.qs);
  if (s != RA_OK) return s;
  if ((tokens > 1 && prm.qs.token == 0) || (pb.heads_q > 1 && prm.qs.head == 0))
    return fail(RA_ERR_INVALID_ARG, "q: rows lie in one place");
  const Route route = route_of(kv, batch, tokens, table_width);
  if (route.chunks && scratch == nullptr)
    return fail(RA_ERR_INVALID_ARG, "null scratch (ra_paged_weigh_scratch_size bytes are needed)");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const void* t16[] = {cache, q, route.chunks ? scratch : nullptr};
  const void* t4[] = {page_table, offset, length, lse, weight_in, weight};
  s = check_call(kv, batch, tokens, table_width, t16, 3, t4, 6, st);
  if (s != RA_OK) return s;
  prm.t = table_of(kv, cache, batch, tokens, page_table, table_width, offset, length);
  ra::PagedWeighChunkParams c{};
  const int grid = chunk_grid(kv);
  if (route.chunks) {
    c.t = prm.t;
    c.t.few = route.rows ? ra::kManyOnly : ra::kAllRows;
    c.heads_q = pb.heads_q;
    c.group = pb.heads_q / pb.heads_kv;
    c.window = (int32_t)std::min(pb.window, kMaxPositions);
    c.sinks = pb.window > 0 ? (int32_t)std::min(pb.sinks, kMaxPositions) : 0;
    c.piece = piece_of(pb);
    c.scale = pb.scale;
    c.scale_log2 = pb.scale * 1.4426950408889634f;
    c.q = q;
    c.qs = prm.qs;
    c.lse = lse;
    c.weight_in = weight_in;
    c.weight = weight;
    c.weight_width = weight_width;
    c.tiles = (int32_t)weigh_tiles(kv, batch, tokens);
    c.extra = reinterpret_cast<uint4*>(scratch);
    c.parts = scratch + (int64_t)pb.heads_kv * c.tiles * 128 * 4;
    c.joins = reinterpret_cast<ra::PagedWeighJoin*>(c.parts + (int64_t)grid * 2 * 256);
    c.extra_at = reinterpret_cast<int32_t*>(c.joins + grid);
    prm.t.few = ra::kFewOnly;
    prm.beside = 1;
  }
  prm.heads_q = pb.heads_q;
  prm.group = pb.heads_q / pb.heads_kv;
  prm.window = (int32_t)std::min(pb.window, kMaxPositions);
  prm.sinks = pb.window > 0 ? (int32_t)std::min(pb.sinks, kMaxPositions) : 0;
  prm.scale_log2 = pb.scale * 1.4426950408889634f;
  prm.q = q;
  prm.lse = lse;
  prm.weight_in = weight_in;
  prm.weight = weight;
  prm.weight_width = weight_width;
  const char* why = "";
  cudaError_t e = cudaSuccess;
  if (route.chunks) e = ra::launch_paged_weigh_chunk(pb.head_dim, c, grid, st, &why);
  if (e == cudaSuccess && route.rows) e = ra::launch_paged_weigh_rows(pb.dtype, pb.head_dim, prm, kv->sm_count, st);
  if (e == cudaSuccess && route.chunks) e = ra::launch_paged_weigh_join(c, grid, st);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "cache weights launch: %s %s", cudaGetErrorString(e), why);
  return launched(kv, e, "cache weights launch", st);
}

ra_status ra_paged_evict(ra_paged_t kv, void* cache, int64_t batch, const int32_t* page_table, int64_t table_width,
                         const int32_t* length, const float* weight_in, float* weight, int64_t weight_width,
                         int64_t keep, int64_t first, int64_t recent, const int32_t* new_table, int64_t new_width,
                         int32_t* kept, int32_t* new_length, void* stream) {
  if (kv == nullptr) return fail(RA_ERR_INVALID_ARG, "null handle");
  if (cache == nullptr || page_table == nullptr || length == nullptr || weight_in == nullptr || new_table == nullptr ||
      kept == nullptr || new_length == nullptr)
    return fail(RA_ERR_INVALID_ARG, "null pointer");
  if (keep < 1 || keep > kMaxPositions) return fail(RA_ERR_INVALID_ARG, "keep must be in 1..2^30");
  if (first < 0 || recent < 0 || first > keep || recent > keep - first)
    return fail(RA_ERR_INVALID_ARG, "first and recent must be >= 0, and no more than keep together");
  if (weight_width < 1 || weight_width > kMaxPositions)
    return fail(RA_ERR_INVALID_ARG, "weight_width must be in 1..2^30");
  const ra_paged_problem& pb = kv->prob;
  if (new_width < 1 || new_width > kMaxPositions / pb.page_rows)
    return fail(RA_ERR_INVALID_ARG, "new_width must be >= 1, and new_width * page_rows at most 2^30");
  if (new_length == length) return fail(RA_ERR_INVALID_ARG, "new_length may not be length");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const void* t16[] = {cache};
  const void* t4[] = {page_table, length, weight_in, weight, new_table, kept, new_length};
  const ra_status s = check_call(kv, batch, 1, table_width, t16, 1, t4, 7, st);
  if (s != RA_OK) return s;
  ra::PagedEvictParams prm{};
  prm.t = table_of(kv, cache, batch, 0, page_table, table_width, nullptr, length);
  prm.d = pb.head_dim;
  prm.new_table = new_table;
  prm.new_width = new_width;
  prm.weight_in = weight_in;
  prm.weight = weight;
  prm.weight_width = weight_width;
  prm.keep = (int32_t)keep;
  prm.first = (int32_t)first;
  prm.recent = (int32_t)recent;
  prm.kept = kept;
  prm.new_length = new_length;
  return launched(kv, ra::launch_paged_evict(pb.dtype, prm, kv->sm_count, st), "cache eviction launch", st);
}

ra_status ra_paged_sync_status(ra_paged_t kv, void* stream) {
  if (kv == nullptr) return fail(RA_ERR_INVALID_ARG, "null handle");
  if (kv->device < 0) return fail(RA_ERR_NO_DEVICE, "the handle was created without a CUDA device");
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "stream synchronize: %s", cudaGetErrorString(e));
  uint32_t word = 0;
  e = cudaMemcpy(&word, kv->d_status, sizeof(word), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "status read: %s", cudaGetErrorString(e));
  if (word == 0) return ok();
  // Cleared before the next call can set it (see ra_kv4_sync_status).
  e = cudaMemset(kv->d_status, 0, sizeof(word));
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "status clear: %s", cudaGetErrorString(e));
  if (word & (ra::kStatusBounds | ra::kStatusTimeouts)) {
    char msg[200];
    const ra_status code = ra::status_word_error(word, msg, sizeof(msg));
    return fail(code, "%s", msg);
  }
  return fail(RA_ERR_INVALID_ARG, "a page index, offset, length or slot was out of range");
}

}  // extern "C"
