// C ABI of the 4-bit key/value cache (include/ra.h, ra_kv4_*): argument checks, handles
// and the split of attention over CTAs.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <new>
#include <vector>

#include "api_internal.h"
#include "kv4_internal.h"

struct ra_kv4_s {
  ra_kv4_problem prob;
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

constexpr int64_t kMaxPositions = int64_t(1) << 30;  // of a sequence: block arithmetic stays in 32 bits

ra_status validate(const ra_kv4_problem* p) {
  if (p->pages < 1 || p->heads_q < 1 || p->heads_kv < 1 || p->head_dim < 1)
    return fail(RA_ERR_INVALID_ARG, "pages, heads and head_dim must be >= 1");
  if (p->page_rows < ra::kKvBlockRows || p->page_rows > 65536 || p->page_rows % ra::kKvBlockRows)
    return fail(RA_ERR_INVALID_ARG, "page_rows must be a multiple of %d in 16..65536 (got %d)", ra::kKvBlockRows,
                p->page_rows);
  if (p->heads_q % p->heads_kv) return fail(RA_ERR_INVALID_ARG, "heads_q %% heads_kv != 0");
  if (p->dtype != RA_DTYPE_F32 && p->dtype != RA_DTYPE_BF16) return fail(RA_ERR_INVALID_ARG, "unknown dtype %d", p->dtype);
  if (p->window < 0 || p->sinks < 0) return fail(RA_ERR_INVALID_ARG, "window and sinks must be >= 0");
  if (!(p->scale >= 0.f) || std::isinf(p->scale)) return fail(RA_ERR_INVALID_ARG, "scale must be finite and >= 0");
  if (p->head_dim != 64 && p->head_dim != 128)
    return fail(RA_ERR_UNSUPPORTED, "the 4-bit cache needs head_dim 64 or 128 (got %d)", p->head_dim);
  if (p->pages > INT32_MAX) return fail(RA_ERR_UNSUPPORTED, "more than 2^31-1 pages");
  const int64_t row = (int64_t)p->head_dim * 5 / 4 * p->page_rows;
  if (p->pages > (int64_t(1) << 62) / row / p->heads_kv) return fail(RA_ERR_UNSUPPORTED, "a cache beyond 2^62 bytes");
  return RA_OK;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// The checks that every launch shares; n16 tensors need 16-byte alignment, n4 tables 4.
ra_status check_call(const ra_kv4_s* kv, int64_t batch, int64_t rows, int64_t table_width, const void* const* t16,
                     int n16, const void* const* t4, int n4, cudaStream_t st) {
  for (int i = 0; i < n16; ++i)
    if (!aligned(t16[i], 16)) return fail(RA_ERR_INVALID_ARG, "pointer %p is not 16-byte aligned", t16[i]);
  for (int i = 0; i < n4; ++i)
    if (!aligned(t4[i], 4)) return fail(RA_ERR_INVALID_ARG, "pointer %p is not 4-byte aligned", t4[i]);
  if (batch < 1 || rows < 1 || table_width < 1)
    return fail(RA_ERR_INVALID_ARG, "batch, rows and table_width must be >= 1");
  const ra_kv4_problem& pb = kv->prob;
  if (table_width > kMaxPositions / pb.page_rows)
    return fail(RA_ERR_UNSUPPORTED, "table_width * page_rows above 2^30");
  if (batch > INT32_MAX || rows > INT32_MAX || batch > INT32_MAX / rows || batch * rows > INT32_MAX / pb.heads_kv)
    return fail(RA_ERR_UNSUPPORTED, "batch * heads_kv * rows above 2^31-1");
  if (kv->device < 0) return fail(RA_ERR_NO_DEVICE, "the handle was created without a CUDA device");
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess || cur != kv->device)
    return fail(RA_ERR_INVALID_ARG, "current device %d differs from the handle's device %d", cur, kv->device);
  ra_status s = ra::check_on_current_device(t16, n16, st);
  return s != RA_OK ? s : ra::check_on_current_device(t4, n4, st);
}

ra::Kv4Table table_of(const ra_kv4_s* kv, const void* cache, int64_t batch, const int32_t* page_table, int64_t width) {
  ra::Kv4Table t{};
  t.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  t.page_table = page_table;
  t.width = width;
  t.pages = kv->prob.pages;
  t.page_rows = kv->prob.page_rows;
  t.blocks_per_page = kv->prob.page_rows / ra::kKvBlockRows;
  t.batch = (int32_t)batch;
  t.heads_kv = kv->prob.heads_kv;
  t.status = kv->d_status;
  return t;
}

ra_status launched(ra_kv4_s* kv, cudaError_t e, const char* what, cudaStream_t st) {
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  const ra_status s = ra::mark_use(&kv->marks, st);
  return s != RA_OK ? s : ok();
}

// Query tiles of a key/value head, and the CTAs among which a tile's keys are split.
struct Split {
  int64_t tiles, slots;
  bool in_row;  // the sequences' blocks are shared in a row
};

// Shares of the keys: as many CTAs as the GPU holds at once -- 3 an SM, fp32 2, few rows of
// d = 64 4 (4 sequences of 64k 36 us, with 3 38) -- each with the same number of blocks: of one
// sequence, or of all sequences laid in a row, where a CTA's share may be the end of one and
// the beginning of the next.  The figures of this rule were taken with 8 query rows a product:
// shares per sequence, of equal number whatever its length, took 86 us for 32 sequences under a
// window of 8192 tokens (in a row 79), 117 for 8 of up to 64k (101) and 41 for 16 of up to 8k
// (37).  Beyond that many sequences each has one CTA and the GPU deals them out, unless they
// are up to twice as many and long: 64 sequences of up to 16k tokens 206 us one a sequence, 163
// in a row, 100 of up to 4k 89 and 87, but 64 of up to 2k 36 and 42; 200 of up to 4k 146 and
// 155 us.
// No CTA gets fewer than 16 blocks of 16 tokens, four a warp: below that the join costs more
// than the share saves (8k tokens, one block a warp at a time: 10.5 us; with 8 blocks 12.1,
// with 32 11.5).  Several sequences are shared out only where one may be of 1536 tokens or
// more: 32 of up to 512 take 11 us with a CTA each, 18 in a row; of up to 1024 15 and 21; 4 of
// up to 1024 12.7 and 15.3, of up to 2048 19.7 and 12.5.
ra_status split_of(const ra_kv4_s* kv, int64_t batch, int64_t rows, int64_t table_width, Split* out) {
  const ra_kv4_problem& pb = kv->prob;
  if (batch < 1 || rows < 1 || table_width < 1)
    return fail(RA_ERR_INVALID_ARG, "batch, rows and table_width must be >= 1");
  if (table_width > kMaxPositions / pb.page_rows)
    return fail(RA_ERR_UNSUPPORTED, "table_width * page_rows above 2^30");
  if (rows > INT32_MAX / pb.heads_q) return fail(RA_ERR_UNSUPPORTED, "heads_q * rows above 2^31-1");
  out->tiles = (rows * (pb.heads_q / pb.heads_kv) + 7) / 8;
  if (batch > 65535 || pb.heads_kv * out->tiles > 65535)
    return fail(RA_ERR_UNSUPPORTED, "batch, or heads_kv times the 8-row query tiles, above 65535");
  int64_t keys = table_width * pb.page_rows;
  if (pb.window > 0 && pb.window < kMaxPositions && pb.sinks < kMaxPositions)
    keys = std::min(keys, pb.window + rows + pb.sinks + 32);
  const int64_t sms = kv->sm_count > 0 ? kv->sm_count : 148;
  const bool half = rows * (pb.heads_q / pb.heads_kv) <= 4;  // the kernel's form for few rows
  const int64_t per_sm = pb.dtype != RA_DTYPE_BF16 ? 2 : half && pb.head_dim == 64 ? 4 : 3;
  const int64_t slots = std::min(per_sm * sms / (pb.heads_kv * out->tiles), int64_t(ra::kMaxSlots));
  if (batch == 1) {
    out->in_row = false;
    out->slots = std::max<int64_t>(1, std::min(slots, keys / (16 * 16)));
  } else {
    const bool countable = batch <= INT32_MAX / (keys / ra::kKvBlockRows + 3);  // blocks in all, in 31 bits
    out->in_row = countable && slots > 1 && keys >= 1536 && (batch <= slots || (batch <= 2 * slots && keys >= 4096));
    out->slots = out->in_row ? slots : batch;
  }
  return RA_OK;
}

// Whether a sequence may be spread over several CTAs, whose parts are then joined.
bool joined(const Split& sp, int64_t batch) { return sp.in_row || sp.slots > batch; }

}  // namespace

extern "C" {

ra_status ra_kv4_plan(const ra_kv4_problem* prob, ra_kv4_t* out) {
  if (prob == nullptr || out == nullptr) return fail(RA_ERR_INVALID_ARG, "null argument");
  *out = nullptr;
  ra_status s = validate(prob);
  if (s != RA_OK) return s;
  ra_kv4_s* kv = new (std::nothrow) ra_kv4_s();
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
      ra_kv4_destroy(kv);
      return f;
    }
  } else {
    cudaGetLastError();  // host-only handle
  }
  *out = kv;
  return ok();
}

ra_status ra_kv4_destroy(ra_kv4_t kv) {
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

ra_status ra_kv4_cache_size(ra_kv4_t kv, int64_t* bytes) {
  if (kv == nullptr || bytes == nullptr) return fail(RA_ERR_INVALID_ARG, "null argument");
  const ra_kv4_problem& pb = kv->prob;
  *bytes = pb.pages * pb.heads_kv * pb.page_rows * (int64_t)(pb.head_dim * 5 / 4);
  return ok();
}

ra_status ra_kv4_write(ra_kv4_t kv, void* cache, int64_t batch, int64_t rows, const void* k, const void* v,
                       const int32_t* page_table, int64_t table_width, const int32_t* first, const int32_t* count,
                       void* stream) {
  if (kv == nullptr) return fail(RA_ERR_INVALID_ARG, "null handle");
  if (cache == nullptr || k == nullptr || v == nullptr || page_table == nullptr || first == nullptr)
    return fail(RA_ERR_INVALID_ARG, "null pointer");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const void* t16[] = {cache, k, v};
  const void* t4[] = {page_table, first, count};
  const ra_status s = check_call(kv, batch, rows, table_width, t16, 3, t4, 3, st);
  if (s != RA_OK) return s;
  const ra::Kv4RowsParams prm{table_of(kv, cache, batch, page_table, table_width), (int32_t)rows, first, count, 0};
  return launched(kv, ra::launch_kv4_write(kv->prob.dtype, kv->prob.head_dim, prm, k, v, st), "cache write launch", st);
}

ra_status ra_kv4_read(ra_kv4_t kv, const void* cache, int64_t batch, int64_t rows, const int32_t* page_table,
                      int64_t table_width, const int32_t* first, const int32_t* count, int32_t zero_rest,
                      void* k, void* v, void* stream) {
  if (kv == nullptr) return fail(RA_ERR_INVALID_ARG, "null handle");
  if (zero_rest != 0 && zero_rest != 1) return fail(RA_ERR_INVALID_ARG, "zero_rest must be 0 or 1");
  if (cache == nullptr || k == nullptr || v == nullptr || page_table == nullptr || first == nullptr)
    return fail(RA_ERR_INVALID_ARG, "null pointer");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const void* t16[] = {cache, k, v};
  const void* t4[] = {page_table, first, count};
  const ra_status s = check_call(kv, batch, rows, table_width, t16, 3, t4, 3, st);
  if (s != RA_OK) return s;
  const ra::Kv4RowsParams prm{table_of(kv, cache, batch, page_table, table_width), (int32_t)rows, first, count, zero_rest};
  return launched(kv, ra::launch_kv4_read(kv->prob.dtype, kv->prob.head_dim, prm, k, v, st), "cache read launch", st);
}

ra_status ra_kv4_attend_scratch_size(ra_kv4_t kv, int64_t batch, int64_t rows, int64_t table_width, int64_t* bytes) {
  if (kv == nullptr || bytes == nullptr) return fail(RA_ERR_INVALID_ARG, "null argument");
  Split sp;
  const ra_status s = split_of(kv, batch, rows, table_width, &sp);
  if (s != RA_OK) return s;
  const int64_t parts = !joined(sp, batch) ? 0 : kv->prob.heads_kv * sp.tiles * sp.slots * 2;
  const int64_t part = 8 * (kv->prob.head_dim + 2) * (int64_t)sizeof(float);
  // (the sequences' first and last slots behind the parts, in as many bytes as whole parts)
  *bytes = parts == 0 ? 0 : (parts + (batch * (int64_t)sizeof(int2) + part - 1) / part) * part;
  return ok();
}

ra_status ra_kv4_attend(ra_kv4_t kv, const void* cache, int64_t batch, int64_t rows, const void* q,
                        const int32_t* page_table, int64_t table_width, const int32_t* length, void* o, float* lse,
                        float* scratch, void* stream) {
  if (kv == nullptr) return fail(RA_ERR_INVALID_ARG, "null handle");
  if (cache == nullptr || q == nullptr || page_table == nullptr || length == nullptr || o == nullptr)
    return fail(RA_ERR_INVALID_ARG, "null pointer");
  const ra_kv4_problem& pb = kv->prob;
  Split sp;
  ra_status s = split_of(kv, batch, rows, table_width, &sp);
  if (s != RA_OK) return s;
  if (joined(sp, batch) && scratch == nullptr)
    return fail(RA_ERR_INVALID_ARG, "null scratch (ra_kv4_attend_scratch_size bytes are needed)");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const void* t16[] = {cache, q, o, lse, joined(sp, batch) ? scratch : nullptr};
  const void* t4[] = {page_table, length};
  s = check_call(kv, batch, rows, table_width, t16, 5, t4, 2, st);
  if (s != RA_OK) return s;
  ra::Kv4AttendParams prm{};
  prm.t = table_of(kv, cache, batch, page_table, table_width);
  prm.heads_q = pb.heads_q;
  prm.group = pb.heads_q / pb.heads_kv;
  prm.rows = (int32_t)rows;
  prm.tiles = (int32_t)sp.tiles;
  prm.slots = (int32_t)sp.slots;
  prm.in_row = sp.in_row;
  prm.window = (int32_t)std::min(pb.window, kMaxPositions);
  prm.sinks = (int32_t)std::min(pb.sinks, kMaxPositions);
  prm.scale_log2 = pb.scale * 1.4426950408889634f;
  prm.length = length;
  prm.q = q;
  prm.o = o;
  prm.lse = lse;
  if (joined(sp, batch)) {
    const int64_t parts = pb.heads_kv * sp.tiles * sp.slots * 2;
    prm.part_o = scratch;
    prm.part_ml = reinterpret_cast<float2*>(scratch + parts * 8 * pb.head_dim);
    prm.shares = reinterpret_cast<int2*>(prm.part_ml + parts * 8);
  }
  return launched(kv, ra::launch_kv4_attend(pb.dtype, pb.head_dim, prm, st), "cache attention launch", st);
}

ra_status ra_kv4_sync_status(ra_kv4_t kv, void* stream) {
  if (kv == nullptr) return fail(RA_ERR_INVALID_ARG, "null handle");
  if (kv->device < 0) return fail(RA_ERR_NO_DEVICE, "the handle was created without a CUDA device");
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "stream synchronize: %s", cudaGetErrorString(e));
  uint32_t word = 0;
  e = cudaMemcpy(&word, kv->d_status, sizeof(word), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "status read: %s", cudaGetErrorString(e));
  if (word == 0) return ok();
  // Cleared before the next call can set it: a stream that does not wait for the default one
  // could otherwise have its report cleared.
  e = cudaMemset(kv->d_status, 0, sizeof(word));
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "status clear: %s", cudaGetErrorString(e));
  if (word & ra::kStatusBounds) {
    char msg[200];
    const ra_status code = ra::status_word_error(word, msg, sizeof(msg));
    return fail(code, "%s", msg);
  }
  return fail(RA_ERR_INVALID_ARG, "a page index, position, length or count was out of range");
}

}  // extern "C"
