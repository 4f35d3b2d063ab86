// New tokens of a packed batch into the paged cache (include/ra.h, ra_paged_append): their
// queries and keys rotated by their positions, keys and values to the pages of their sequences.
//
// Bound by HBM: every row is read and written once, in one launch.  As in the ring's rotation
// (rope.cu) a thread has two 16-byte vectors of one token, computes their angles once and takes
// the rows of the token in turn, queries, keys, values, four read before the first is written.
// Measured: 8192 tokens of 32 and 8 heads (201 MB) 39 us, 5.2 TB/s (two rows at a time 46); one
// token of 64 sequences 6.8 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "paged_internal.h"

namespace ra {
namespace {

constexpr int kThreads = 128;
constexpr int kAtOnce = 4;  // rows
constexpr int kKnown = 256;  // sequences whose offsets a block keeps in shared memory

template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads) append_kernel(const PagedAppendParams P) {
  constexpr int kPairs = kWide ? RopeUnit<T>::kPairs : 1;
  __shared__ int32_t offsets[kKnown];
  const bool known = P.t.batch <= kKnown;
  bool falls = false;  // the offsets do somewhere: they are no order to search by
  for (int b = threadIdx.x; b < P.t.batch; b += kThreads) {
    const int a = __ldg(P.t.offset + b);
    falls |= __ldg(P.t.offset + b + 1) < a;
    if (known) offsets[b] = a;
  }
  falls = __syncthreads_or(falls);
  if (blockIdx.x == 0 && blockIdx.y == 0)  // the sequences that no token is found in are checked too
    for (int b = threadIdx.x; b < P.t.batch; b += kThreads) paged_seq(P.t, b);
  const int units = rope_units<T>(P.rope, kWide, P.d);
  const int64_t n = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (n / units >= P.t.tokens) return;
  const int token = (int)(n / units), unit = (int)(n - (int64_t)token * units);
  int b = 0;
  if (!falls) {  // the last sequence that begins at the token or before it
    for (int end = P.t.batch; end - b > 1;) {
      const int mid = (b + end) >> 1;
      ((known ? offsets[mid] : __ldg(P.t.offset + mid)) <= token ? b : end) = mid;
    }
  } else {  // the first one that has the token
    auto has = [&](int b) {
      return __ldg(P.t.offset + b) <= token && token < __ldg(P.t.offset + b + 1) && paged_seq(P.t, b).count > 0;
    };
    while (b + 1 < P.t.batch && !has(b)) ++b;
  }
  const PagedSeq seq = paged_seq(P.t, b);
  const int i = token - seq.token0;
  if (i < 0 || i >= seq.count) return;  // a token of no sequence
  const int slot = seq.slot0() + i;
  const RopePlace at = rope_place<T>(P.rope, kWide, unit);

  const bool turned = at.pair >= 0 && P.rope.speed != nullptr;
  float c[kPairs], s[kPairs];
  if (turned) {
    const int64_t pos = P.position != nullptr ? P.position[token] : slot;
#pragma unroll
    for (int e = 0; e < kPairs; ++e) rope_angle(P.rope.speed[at.pair + e], pos, P.rope.amplitude, 1.0f, c[e], s[e]);
  }
  const int page = paged_page(P.t, b, slot / P.t.page_rows);
  T* cache = static_cast<T*>(P.t.cache);
  const int hk = P.t.heads_kv, heads = P.heads_q + 2 * hk;
  // kWide: the loads of a few rows before their stores.
  constexpr int kRows = kWide ? kAtOnce : 1;
  for (int h0 = blockIdx.y * kRows; h0 < heads; h0 += gridDim.y * kRows) {
    const T* src[kRows];
    T* dst[kRows];
    bool live[kRows], turn[kRows];
#pragma unroll
    for (int e = 0; e < kRows; ++e) {
      const int h = min(h0 + e, heads - 1), g = h - P.heads_q;  // g: key (below heads_kv) or value head
      live[e] = h0 + e < heads && (g < 0 || page >= 0);
      turn[e] = turned && g < hk;
      if (g < 0) {
        src[e] = static_cast<const T*>(P.q) + token * P.qs.token + h * P.qs.head;
        dst[e] = static_cast<T*>(P.q_out) + token * P.qos.token + h * P.qos.head;
      } else {
        const int which = g >= hk;
        const int64_t row = paged_row(P.t, max(page, 0), which, which ? g - hk : g, slot % P.t.page_rows);
        src[e] = which ? static_cast<const T*>(P.v) + token * P.vs.token + (g - hk) * P.vs.head
                       : static_cast<const T*>(P.k) + token * P.ks.token + g * P.ks.head;
        dst[e] = cache + row * P.d;
        RA_BOUNDS(P.t.status, row >= 0 && row < (int64_t)P.t.pages * 2 * hk * P.t.page_rows, 110);
      }
    }
    if constexpr (kWide) {
      RopeUnit<T> u[kRows];
#pragma unroll
      for (int e = 0; e < kRows; ++e)
        if (live[e]) u[e].load(src[e], at.first, at.second);
#pragma unroll
      for (int e = 0; e < kRows; ++e) {
        if (!live[e]) continue;
        if (turn[e]) u[e].turn(c, s, P.rope.interleaved);
        u[e].store(dst[e], at.first, at.second);
      }
    } else {
      if (!live[0]) continue;
      const T x1 = src[0][at.first];
      if (at.second < 0) {
        dst[0][at.first] = x1;
        continue;
      }
      const T x2 = src[0][at.second];
      if (turn[0]) {
        const float a = rope_load(&x1), e = rope_load(&x2);
        rope_store(dst[0] + at.first, a * c[0] - e * s[0]);
        rope_store(dst[0] + at.second, a * s[0] + e * c[0]);
      } else {
        dst[0][at.first] = x1;
        dst[0][at.second] = x2;
      }
    }
  }
}

template <typename T>
cudaError_t launch(const PagedAppendParams& prm, int sm_count, cudaStream_t stream) {
  const int units = prm.wide ? prm.d / (2 * RopeUnit<T>::kVec) : (prm.rope.rot >> 1) + (prm.d - prm.rope.rot);
  const int64_t blocks = ((int64_t)prm.t.tokens * units + kThreads - 1) / kThreads;
  // Rows of a token are shared out among blocks where the tokens alone leave the GPU idle.
  const int heads = prm.heads_q + 2 * prm.t.heads_kv;
  const int split = (int)std::min<int64_t>(std::min(heads, 65535), std::max<int64_t>(1, (int64_t)sm_count * 8 / blocks));
  const dim3 grid((unsigned)blocks, (unsigned)split);
  if (prm.wide) append_kernel<T, true><<<grid, kThreads, 0, stream>>>(prm);
  else append_kernel<T, false><<<grid, kThreads, 0, stream>>>(prm);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(int dtype, const PagedAppendParams& prm, int sm_count, cudaStream_t stream) {
  return dtype == RA_DTYPE_BF16 ? launch<__nv_bfloat16>(prm, sm_count, stream) : launch<float>(prm, sm_count, stream);
}

}  // namespace ra
