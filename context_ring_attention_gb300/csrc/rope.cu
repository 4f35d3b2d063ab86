// Rotary positions: queries and keys rotated by their positions, and the transposed rotation
// for their gradients (include/ra.h, ra_rope_*).
//
// The pair (x1, x2) of a row at position n, with the pair's speed w, becomes
//   A (x1 cos nw - x2 sin nw),  A (x1 sin nw + x2 cos nw);
// the gradient goes back through the same with -sin.  Bound by HBM: every row is read and
// written once.  A thread has the pairs of two 16-byte vectors of one position, computes their
// angles once and takes the heads in turn, so that the angles cost nothing next to the rows.
// Speeds are 64-bit fractions of a turn, so that position times speed is brought within a turn,
// to 2^-33 of it at any position, without 64-bit floating point; the speed's own error is that of
// float64 (rope_internal.h).  Measured: 32768 positions of 32 and 8 heads, d 128, strided queries
// and keys (671 MB) 106 us, 6.3 TB/s.
//
// Rows whose rotated part, length, address or strides do not divide into 16-byte vectors take
// a thread per pair.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "rope_internal.h"

namespace ra {
namespace {

constexpr int kThreads = 128;
constexpr int kAtOnce = 4;  // heads

template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams P) {
  constexpr int kPairs = kWide ? RopeUnit<T>::kPairs : 1;
  const int units = rope_units<T>(P.t, kWide, P.d);
  const int64_t n = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t row = n / units;
  if (row >= P.batch * P.seq) return;
  const RopePlace at = rope_place<T>(P.t, kWide, (int)(n - row * units));
  const int64_t b = row / P.seq, i = row - b * P.seq;

  float c[kPairs], s[kPairs];
  if (at.pair >= 0) {
    int64_t pos;
    if (P.position != nullptr) {
      pos = P.position[row];
    } else {
      const int64_t s_n = P.seq / P.n_shards;
      pos = pos_of(P.layout, P.n_shards, s_n, (int)(i / s_n), i % s_n);
    }
#pragma unroll
    for (int e = 0; e < kPairs; ++e) rope_angle(P.t.speed[at.pair + e], pos, P.t.amplitude, P.sign, c[e], s[e]);
  }
  const T* q = static_cast<const T*>(P.q) + b * P.qs.batch + i * P.qs.row;
  T* qo = static_cast<T*>(P.q_out) + b * P.qos.batch + i * P.qos.row;
  const T* k = static_cast<const T*>(P.k) + b * P.ks.batch + i * P.ks.row;
  T* ko = static_cast<T*>(P.k_out) + b * P.kos.batch + i * P.kos.row;
  const int heads = P.heads_q + P.heads_kv;
  // kWide: the loads of a few heads before their stores.
  constexpr int kHeads = kWide ? kAtOnce : 1;
  for (int h0 = blockIdx.y * kHeads; h0 < heads; h0 += gridDim.y * kHeads) {
    const T* src[kHeads];
    T* dst[kHeads];
#pragma unroll
    for (int e = 0; e < kHeads; ++e) {
      const int h = min(h0 + e, heads - 1);
      const bool key = h >= P.heads_q;
      src[e] = key ? k + (h - P.heads_q) * P.ks.head : q + h * P.qs.head;
      dst[e] = key ? ko + (h - P.heads_q) * P.kos.head : qo + h * P.qos.head;
    }
    if constexpr (kWide) {
      RopeUnit<T> u[kHeads];
#pragma unroll
      for (int e = 0; e < kHeads; ++e)
        if (h0 + e < heads) u[e].load(src[e], at.first, at.second);
#pragma unroll
      for (int e = 0; e < kHeads; ++e) {
        if (h0 + e >= heads) break;
        if (at.pair >= 0) u[e].turn(c, s, P.t.interleaved);
        u[e].store(dst[e], at.first, at.second);
      }
    } else if (at.pair >= 0) {
      const float x1 = rope_load(src[0] + at.first), x2 = rope_load(src[0] + at.second);
      rope_store(dst[0] + at.first, x1 * c[0] - x2 * s[0]);
      rope_store(dst[0] + at.second, x1 * s[0] + x2 * c[0]);
    } else {
      dst[0][at.first] = src[0][at.first];
    }
  }
}

template <typename T>
cudaError_t launch(const RopeParams& prm, int sm_count, cudaStream_t stream) {
  const int units = prm.wide ? prm.d / (2 * RopeUnit<T>::kVec) : (prm.t.rot >> 1) + (prm.d - prm.t.rot);
  const int64_t blocks = (prm.batch * prm.seq * units + kThreads - 1) / kThreads;
  // Heads are shared out among blocks where the positions alone leave the GPU idle.
  const int heads = prm.heads_q + prm.heads_kv;
  const int64_t want = (int64_t)sm_count * 8;
  const int split = (int)std::min<int64_t>(std::min(heads, 65535), std::max<int64_t>(1, want / blocks));
  const dim3 grid((unsigned)blocks, (unsigned)split);
  if (prm.wide) rope_kernel<T, true><<<grid, kThreads, 0, stream>>>(prm);
  else rope_kernel<T, false><<<grid, kThreads, 0, stream>>>(prm);
  return cudaGetLastError();
}

ra_status fail(ra_status s, const char* fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  set_last_error(msg);
  return s;
}
ra_status ok() {
  set_last_error("");
  return RA_OK;
}

ra_status validate(const ra_rope_problem* p) {
  if (p->dtype != RA_DTYPE_F32 && p->dtype != RA_DTYPE_BF16) return fail(RA_ERR_INVALID_ARG, "unknown dtype %d", p->dtype);
  if (p->head_dim < 2 || p->rotary_dim < 2 || p->rotary_dim % 2 || p->rotary_dim > p->head_dim)
    return fail(RA_ERR_INVALID_ARG, "rotary_dim must be even, in 2..head_dim (got %d of %d)", p->rotary_dim, p->head_dim);
  if (p->interleaved != 0 && p->interleaved != 1) return fail(RA_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (!(p->base > 1.0) || std::isinf(p->base)) return fail(RA_ERR_INVALID_ARG, "base must be finite and > 1");
  // (it multiplies in float32)
  if (p->amplitude != 0.0 && !(p->amplitude >= FLT_MIN && p->amplitude <= FLT_MAX))
    return fail(RA_ERR_INVALID_ARG, "amplitude must be 0 or a normal float32 above 0");
  if (p->scaling < RA_ROPE_NONE || p->scaling > RA_ROPE_RAMP) return fail(RA_ERR_INVALID_ARG, "unknown scaling %d", p->scaling);
  if (p->scaling != RA_ROPE_NONE && (!(p->factor >= 1.0) || std::isinf(p->factor)))
    return fail(RA_ERR_INVALID_ARG, "factor must be finite and >= 1");
  if (p->scaling == RA_ROPE_BANDS || p->scaling == RA_ROPE_RAMP) {
    if (p->original < 1) return fail(RA_ERR_INVALID_ARG, "original must be >= 1");
    if (!(p->low > 0.0) || !(p->high > p->low) || std::isinf(p->high))
      return fail(RA_ERR_INVALID_ARG, "0 < low < high, both finite, is needed");
  }
  if (p->head_dim > 1024) return fail(RA_ERR_UNSUPPORTED, "head_dim above 1024");
  return RA_OK;
}

// The angle that a pair advances by per position, in radians, scaled for long contexts.
double speed_of(const ra_rope_problem& p, int j) {
  const double rot = p.rotary_dim, two_pi = 6.283185307179586476925;
  double base = p.base;
  if (p.scaling == RA_ROPE_BASE && p.rotary_dim > 2) base *= std::pow(p.factor, rot / (rot - 2.0));
  const double w = std::pow(base, -2.0 * j / rot);
  switch (p.scaling) {
    case RA_ROPE_LINEAR:
      return w / p.factor;
    case RA_ROPE_BANDS: {
      const double turns = (double)p.original * w / two_pi;
      const double own = std::min(1.0, std::max(0.0, (turns - p.low) / (p.high - p.low)));
      return own * w + (1.0 - own) * w / p.factor;
    }
    case RA_ROPE_RAMP: {
      auto index = [&](double t) { return rot * std::log((double)p.original / (two_pi * t)) / (2.0 * std::log(p.base)); };
      const double lo = std::max(std::floor(index(p.high)), 0.0), hi = std::min(std::ceil(index(p.low)), rot - 1.0);
      // (lo may lie behind hi: every pair turns more than `high` times, or none turns `low` times)
      const double part = std::min(1.0, std::max(0.0, (j - lo) / std::max(hi - lo, 0.001)));
      return (1.0 - part) * w + part * w / p.factor;
    }
    default:
      return w;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Strides of a [batch, heads, rows] tensor of rows of d elements: not negative, and for a
// tensor that is written no two rows in one place.
ra_status check_strides(const char* what, const RopeStrides& s, int64_t batch, int64_t heads, int64_t rows, int64_t d,
                        bool written) {
  struct Dim {
    int64_t extent, stride;
  } dims[3] = {{batch, s.batch}, {heads, s.head}, {rows, s.row}};
  // (the largest element index, so that no address arithmetic wraps)
  for (const Dim& x : dims)
    if (x.stride < 0 || (x.extent > 1 && x.stride > (int64_t(1) << 58) / x.extent))
      return fail(RA_ERR_INVALID_ARG, "%s: a stride is negative or beyond 2^58 elements", what);
  if (!written) return RA_OK;
  std::sort(dims, dims + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  int64_t span = d;
  for (const Dim& x : dims) {
    if (x.extent <= 1) continue;
    if (x.stride < span) return fail(RA_ERR_INVALID_ARG, "%s: rows overlap in memory", what);
    span = x.stride * (x.extent - 1) + span;
  }
  return RA_OK;
}

ra_status rotate(ra_rope_t rope, int64_t batch, int64_t seq, int32_t heads_q, int32_t heads_kv, int32_t layout,
                 int32_t n_shards, const int32_t* position, const void* q, const int64_t* q_strides, const void* k,
                 const int64_t* k_strides, void* q_out, const int64_t* q_out_strides, void* k_out,
                 const int64_t* k_out_strides, float sign, void* stream) {
  if (rope == nullptr) return fail(RA_ERR_INVALID_ARG, "null handle");
  if (batch < 1 || seq < 1 || heads_q < 1 || heads_kv < 0)
    return fail(RA_ERR_INVALID_ARG, "batch, seq, heads_q >= 1 and heads_kv >= 0 required");
  if (q == nullptr || q_out == nullptr || q_strides == nullptr || q_out_strides == nullptr ||
      (heads_kv > 0 && (k == nullptr || k_out == nullptr || k_strides == nullptr || k_out_strides == nullptr)))
    return fail(RA_ERR_INVALID_ARG, "null pointer");
  if (layout < RA_LAYOUT_CONTIGUOUS || layout > RA_LAYOUT_ZIGZAG) return fail(RA_ERR_INVALID_ARG, "unknown layout %d", layout);
  if (n_shards < 1) return fail(RA_ERR_INVALID_ARG, "n_shards must be >= 1");
  if (position == nullptr && seq % ((int64_t)n_shards * (layout == RA_LAYOUT_ZIGZAG ? 2 : 1)))
    return fail(RA_ERR_INVALID_ARG, "seq does not divide into the layout's shards");
  if (reinterpret_cast<uintptr_t>(position) & 3) return fail(RA_ERR_INVALID_ARG, "position is not 4-byte aligned");
  const ra_rope_problem& pb = rope->prob;
  const int64_t esize = pb.dtype == RA_DTYPE_BF16 ? 2 : 4;
  if (seq > INT32_MAX || batch > INT32_MAX || batch * seq > (int64_t(1) << 38) / pb.head_dim)
    return fail(RA_ERR_UNSUPPORTED, "batch * seq * head_dim above 2^38, or one of them above 2^31-1");
  if (heads_q > (1 << 20) || heads_kv > (1 << 20)) return fail(RA_ERR_UNSUPPORTED, "more than 2^20 heads");
  RopeParams prm{};
  prm.wide = rope_wide(pb.dtype, pb.head_dim, pb.rotary_dim);
  struct Tensor {
    const char* what;
    const void* p;
    const int64_t* s;
    RopeStrides* to;
    int32_t heads;
    bool written;
  } tensors[] = {{"q", q, q_strides, &prm.qs, heads_q, false},
                 {"q_out", q_out, q_out_strides, &prm.qos, heads_q, true},
                 {"k", k, k_strides, &prm.ks, heads_kv, false},
                 {"k_out", k_out, k_out_strides, &prm.kos, heads_kv, true}};
  for (const Tensor& x : tensors) {
    if (x.heads == 0) continue;
    *x.to = {x.s[0], x.s[1], x.s[2]};
    const ra_status s = check_strides(x.what, *x.to, batch, x.heads, seq, pb.head_dim, x.written);
    if (s != RA_OK) return s;
    if (reinterpret_cast<uintptr_t>(x.p) % esize) return fail(RA_ERR_INVALID_ARG, "%s is not aligned to its elements", x.what);
    if (!aligned16(x.p)) prm.wide = false;
    for (int i = 0; i < 3; ++i)
      if (x.s[i] * esize % 16) prm.wide = false;
  }
  if (rope->device < 0) return fail(RA_ERR_NO_DEVICE, "the handle was created without a CUDA device");
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess || cur != rope->device)
    return fail(RA_ERR_INVALID_ARG, "current device %d differs from the handle's device %d", cur, rope->device);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const void* ptrs[] = {q, q_out, heads_kv ? k : nullptr, heads_kv ? k_out : nullptr, position};
  ra_status s = check_on_current_device(ptrs, 5, st);
  if (s != RA_OK) return s;
  prm.t = {rope->d_speed, pb.amplitude == 0.0 ? 1.0f : (float)pb.amplitude, pb.rotary_dim, pb.interleaved};
  prm.d = pb.head_dim;
  prm.heads_q = heads_q;
  prm.heads_kv = heads_kv;
  prm.layout = layout;
  prm.n_shards = n_shards;
  prm.batch = batch;
  prm.seq = seq;
  prm.sign = sign;
  prm.position = position;
  prm.q = q;
  prm.k = k;
  prm.q_out = q_out;
  prm.k_out = k_out;
  const cudaError_t e = launch_rope(pb.dtype, prm, rope->sm_count, st);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "rotation launch: %s", cudaGetErrorString(e));
  s = mark_use(&rope->marks, st);
  return s != RA_OK ? s : ok();
}

}  // namespace

cudaError_t launch_rope(int dtype, const RopeParams& prm, int sm_count, cudaStream_t stream) {
  return dtype == RA_DTYPE_BF16 ? launch<__nv_bfloat16>(prm, sm_count, stream) : launch<float>(prm, sm_count, stream);
}

}  // namespace ra

extern "C" {

ra_status ra_rope_plan(const ra_rope_problem* prob, ra_rope_t* out) {
  using ra::fail;
  if (prob == nullptr || out == nullptr) return fail(RA_ERR_INVALID_ARG, "null argument");
  *out = nullptr;
  const ra_status s = ra::validate(prob);
  if (s != RA_OK) return s;
  ra_rope_s* rope = new (std::nothrow) ra_rope_s();
  if (rope == nullptr) return fail(RA_ERR_UNSUPPORTED, "out of host memory");
  rope->prob = *prob;
  uint64_t speed[512];
  const int half = prob->rotary_dim / 2;
  for (int j = 0; j < half; ++j)  // radians (at most 1) -> 2^-64 turns
    speed[j] = (uint64_t)std::ldexp(ra::speed_of(*prob, j) / 6.283185307179586476925, 64);
  int dev = -1, count = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && cudaGetDeviceCount(&count) == cudaSuccess && count > 0) {
    rope->device = dev;
    cudaDeviceGetAttribute(&rope->sm_count, cudaDevAttrMultiProcessorCount, dev);
    cudaError_t e = cudaStreamCreateWithFlags(&rope->mem_stream, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaMallocAsync(reinterpret_cast<void**>(&rope->d_speed), half * 8, rope->mem_stream);
    if (e == cudaSuccess) e = cudaMemcpyAsync(rope->d_speed, speed, half * 8, cudaMemcpyHostToDevice, rope->mem_stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(rope->mem_stream);
    if (e != cudaSuccess) {
      const ra_status f = fail(RA_ERR_CUDA, "rotation handle: %s", cudaGetErrorString(e));
      ra_rope_destroy(rope);
      return f;
    }
  } else {
    cudaGetLastError();  // host-only handle
  }
  *out = rope;
  return ra::ok();
}

ra_status ra_rope_destroy(ra_rope_t rope) {
  if (rope == nullptr) return RA_OK;
  if (rope->device >= 0) {
    int cur = -1;
    cudaGetDevice(&cur);
    if (cur != rope->device) cudaSetDevice(rope->device);
    if (rope->mem_stream != nullptr) {
      for (const ra::StreamMark& m : rope->marks) cudaStreamWaitEvent(rope->mem_stream, m.done, 0);
      if (rope->d_speed != nullptr) cudaFreeAsync(rope->d_speed, rope->mem_stream);
      cudaStreamDestroy(rope->mem_stream);  // released once its queued free has run
    }
    for (const ra::StreamMark& m : rope->marks) cudaEventDestroy(m.done);
    cudaGetLastError();
    if (cur >= 0 && cur != rope->device) cudaSetDevice(cur);
  }
  delete rope;
  return RA_OK;
}

ra_status ra_rope(ra_rope_t rope, int64_t batch, int64_t seq, int32_t heads_q, int32_t heads_kv, int32_t layout,
                  int32_t n_shards, const int32_t* position, const void* q, const int64_t* q_strides, const void* k,
                  const int64_t* k_strides, void* q_out, const int64_t* q_out_strides, void* k_out,
                  const int64_t* k_out_strides, void* stream) {
  return ra::rotate(rope, batch, seq, heads_q, heads_kv, layout, n_shards, position, q, q_strides, k, k_strides, q_out,
                    q_out_strides, k_out, k_out_strides, 1.0f, stream);
}

ra_status ra_rope_bwd(ra_rope_t rope, int64_t batch, int64_t seq, int32_t heads_q, int32_t heads_kv, int32_t layout,
                      int32_t n_shards, const int32_t* position, const void* dq, const int64_t* dq_strides,
                      const void* dk, const int64_t* dk_strides, void* dq_out, const int64_t* dq_out_strides,
                      void* dk_out, const int64_t* dk_out_strides, void* stream) {
  return ra::rotate(rope, batch, seq, heads_q, heads_kv, layout, n_shards, position, dq, dq_strides, dk, dk_strides,
                    dq_out, dq_out_strides, dk_out, dk_out_strides, -1.0f, stream);
}

}  // extern "C"
