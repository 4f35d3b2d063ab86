// The attention weight that cached keys receive from a packed batch of new tokens
// (include/ra.h, ra_paged_weigh): for every slot j of a sequence and key/value head,
//   weight_j = (weight_in_j, of slots before the call's tokens) + sum_i e^(scale * q_i.k_j - LSE_i)
// over the query rows i of the head's group that see j.  Given the rows' LSE no softmax is
// left: the sums run down the columns, each column belongs to one warp, and no order varies.
//
// Bound by HBM for few rows: the keys are read once.  bf16: a warp has 32 keys in registers as
// the second operand of m16n8k16 and takes the query rows 16 at a time.  The products run over
// channels in the order in which a 16-byte load of a row brings them, the same for queries and
// keys, so that neither passes through shared memory.  float32: a warp has 32 keys, one a lane.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "paged_share.cuh"
#include "sm100_ptx.cuh"

namespace ra {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kKeys = 32;                  // of a warp
constexpr int kChunk = kWarps * kKeys;     // of a CTA at a time
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Sums of the sequences' chunks of keys (as paged_prefix, of lengths).
__device__ void chunk_prefix(const PagedTable& t, int32_t* prefix) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    int before = 0;
    for (int b0 = 0; b0 < t.batch; b0 += 32) {
      int x = b0 + lane < t.batch ? (paged_seq(t, b0 + lane).length + kChunk - 1) / kChunk : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b0 + lane < t.batch) prefix[b0 + lane + 1] = before + x;
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) prefix[0] = 0;
  }
  __syncthreads();
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) weigh_kernel(const PagedWeighParams P) {
  extern __shared__ int32_t prefix[];
  chunk_prefix(P.t, prefix);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, head = (int)blockIdx.y;
  const int chunks = prefix[P.t.batch];
  const T* cache = static_cast<const T*>(P.t.cache);
  int b = 0;
  for (int c = (int)blockIdx.x; c < chunks; c += (int)gridDim.x) {
    while (prefix[b + 1] <= c) ++b;
    const PagedSeq seq = paged_seq(P.t, b);
    const int j0 = (c - prefix[b]) * kChunk + warp * kKeys;
    if (j0 >= seq.length) continue;
    RA_BOUNDS(P.t.status, b < P.t.batch && seq.token0 + seq.count <= P.t.tokens, 115);
    const int rows = seq.count * P.group, row0 = seq.token0 * P.group;
    // Tiles of 16 rows that see one of this warp's keys: behind a key's own slot all tokens of
    // the call do, up to the window (sinks: to the end).
    const int jl = min(j0 + kKeys, seq.length) - 1;
    const int tok0 = max(0, j0 - seq.slot0());
    const int64_t far = P.window > 0 && j0 >= P.sinks ? (int64_t)jl + P.window - seq.slot0() : seq.count;
    const int tok1 = (int)max((int64_t)0, min((int64_t)seq.count, far));
    const int tile1 = tok1 > tok0 ? (tok1 * P.group + 15) / 16 : 0, tile0 = tok0 * P.group / 16;
    // Slots that no token of the call sees keep what they had; their pages are not looked up.
    auto seen = [&](int j) {
      return seq.count > 0 && (P.window == 0 || j > seq.slot0() - P.window || j < P.sinks);
    };
    auto row_ptr = [&](int r) {
      const int row = row0 + r, token = row / P.group;
      return static_cast<const T*>(P.q) + token * P.qs.token + (int64_t)(head * P.group + row - token * P.group) * P.qs.head;
    };
    auto lse_of = [&](int r) {
      const int row = row0 + r, token = row / P.group;
      return __ldg(P.lse + (int64_t)token * P.heads_q + head * P.group + row - token * P.group);
    };
    auto put = [&](int j, float sum) {
      if (j >= P.weight_width) {
        atomicOr(P.t.status, kPagedStatusRange);
        return;
      }
      const int64_t at = ((int64_t)b * P.t.heads_kv + head) * P.weight_width + j;
      RA_BOUNDS(P.t.status, j >= 0 && j < seq.length && at < (int64_t)P.t.batch * P.t.heads_kv * P.weight_width, 112);
      P.weight[at] = (P.weight_in != nullptr && j < seq.slot0() ? P.weight_in[at] : 0.f) + sum;
    };
    if constexpr (sizeof(T) == 2) {
      const int quad = lane >> 2, two = (lane & 3) * 2, ch = (lane & 3) * 8;
      uint4 k[kKeys / 8][D / 32];
      uint32_t there = 0u;  // keys quad + 8 i, unless their page is none
#pragma unroll
      for (int i = 0; i < kKeys / 8; ++i) {
        const int j = j0 + quad + 8 * i;
        const bool look = j < seq.length && seen(j);
        const int page = look ? paged_page(P.t, b, j / P.t.page_rows) : -1;
        if (page >= 0 || !look) there |= 1u << i;
        const T* src = cache + paged_row(P.t, max(page, 0), 0, head, j % P.t.page_rows) * D + ch;
#pragma unroll
        for (int x = 0; x < D / 32; ++x)
          k[i][x] = page >= 0 ? __ldg(reinterpret_cast<const uint4*>(src + 32 * x)) : make_uint4(0u, 0u, 0u, 0u);
      }
      float sum[kKeys / 8][2];
#pragma unroll
      for (int i = 0; i < kKeys / 8; ++i) sum[i][0] = sum[i][1] = 0.f;
      for (int t = tile0; t < tile1; ++t) {
        const int ra = t * 16 + quad;
        uint4 q[2][D / 32];
        float lse2[2];
        int slot[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool live = ra + 8 * i < rows;
          slot[i] = live ? seq.slot0() + (ra + 8 * i) / P.group : -1;
          const T* src = live ? row_ptr(ra + 8 * i) + ch : nullptr;
          lse2[i] = live ? lse_of(ra + 8 * i) * kLog2e : 0.f;
#pragma unroll
          for (int x = 0; x < D / 32; ++x)
            q[i][x] = live ? __ldg(reinterpret_cast<const uint4*>(src + 32 * x)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < kKeys / 8; ++i) {
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            mma16816(s, q[0][x].x, q[1][x].x, q[0][x].y, q[1][x].y, k[i][x].x, k[i][x].y);
            mma16816(s, q[0][x].z, q[1][x].z, q[0][x].w, q[1][x].w, k[i][x].z, k[i][x].w);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool sees = paged_sees(P.window, P.sinks, slot[e >> 1], j0 + 8 * i + two + (e & 1));
            const float p = ptx::ex2_approx(fmaf(s[e], P.scale_log2, -lse2[e >> 1]));
            sum[i][e & 1] += sees ? p : 0.f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kKeys / 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) sum[i][e] += __shfl_xor_sync(0xffffffffu, sum[i][e], o);
          const int j = j0 + 8 * i + two + e;
          // (the lane with this key's page: quad == two + e)
          const uint32_t ok = __shfl_sync(0xffffffffu, there, (two + e) * 4);
          if (quad == 0 && j < seq.length && ((ok >> i) & 1u)) put(j, sum[i][e]);
        }
    } else {
      const int j = j0 + lane;
      const bool look = j < seq.length && seen(j);
      const int page = look ? paged_page(P.t, b, j / P.t.page_rows) : -1;
      const float4* k = reinterpret_cast<const float4*>(cache + paged_row(P.t, max(page, 0), 0, head, j % P.t.page_rows) * D);
      float sum = 0.f;
      for (int r0 = tile0 * 16; r0 < min(rows, tile1 * 16); r0 += 4) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const float4* q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = reinterpret_cast<const float4*>(row_ptr(min(r0 + i, rows - 1)));
#pragma unroll 4
        for (int c4 = 0; c4 < D / 4; ++c4) {
          const float4 kk = page >= 0 ? __ldg(k + c4) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 qq = __ldg(q[i] + c4);
            s[i] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, s[i]))));
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (r0 + i >= rows) break;
          const bool sees = paged_sees(P.window, P.sinks, seq.slot0() + (r0 + i) / P.group, j);
          const float p = exp2f(fmaf(s[i], P.scale_log2, -lse_of(r0 + i) * kLog2e));
          sum += sees ? p : 0.f;
        }
      }
      if (j < seq.length && (page >= 0 || !look)) put(j, sum);
    }
  }
}

template <typename T, int D>
cudaError_t launch(const PagedWeighParams& prm, int sm_count, cudaStream_t stream) {
  const int64_t most = (int64_t)prm.t.batch * ((prm.t.width * prm.t.page_rows + kChunk - 1) / kChunk);
  const int64_t want = std::max<int64_t>(1, (int64_t)sm_count * 4 / prm.t.heads_kv);
  const dim3 grid((unsigned)std::min(most, want), (unsigned)prm.t.heads_kv);
  weigh_kernel<T, D><<<grid, kThreads, (prm.t.batch + 1) * 4, stream>>>(prm);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_weigh_rows(int dtype, int head_dim, const PagedWeighParams& prm, int sm_count,
                                    cudaStream_t stream) {
  if (dtype == RA_DTYPE_BF16)
    return head_dim == 128 ? launch<__nv_bfloat16, 128>(prm, sm_count, stream)
                           : launch<__nv_bfloat16, 64>(prm, sm_count, stream);
  return head_dim == 128 ? launch<float, 128>(prm, sm_count, stream) : launch<float, 64>(prm, sm_count, stream);
}

}  // namespace ra
