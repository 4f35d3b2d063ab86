// What the paged cache's tensor-core kernels share: bounded waits, and loads of packed rows.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged_share.cuh"
#include "sm100_ptx.cuh"

namespace ra {

constexpr uint64_t kWaitBudgetNs = 1000000000ull;
constexpr uint32_t kSuspendHintNs = 2000u;  // a waiting thread sleeps up to this long per try

struct Ctl {
  uint32_t bars;
  volatile uint32_t* abort;
  uint32_t* status;
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * (uint32_t)i; }
};

// Bounded wait for phase `parity` of a barrier; false on abort or expiry.
__device__ __forceinline__ bool wait_bar(const Ctl& c, uint32_t bar, uint32_t parity, uint32_t who) {
  if (ptx::mbar_test(bar, parity)) return true;
  const uint64_t t0 = ptx::global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (ptx::mbar_wait_hint(bar, parity, kSuspendHintNs)) return true;
    if ((it & 15u) == 0) {
      if (*c.abort) return false;
      if (ptx::global_timer_ns() - t0 > kWaitBudgetNs) {
        *c.abort = 1u;
        atomicOr(c.status, who);
        return false;
      }
    }
  }
}
// Teardown wait: ignores the abort flag, still bounded.
__device__ __forceinline__ void drain_bar(const Ctl& c, uint32_t bar, uint32_t parity) {
  const uint64_t t0 = ptx::global_timer_ns();
  while (!ptx::mbar_test(bar, parity)) {
    if (ptx::global_timer_ns() - t0 > kWaitBudgetNs) {
      atomicOr(c.status, kStatusTimeoutTeardown);
      return;
    }
  }
}
#define RA_WAIT(n, phase, who) __all_sync(0xffffffffu, wait_bar(c, c.bar(n), (phase) & 1u, who))

__device__ __forceinline__ void tma_load_3d_warp(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y,
                                                 int32_t z) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// As ptx::tma_load_2d, with an L2 policy.
__device__ __forceinline__ void tma_load_2d_hint(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy)
      : "memory");
}

// Prefix sums over a batch, of what `own(b)` says of a sequence (a whole warp calls it and agrees):
// prefix[b] of the sequences before b.  Every thread of the CTA calls it; it ends with a barrier.
template <int kWarps, typename Own>
__device__ __forceinline__ void paged_sums(int batch, int64_t* prefix, Own own) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int b = warp; b < batch; b += kWarps) {
    const int64_t sum = own(b);
    if (lane == 0) prefix[b + 1] = sum;
  }
  __syncthreads();
  if (warp == 0) paged_scan(batch, prefix);
  __syncthreads();
}
// Sum of units(i) over i < n, the whole warp's.
template <typename Units>
__device__ __forceinline__ int64_t warp_total(int n, Units units) {
  int64_t sum = 0;
  for (int i = threadIdx.x & 31; i < n; i += 32) sum += units(i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}
// The i < n in whose units the y-th of all falls (a whole warp calls it), and the units before it.
template <typename Units>
__device__ __forceinline__ int warp_find(int n, int64_t y, int64_t& first, Units units) {
  const int lane = threadIdx.x & 31;
  first = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int64_t own = i0 + lane < n ? units(i0 + lane) : 0;
    int64_t z = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, z, o);
      if (lane >= o) z += v;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, first + z > y);
    if (past) {
      const int src = __ffs(past) - 1;
      first += __shfl_sync(0xffffffffu, z - own, src);
      return i0 + src;
    }
    first += __shfl_sync(0xffffffffu, z, 31);
  }
  return n;
}

}  // namespace ra
