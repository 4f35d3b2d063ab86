// Rotary positions (include/ra.h, ra_rope_*): what the ring's rotation and the paged cache's
// append share, and the launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <vector>

#include "api_internal.h"
#include "ra_internal.h"

struct ra_rope_s {
  ra_rope_problem prob;
  int device = -1;
  int sm_count = 0;
  uint64_t* d_speed = nullptr;  // [rotary_dim / 2], see RopeTable
  // Stream of the handle's own allocation and free (see ra_plan_s::mem_stream).
  cudaStream_t mem_stream = nullptr;
  std::vector<ra::StreamMark> marks;
};

namespace ra {

// Speeds as fractions of a full turn per position, in units of 2^-64 turns: position * speed,
// wrapped to 64 bits, is that speed's angle within a turn without error for any position.  The
// speeds are computed in float64, a few 2^-53 of themselves off, and so are the angles: 2^-24 of a
// turn for the fastest pair at position 2^31, 2^-33 at 2^22.
struct RopeTable {
  const uint64_t* speed;
  float amplitude;
  int32_t rot;  // rotated channels, the first ones
  int32_t interleaved;
};

struct RopeStrides {  // elements
  int64_t batch, head, row;
};

struct RopeParams {
  RopeTable t;
  int32_t d, heads_q, heads_kv, layout, n_shards;
  int64_t batch, seq;
  float sign;  // -1: the transposed rotation
  const int32_t* position;  // [batch, seq] or nullptr: the layout's
  const void *q, *k;
  void *q_out, *k_out;
  RopeStrides qs, ks, qos, kos;
  bool wide;  // 16-byte accesses
};

cudaError_t launch_rope(int dtype, const RopeParams& prm, int sm_count, cudaStream_t stream);

#ifdef __CUDACC__
// Cosine and sine, times the amplitude, of the angle position * speed.  The wrapped 64-bit
// product is cut to 32 bits (2^-33 of a turn), brought to an eighth of a turn around the next
// quarter, where a float keeps it to 2^-27 of a turn, and turned back by exchanging the two.
__device__ __forceinline__ void rope_angle(uint64_t speed, int64_t pos, float amplitude, float sign, float& c, float& s) {
  const uint32_t turn = (uint32_t)(((uint64_t)pos * speed + (1ull << 31)) >> 32);
  const uint32_t quarter = (turn + (1u << 29)) >> 30;
  const int32_t rest = (int32_t)(turn - (quarter << 30));
  float ss, cc;
  sincospif((float)rest * 0x1p-31f, &ss, &cc);
  const bool swap = quarter & 1u;
  c = swap ? ss : cc;
  s = swap ? cc : ss;
  c = ((quarter + 1u) & 2u) ? -c : c;  // quarters 1, 2
  s = (quarter & 2u) ? -s : s;         // quarters 2, 3
  c *= amplitude;
  s *= amplitude * sign;
}

// A thread's share of a row: two vectors of 16 bytes that hold kPairs pairs of channels (or,
// behind the rotated channels, channels that are copied).
template <typename T>
struct RopeUnit {
  static constexpr int kVec = 16 / sizeof(T);
  static constexpr int kPairs = kVec;
  uint4 a, b;
  __device__ __forceinline__ void load(const T* row, int first, int second) {
    a = *reinterpret_cast<const uint4*>(row + first);
    b = *reinterpret_cast<const uint4*>(row + second);
  }
  __device__ __forceinline__ void store(T* row, int first, int second) const {
    *reinterpret_cast<uint4*>(row + first) = a;
    *reinterpret_cast<uint4*>(row + second) = b;
  }
  __device__ __forceinline__ void turn(const float (&c)[kPairs], const float (&s)[kPairs], bool interleaved) {
    float x[2 * kVec], y[2 * kVec];
    unpack(a, x);
    unpack(b, x + kVec);
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        y[2 * i] = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
        y[2 * i + 1] = x[2 * i] * s[i] + x[2 * i + 1] * c[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        y[i] = x[i] * c[i] - x[kVec + i] * s[i];
        y[kVec + i] = x[i] * s[i] + x[kVec + i] * c[i];
      }
    }
    a = pack(y);
    b = pack(y + kVec);
  }

 private:
  static __device__ __forceinline__ void unpack(const uint4& w, float* x) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (sizeof(T) == 2) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
      } else {
        x[i] = __uint_as_float(v[i]);
      }
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* y) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (sizeof(T) == 2) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        v[i] = *reinterpret_cast<const uint32_t*>(&p);
      } else {
        v[i] = __float_as_uint(y[i]);
      }
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
};

__device__ __forceinline__ float rope_load(const float* p) { return *p; }
__device__ __forceinline__ float rope_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void rope_store(float* p, float x) { *p = x; }
__device__ __forceinline__ void rope_store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Where a thread's unit u of a row lies.  Wide units: rot / (2 kPairs) of pairs, then copies.
// Narrow units: rot / 2 pairs, then single channels that are copied (second < 0).
struct RopePlace {
  int first, second, pair;  // pair < 0: a copy
};
template <typename T>
__device__ __forceinline__ RopePlace rope_place(const RopeTable& t, bool wide, int u) {
  constexpr int kVec = RopeUnit<T>::kVec;
  const int half = t.rot >> 1;
  if (wide) {
    const int turned = half / kVec;
    if (u >= turned) return {2 * kVec * u, 2 * kVec * u + kVec, -1};
    if (t.interleaved) return {2 * kVec * u, 2 * kVec * u + kVec, kVec * u};
    return {kVec * u, half + kVec * u, kVec * u};
  }
  if (u >= half) return {t.rot + (u - half), -1, -1};
  if (t.interleaved) return {2 * u, 2 * u + 1, u};
  return {u, half + u, u};
}
template <typename T>
__device__ __forceinline__ int rope_units(const RopeTable& t, bool wide, int d) {
  return wide ? d / (2 * RopeUnit<T>::kVec) : (t.rot >> 1) + (d - t.rot);
}
#endif

// Whether rows of d channels, rot of them rotated, divide into wide units.
inline bool rope_wide(int dtype, int d, int rot) {
  const int unit = dtype == RA_DTYPE_BF16 ? 16 : 8;
  return d % unit == 0 && rot % unit == 0;
}

}  // namespace ra
