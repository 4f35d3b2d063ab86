// The 4-bit key/value cache (include/ra.h, ra_kv4_*): format and launchers.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ra_internal.h"

namespace ra {

constexpr int kKvBlockRows = 16;  // tokens of a cache block

// Offsets within a block of 16 tokens (20 * d bytes).
template <int D>
struct Kv4Block {
  static constexpr int kGroups = D / 32;        // groups of 32 channels
  static constexpr int kCodeBytes = D / 2;      // code bytes of a row
  static constexpr int kParBytes = D / 8;       // parameter bytes of a row
  static constexpr int kOffK = 0;
  static constexpr int kOffKPar = 16 * kCodeBytes;
  static constexpr int kOffV = kOffKPar + 16 * kParBytes;
  static constexpr int kOffVPar = kOffV + 16 * kCodeBytes;
  static constexpr int kBytes = kOffVPar + 16 * kParBytes;
};

// What write, read and attend share: the cache and its sequences.
struct Kv4Table {
  uint8_t* cache;
  const int32_t* page_table;  // [batch, width]
  int64_t width;
  int64_t pages;
  int32_t page_rows;
  int32_t blocks_per_page;
  int32_t batch, heads_kv;
  uint32_t* status;
};

// Whether block `at` lies in the pool (debug bounds checks).
template <int D>
__device__ __forceinline__ bool in_pool(const Kv4Table& t, const uint8_t* at) {
  const int64_t off = at - t.cache;
  return off >= 0 && off % Kv4Block<D>::kBytes == 0 &&
         off / Kv4Block<D>::kBytes < t.pages * t.heads_kv * t.blocks_per_page;
}

// Kernel-side status bit: an index of the page table, a length or a count out of range.
constexpr uint32_t kKv4StatusRange = 1u;

struct Kv4RowsParams {  // write, read
  Kv4Table t;
  int32_t rows;
  const int32_t* first;
  const int32_t* count;  // or nullptr: rows
  int32_t zero_rest;     // read: rows that receive nothing become zeros
};

constexpr int kMaxSlots = 1024;  // CTAs among which the sequences of a head and query tile are split

struct Kv4AttendParams {
  Kv4Table t;
  int32_t heads_q, group, rows;  // query rows per sequence
  int32_t tiles;                 // 8-row query tiles per key/value head
  int32_t slots;                 // CTAs of a key/value head and tile
  int32_t in_row;                // they share the sequences' blocks in a row; else one a sequence (or several for one)
  int32_t window, sinks;         // window 0: the whole prefix
  float scale_log2;
  const int32_t* length;
  const void* q;
  void* o;
  float* lse;      // or nullptr
  // in_row, or several slots for one sequence:
  float* part_o;   // [head * tiles + tile, slot, 2, 8, D]
  float2* part_ml; // [head * tiles + tile, slot, 2, 8]: running maximum (log2 units) and sum
  int2* shares;    // [batch]: a sequence's first and last slot (batch > 1)
};

cudaError_t launch_kv4_write(int dtype, int head_dim, const Kv4RowsParams& prm, const void* k, const void* v,
                             cudaStream_t stream);
cudaError_t launch_kv4_read(int dtype, int head_dim, const Kv4RowsParams& prm, void* k, void* v, cudaStream_t stream);
cudaError_t launch_kv4_attend(int dtype, int head_dim, const Kv4AttendParams& prm, cudaStream_t stream);

}  // namespace ra
