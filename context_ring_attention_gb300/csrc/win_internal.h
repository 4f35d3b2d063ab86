// Windowed attention: a query at position i sees the keys j <= i with j > i - window
// or j < sinks (the first tokens of the sequence, which stay visible).  Declarations
// shared by the planner (ra_api.cu) and the kernels (win_fwd_bf16_sm103.cu,
// win_bwd_bf16_sm103.cu, win_f32.cu).
//
// Positions rise with the local row in every layout, so the keys of shard r that a
// query at position P sees are the rows
//   [0, first)  with first = rows of r at positions < sinks          (the sinks), and
//   [lo, hi)    with lo = rows at positions <= P - window,
//                    hi = rows at positions <= P                      (the window).
#pragma once

#include "bwd_internal.h"

namespace ra {

// Rows of shard r at positions <= P (P may be negative): last_le + 1 in 32 bits.
RA_HD int32_t rows_le(int layout, int n_shards, int32_t s_n, int r, int32_t P) {
  int32_t n;
  if (layout == RA_LAYOUT_STRIPED) {
    n = P < r ? 0 : (int32_t)((uint32_t)(P - r) / (uint32_t)n_shards) + 1;
  } else if (layout == RA_LAYOUT_ZIGZAG) {
    const int32_t c = s_n >> 1;
    const int32_t lo = r * c, hi = (2 * n_shards - 1 - r) * c;
    if (P < hi) {
      n = P < lo ? 0 : P - lo + 1;
      n = n < c ? n : c;
    } else {
      n = c + (P - hi) + 1;
    }
  } else {
    n = P < r * s_n ? 0 : P - r * s_n + 1;
  }
  return n < s_n ? n : s_n;
}

// End of the run of consecutive positions (contiguous, zigzag) or of equal steps
// (striped) that local row `row` lies in.  Query and key tiles of a windowed plan stop
// there: a tile across the two chunks of a zigzag shard would span most of the
// sequence, and meet as many tiles.
RA_HD int32_t run_end(int layout, int32_t s_n, int32_t row) {
  return layout == RA_LAYOUT_ZIGZAG && row < (s_n >> 1) ? (s_n >> 1) : s_n;
}

// Key rows of shard r that some query at positions [minpos, maxpos] sees: [0, first)
// and [lo, hi), merged into [lo, hi) (first == 0) when they touch.
struct WinSpan {
  int32_t first, lo, hi;
};
RA_HD WinSpan win_span(int layout, int n_shards, int32_t s_n, int32_t window, int32_t sinks, int r, int32_t minpos,
                       int32_t maxpos) {
  WinSpan s;
  s.hi = rows_le(layout, n_shards, s_n, r, maxpos);
  s.lo = rows_le(layout, n_shards, s_n, r, minpos - window);
  s.first = rows_le(layout, n_shards, s_n, r, sinks - 1);
  if (s.first > s.hi) s.first = s.hi;
  if (s.first >= s.lo) {
    if (s.first > 0) s.lo = 0;
    s.first = 0;
  }
  return s;
}

// How the rows of a head are walked: as `shards` shards of s_n rows in their layout, or
// (shards == 1) in the order of their positions.  stripe > 1: position x lies at row
// (x mod stripe) * (S / stripe) + x / stripe, a striped layout walked in natural order; its
// tiles begin at multiples of the stripe and hold `tile` rows, the largest multiple of it
// up to 128 (one tensor-map box of stripe x tile/stripe rows).
struct WinView {
  int32_t layout, shards, s_n;
  int32_t stripe, tile;
  int32_t apart;  // positions between neighbouring rows (shards, when striped shard by shard)
};

// Forward work item of a windowed plan: one or two tiles of query rows (one tile for two
// heads, or two consecutive tiles of one head) with the key ranges they meet.
struct alignas(16) WinItem {
  int32_t bh0, bh1;          // b*Hq + h of tile 0 and of tile 1 (-1: one tile)
  int32_t shard, row0;       // tile 0: local rows row0 .. min(row0 + tile, row_end)
  int32_t row1, row_end;     // tile 1's first row
  int32_t range0, n_ranges;  // its key ranges
  int32_t n_tiles;           // key tiles over all of them
  int32_t pos0, pos1;        // positions of the tiles' first rows
  int32_t pad;
};
// Key rows [row0, end) of shard r, met at ring step `step` in tiles from row0 on (the rows
// of the last tile from `end` on belong to another range or to nobody).  Row row0 + x is at
// position pos0 + x * apart.
struct alignas(16) WinRange {
  int16_t step, r;
  int32_t row0, end, pos0;
};
RA_HD int32_t range_tiles(const WinRange& rg, int32_t tile) {
  const int32_t rows = rg.end - rg.row0;
  return tile == kTileRows ? (rows + kTileRows - 1) / kTileRows : (rows + tile - 1) / tile;
}

// The keys of a range that the query at position pos sees, as columns counted from the range's
// first row: those below sk, and [lo, hi) -- rows at positions up to its own, and not up to
// window positions before it unless they are sinks.
struct WinColumns {
  int32_t lo, hi, sk;
};
RA_HD WinColumns range_columns(const WinRange& rg, int32_t apart, int32_t window, int32_t sinks, int32_t pos) {
  const int32_t rows = rg.end - rg.row0;
  const int32_t d_hi = pos - rg.pos0, d_lo = d_hi - window, d_sk = sinks - 1 - rg.pos0;
  WinColumns c{d_lo + 1, d_hi + 1, d_sk + 1};
  if (apart > 1) {
    c.hi = d_hi < 0 ? 0 : d_hi / apart + 1;
    c.lo = d_lo < 0 ? 0 : d_lo / apart + 1;
    c.sk = d_sk < 0 ? 0 : d_sk / apart + 1;
  }
  c.hi = c.hi < rows ? c.hi : rows;
  return c;
}

struct WinParams {
  int32_t batch, heads_q, heads_kv, group, head_dim;
  WinView q, k;
  int32_t window, sinks;
  int32_t seq;
  int32_t n_items;
  float scale, scale_log2;
  int32_t step_lo, step_hi;  // ring steps of this launch
  int32_t kv_rotated;        // as FwdParams::kv_rotated
  const WinItem* items;
  const WinRange* ranges;
  void* o;
  float* lse;
  float* o_parts;
  float* lse_parts;
  uint32_t* status;
};

// Rows of shard r of a view at positions <= P.
RA_HD int32_t view_rows_le(const WinView& v, int r, int32_t P) {
  if (v.shards > 1) return rows_le(v.layout, v.shards, v.s_n, r, P);
  return P < 0 ? 0 : (P < v.s_n ? P + 1 : v.s_n);
}

// Backward.  Rows [first, end) of shard r, streamed in tiles of the view's rows from row0 on,
// the start of the tile that `first` lies in.
struct alignas(16) WinBwdRange {
  int32_t r, row0, end, first;
};
RA_HD int32_t range_tiles64(const WinBwdRange& rg, int32_t tile) {
  const int32_t rows = rg.end - rg.row0;
  return tile == 64 ? (rows + 63) / 64 : (rows + tile - 1) / tile;
}
// One own tile (pass 0: keys, bh = b*Hkv + kv head; pass 1: queries, bh = b*Hq + h) and the
// ranges it meets, for heads g0 .. g1 - 1 of the group (pass 1: one).
struct alignas(16) WinBwdItem {
  int32_t bh, shard, row0, row_end;
  int32_t range0, n_ranges, n_tiles, pos0;
  int32_t g0, g1;
  int32_t part_rows;  // rows of the partial sums
  int32_t pad;
  int64_t part;       // pass 0: where they go (float index in parts), -1: straight to dV, dK
  int64_t pad2;
};
// A key tile that was cut: n_near parts of all its rows (128) from the queries that may see any
// of them, n_far parts of its sinks' rows from the others; each holds dV rows, then dK rows.
struct alignas(16) WinBwdSplit {
  int32_t bh, shard, row0, row_end;
  int64_t near, far;
  int32_t n_far, far_rows, n_near;
  int32_t pad;
};

struct WinBwdParams {
  int32_t batch, heads_q, heads_kv, group;
  WinView own, str;     // the items' tiles (up to 128 rows) and the streamed ones (up to 64)
  int32_t window, sinks;
  int32_t seq;
  int32_t n_items;
  int32_t blocks;       // streamed tiles of a shard
  float scale, scale_log2;
  const float* lse2d;   // per streamed tile of queries 64 lse2 values, then 64 D values
  int64_t n_scalars;
  void* dq;
  void* dk;
  void* dv;
  const void* q;        // pass 1 reads its own query rows of Q and dO directly
  const void* dout;
  float* parts;
  const WinBwdItem* items;
  const WinBwdRange* ranges;
  uint32_t* status;
};
// The rows of a range that are live for the own row at position pos, counted from the range's
// row0: [lo, hi) and [from, sk), of both the range's own.  Pass 0: the queries from the key's
// position on, up to window - 1 later, or all of them when the key is a sink.  Pass 1: the
// window's keys, and the sinks.
struct WinBwdColumns {
  int32_t lo, hi, sk, from;  // (rows before `from` belong to another range)
};
template <int kPass>
RA_HD WinBwdColumns range_columns(const WinBwdParams& P, const WinBwdRange& rg, int32_t pos) {
  WinBwdColumns c{0, 0, 0, 0};
  if (kPass == 0) {
    const int64_t far = (int64_t)pos + P.window - 1;
    const int32_t last = pos < P.sinks || far > P.seq - 1 ? P.seq - 1 : (int32_t)far;
    c.lo = view_rows_le(P.str, rg.r, pos - 1);
    c.hi = view_rows_le(P.str, rg.r, last);
  } else {
    c.lo = view_rows_le(P.str, rg.r, pos - P.window);
    c.hi = view_rows_le(P.str, rg.r, pos);
    c.sk = view_rows_le(P.str, rg.r, P.sinks - 1);
  }
  c.lo = (c.lo > rg.first ? c.lo : rg.first) - rg.row0;
  c.hi = (c.hi < rg.end ? c.hi : rg.end) - rg.row0;
  c.sk = (c.sk < rg.end ? c.sk : rg.end) - rg.row0;
  c.sk = c.sk < c.hi ? c.sk : c.hi;
  c.from = rg.first - rg.row0;
  return c;
}
// Block of scalars of streamed tile `tile` of a shard (bh = b*Hq + h).
RA_HD int64_t win_scalar_block(const WinBwdParams& P, int64_t bh, int shard, int tile) {
  return (bh * P.str.shards + shard) * P.blocks + tile;
}

cudaError_t launch_win_bwd_prep(const WinBwdParams& prm, const void* o, const float* lse, float* out, int sms,
                                cudaStream_t stream);
// pass 0: dK and dV (items are key tiles); pass 1: dQ (items are query tiles); each with grid
// CTAs, one after the other or (both) side by side in one launch.
cudaError_t launch_win_bwd_bf16(const WinBwdParams (&prm)[2], const void* q, const void* k, const void* v,
                                const void* dout, const int (&grid)[2], bool both, cudaStream_t stream, const char** why);
cudaError_t launch_win_bwd_join(const WinBwdParams& prm, const WinBwdSplit* splits, int n, cudaStream_t stream);
cudaError_t launch_win_fwd_bf16(const WinParams& prm, const void* q, const void* k, const void* v, int grid,
                                cudaStream_t stream, const char** why);
cudaError_t launch_win_fwd_f32(const WinParams& prm, const float* q, const float* k, const float* v,
                               cudaStream_t stream);
cudaError_t launch_win_bwd_f32(const BwdParams& prm, int window, int sinks, const float* q, const float* k,
                               const float* v, const float* dout, cudaStream_t stream);

}  // namespace ra
