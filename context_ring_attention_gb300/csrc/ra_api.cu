// C ABI of libra.so: argument checks, the ring planner and kernel dispatch.
//
// The planner turns a problem into the work list of the tensor-core kernel: one
// item per pair of 128-row query tiles that share a key/value head and a tile
// schedule (two query heads of one GQA group at the same rows, or two
// consecutive row tiles of one head), each with the number of key tiles it
// visits over the N ring steps.  Items are ordered longest first so the
// persistent grid ends evenly under a causal mask, whose per-shard work is
// uneven for contiguous shards (Module 23, "The Causal Imbalance -- and the
// Striped Fix").  For per-step launches (ra_fwd_step, ra_ring_fwd) the plan also
// holds one list per ring step, ordered by that step's cost alone.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>
#include <new>
#include <vector>

#include "api_internal.h"
#include "bwd_internal.h"
#include "ra_internal.h"
#include "win_internal.h"

struct ra_plan_s {
  ra_problem prob;
  int64_t s_n;
  int n_qtiles, n_ktiles;
  std::vector<ra::WorkItem> items;       // whole forward: all N steps per item
  std::vector<ra::WorkItem> step_items;  // per-step lists, concatenated
  std::vector<ra::WorkItem> bwd_items;   // backward: key tiles (dK, dV), then query tiles (dQ)
  std::vector<ra::WorkItem> gather_items;  // forward over gathered (natural-order) K/V
  bool gather_round_sync = false;
  int64_t n_bwd_kv = 0;                  // how many of bwd_items are key tiles
  bool bwd_round_sync[2] = {false, false};  // per backward pass (ra::use_round_sync)
  std::vector<int64_t> step_off;         // list of step t is [step_off[t], step_off[t+1])
  std::vector<int64_t> full, partial, skip;
  int device = -1;
  ra::WorkItem* d_items = nullptr;
  ra::WorkItem* d_step_items = nullptr;
  ra::WorkItem* d_bwd_items = nullptr;
  ra::WorkItem* d_gather_items = nullptr;
  uint32_t* d_status = nullptr;
  // Stream of the plan's own allocations: its device tables are allocated and freed
  // in stream order on it (cudaMallocAsync / cudaFreeAsync), so that destroying a plan
  // never waits on the host for the device.
  cudaStream_t mem_stream = nullptr;
  cudaEvent_t ev_entry = nullptr, ev_rot = nullptr, ev_step = nullptr;  // ra_ring_fwd ordering
  bool round_sync = false;  // forward kernel schedule (ra::use_round_sync)
  int sm_count = 0;
  // Windowed plans (ra_plan_window): window 0 is the whole causal prefix.  Three work lists:
  // over the ring's key blocks (partials, steps), for the fused forward, and over gathered
  // (natural-order) keys; those that are alike share their items.
  int32_t window = 0, sinks = 0;
  struct WinList {
    ra::WinView q, k;
    int64_t first, count;
  } win_lists[3] = {};
  std::vector<ra::WinItem> win_items;
  std::vector<ra::WinRange> win_ranges;
  // Backward: pass 0's items (key tiles), then pass 1's (query tiles); the key tiles that were
  // cut, and the floats of scratch for the rows' scalars and for their parts.
  std::vector<ra::WinBwdItem> win_bwd_items;
  std::vector<ra::WinBwdRange> win_bwd_ranges;
  std::vector<ra::WinBwdSplit> win_splits;
  ra::WinView win_own{}, win_str{};
  int64_t n_win_bwd_kv = 0, win_scalars = 0, win_parts = 0;
  int win_bwd_grid[2] = {0, 0};  // CTAs of the two passes,
  bool win_bwd_both = false;     // which run side by side
  ra::WinBwdItem* d_win_bwd_items = nullptr;
  ra::WinBwdRange* d_win_bwd_ranges = nullptr;
  ra::WinBwdSplit* d_win_splits = nullptr;
  ra::WinItem* d_win_items = nullptr;
  ra::WinRange* d_win_ranges = nullptr;
  // ra_plan_destroy queues the frees of the device tables behind exactly this work.
  std::vector<ra::StreamMark> marks;
};

namespace {

thread_local char g_err[512] = "";

ra_status fail(ra_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return s;
}

ra_status ok() {
  g_err[0] = '\0';
  return RA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

ra_status check_layout(int32_t layout, int64_t seq, int32_t n) {
  if (layout < RA_LAYOUT_CONTIGUOUS || layout > RA_LAYOUT_ZIGZAG)
    return fail(RA_ERR_INVALID_ARG, "unknown layout %d", layout);
  if (seq < 1 || n < 1) return fail(RA_ERR_INVALID_ARG, "seq and n_shards must be >= 1");
  if (seq % n) return fail(RA_ERR_INVALID_ARG, "seq %lld is not a multiple of n_shards %d (uneven shards)", (long long)seq, n);
  if (layout == RA_LAYOUT_ZIGZAG && seq % (2 * (int64_t)n))
    return fail(RA_ERR_INVALID_ARG, "zigzag needs seq %lld to be a multiple of 2*n_shards", (long long)seq);
  if (seq > INT32_MAX) return fail(RA_ERR_UNSUPPORTED, "seq above 2^31-1");
  if (n > INT16_MAX) return fail(RA_ERR_UNSUPPORTED, "n_shards above 32767");
  return RA_OK;
}

constexpr int64_t kMaxPlanPairs = int64_t(1) << 30;
constexpr int64_t kMaxListEntries = int64_t(1) << 27;

ra_status validate(const ra_problem* p) {
  if (p->batch < 1 || p->heads_q < 1 || p->heads_kv < 1 || p->head_dim < 1)
    return fail(RA_ERR_INVALID_ARG, "batch, heads and head_dim must be >= 1");
  ra_status s = check_layout(p->layout, p->seq, p->n_shards);
  if (s != RA_OK) return s;
  if (p->heads_q % p->heads_kv) return fail(RA_ERR_INVALID_ARG, "heads_q %% heads_kv != 0");
  if (p->causal != 0 && p->causal != 1) return fail(RA_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (!(p->scale >= 0.f) || std::isinf(p->scale)) return fail(RA_ERR_INVALID_ARG, "scale must be finite and >= 0");
  if (p->dtype == RA_DTYPE_BF16) {
    if (p->head_dim != 128) return fail(RA_ERR_UNSUPPORTED, "bf16 path needs head_dim == 128 (got %d)", p->head_dim);
  } else if (p->dtype == RA_DTYPE_F32) {
    if (p->head_dim > 128) return fail(RA_ERR_UNSUPPORTED, "f32 path needs head_dim <= 128 (got %d)", p->head_dim);
  } else {
    return fail(RA_ERR_INVALID_ARG, "unknown dtype %d", p->dtype);
  }
  if (p->batch > INT32_MAX / p->heads_q || p->batch * (int64_t)p->heads_q * p->seq > INT32_MAX)
    return fail(RA_ERR_UNSUPPORTED, "B*Hq*S above 2^31-1 rows");
  // The planner's own work: the tile classification visits N x n_qtiles x N
  // (query tile, ring step) pairs, and the tensor-core work lists hold about
  // n_items x (N + 2) entries.  Past these limits planning alone would take
  // tens of seconds to hours and gigabytes of host memory.
  const int64_t N = p->n_shards;
  const int64_t n_qt = (p->seq / N + ra::kTileRows - 1) / ra::kTileRows;
  if (N * N * n_qt > kMaxPlanPairs)
    return fail(RA_ERR_UNSUPPORTED, "ring too large to plan: n_shards^2 x query tiles per shard above 2^30");
  if (p->dtype == RA_DTYPE_BF16) {
    const int64_t per_shard = ra::fwd_items_per_shard(*p, p->seq / N);
    if (per_shard * N * (N + 2) > kMaxListEntries)
      return fail(RA_ERR_UNSUPPORTED, "work lists too large to plan: items x (n_shards + 2) above 2^27");
  }
  return RA_OK;
}

int64_t last_row_pos(const ra_problem& pb, int64_t s_n, int p, int64_t row_start) {
  const int64_t last = std::min<int64_t>(row_start + ra::kTileRows, s_n) - 1;
  return ra::pos_of(pb.layout, pb.n_shards, s_n, p, last);
}

struct Keyed {
  ra::WorkItem w;
  int64_t order;  // creation order, the last tie-break
};

// Items in schedule order (ra::schedule_before on their current cost).
std::vector<ra::WorkItem> schedule(const std::vector<Keyed>& list, int heads_q, int group) {
  int64_t max_cost = 1;
  for (const Keyed& k : list) max_cost = std::max<int64_t>(max_cost, k.w.cost);
  const int64_t width = ra::schedule_bucket_width(max_cost);
  std::vector<ra::ScheduleKey> keys(list.size());
  for (size_t n = 0; n < list.size(); ++n) keys[n] = ra::schedule_key(list[n].w, heads_q, group, width, list[n].order);
  std::vector<size_t> idx(list.size());
  for (size_t n = 0; n < idx.size(); ++n) idx[n] = n;
  std::sort(idx.begin(), idx.end(), [&](size_t a, size_t b) { return ra::schedule_before(keys[a], keys[b]); });
  std::vector<ra::WorkItem> out(list.size());
  for (size_t n = 0; n < list.size(); ++n) out[n] = list[idx[n]].w;
  return out;
}

// Backward work lists.  dK/dV: one item per 128-row key tile (bh0 = b*Hkv + kv
// head, shard r, row0, maxq = position of the tile's first key), costed by the
// 64-row query tiles it meets over the ring (every query head of its group).
// dQ: one item per 128-row query tile (bh0 = b*Hq + h, shard p, row0, maxq =
// position of its last query), costed by the 64-row key tiles it meets.  Both in
// the forward's order rule (longest first, key/value heads grouped).
void build_bwd_schedule(ra_plan_s* pl) {
  const ra_problem& pb = pl->prob;
  const int N = pb.n_shards;
  const int64_t s_n = pl->s_n;
  const int G = pb.heads_q / pb.heads_kv;
  const int n128 = (int)((s_n + 127) / 128), n64 = (int)((s_n + 63) / 64);
  std::vector<Keyed> kv, qs;
  int64_t seqno = 0;
  for (int r = 0; r < N; ++r)
    for (int kt = 0; kt < n128; ++kt)
      for (int64_t b = 0; b < pb.batch; ++b)
        for (int hk = 0; hk < pb.heads_kv; ++hk) {
          ra::WorkItem w{};
          w.bh0 = (int32_t)(b * pb.heads_kv + hk);
          w.bh1 = -1;
          w.shard = r;
          w.row0 = kt * 128;
          w.maxq = (int32_t)ra::pos_of(pb.layout, N, s_n, r, w.row0);
          int cost = 0;
          for (int t = 0; t < N; ++t) {
            const int p = (r + t) % N;
            int lo = 0;
            if (pb.causal) {
              const int64_t f = ra::first_ge(pb.layout, N, s_n, p, w.maxq);
              lo = f >= s_n ? n64 : (int)(f / 64);
            }
            cost += (n64 - lo) * G;
          }
          w.cost = cost;
          kv.push_back({w, seqno++});
        }
  for (int p = 0; p < N; ++p)
    for (int qt = 0; qt < n128; ++qt)
      for (int64_t b = 0; b < pb.batch; ++b)
        for (int h = 0; h < pb.heads_q; ++h) {
          ra::WorkItem w{};
          w.bh0 = (int32_t)(b * pb.heads_q + h);
          w.bh1 = -1;
          w.shard = p;
          w.row0 = qt * 128;
          w.maxq = (int32_t)last_row_pos(pb, s_n, p, w.row0);
          int cost = 0;
          for (int t = 0; t < N; ++t) {
            const int r = (p - t + N) % N;
            if (!pb.causal) {
              cost += n64;
            } else {
              const int64_t j = ra::last_le(pb.layout, N, s_n, r, w.maxq);
              cost += j < 0 ? 0 : (int)(j / 64) + 1;
            }
          }
          w.cost = cost;
          qs.push_back({w, seqno++});
        }
  // schedule_key groups by key/value head from bh0 / heads_q: give the key-tile
  // items a query-head index of their group so that they group the same way.
  std::vector<Keyed> kv_keyed = kv;
  for (Keyed& k : kv_keyed) {
    const int64_t b = k.w.bh0 / pb.heads_kv, hk = k.w.bh0 % pb.heads_kv;
    k.w.bh0 = (int32_t)(b * pb.heads_q + hk * G);
  }
  std::vector<ra::WorkItem> kv_sorted = schedule(kv_keyed, pb.heads_q, G);
  for (ra::WorkItem& w : kv_sorted) {
    const int64_t b = w.bh0 / pb.heads_q, hk = (w.bh0 % pb.heads_q) / G;
    w.bh0 = (int32_t)(b * pb.heads_kv + hk);
  }
  const std::vector<ra::WorkItem> q_sorted = schedule(qs, pb.heads_q, G);
  // Round sync when the streamed data of a head exceeds L2's reach and the longest
  // item (in 64-row tiles, counted as half of a 128-row tile) stays short.
  int64_t max_kv = 0, max_q = 0;
  for (const Keyed& k : kv) max_kv = std::max<int64_t>(max_kv, k.w.cost);
  for (const Keyed& k : qs) max_q = std::max<int64_t>(max_q, k.w.cost);
  pl->bwd_round_sync[0] = ra::use_round_sync(pb.seq, pb.head_dim, max_kv / 2);
  pl->bwd_round_sync[1] = ra::use_round_sync(pb.seq, pb.head_dim, max_q / 2);
  pl->bwd_items = kv_sorted;
  pl->bwd_items.insert(pl->bwd_items.end(), q_sorted.begin(), q_sorted.end());
  pl->n_bwd_kv = (int64_t)kv_sorted.size();
}

void build_schedule(ra_plan_s* pl) {
  const ra_problem& pb = pl->prob;
  const int N = pb.n_shards;
  const int64_t s_n = pl->s_n;
  pl->n_qtiles = (int)((s_n + ra::kTileRows - 1) / ra::kTileRows);
  pl->n_ktiles = pl->n_qtiles;

  // Per-shard tile classification of one 128-row query tile against every key
  // tile it meets over the ring (FULL / PARTIAL / SKIP).
  pl->full.assign(N, 0);
  pl->partial.assign(N, 0);
  pl->skip.assign(N, 0);
  for (int p = 0; p < N; ++p) {
    for (int qt = 0; qt < pl->n_qtiles; ++qt) {
      const int64_t i0 = (int64_t)qt * ra::kTileRows;
      const int64_t qmin = ra::pos_of(pb.layout, N, s_n, p, i0);
      const int64_t qmax = last_row_pos(pb, s_n, p, i0);
      for (int t = 0; t < N; ++t) {
        const int r = (p - t + N) % N;
        if (!pb.causal) {
          pl->full[p] += pl->n_ktiles;
          continue;
        }
        const int visit = ra::visit_tiles(pb.layout, N, s_n, 1, r, qmax);
        const int64_t jmin = ra::last_le(pb.layout, N, s_n, r, qmin);
        // a key tile is FULL when its last key is causal for the tile's first query
        int64_t nfull = 0;
        if (jmin >= s_n - 1) nfull = pl->n_ktiles;
        else if (jmin >= 0) nfull = (jmin + 1) / ra::kTileRows;
        pl->full[p] += nfull;
        pl->partial[p] += visit - nfull;
        pl->skip[p] += pl->n_ktiles - visit;
      }
    }
  }

  if (pb.dtype != RA_DTYPE_BF16) return;  // the SIMT kernel walks rows, not items

  const int G = pb.heads_q / pb.heads_kv;
  std::vector<Keyed> list;
  int64_t seqno = 0;
  ra::for_each_fwd_item(pb, s_n, [&](const ra::WorkItem& w) { list.push_back({w, seqno++}); });
  pl->items = schedule(list, pb.heads_q, G);
  int64_t max_cost = 0;
  for (const Keyed& k : list) max_cost = std::max<int64_t>(max_cost, k.w.cost);
  pl->round_sync = ra::use_round_sync(pb.seq, pb.head_dim, max_cost);

  build_bwd_schedule(pl);

  // The all-gather variant: the same items, each meeting one natural-order block of
  // all S keys (the keys at or before its last query, when causal).
  {
    std::vector<Keyed> g = list;
    int64_t gmax = 0;
    for (Keyed& k : g) {
      k.w.cost = ra::visit_tiles(RA_LAYOUT_CONTIGUOUS, 1, pb.seq, pb.causal, 0, k.w.maxq);
      gmax = std::max<int64_t>(gmax, k.w.cost);
    }
    pl->gather_items = schedule(g, pb.heads_q, G);
    pl->gather_round_sync = ra::use_round_sync(pb.seq, pb.head_dim, gmax);
  }

  // One list per ring step: the same items, costed by that step's key tiles alone.
  // Items with no causal key in the step stay in the list (they write the empty
  // partial: O_t = 0, LSE_t = -inf).
  pl->step_items.clear();
  pl->step_off.assign(1, 0);
  for (int t = 0; t < N; ++t) {
    std::vector<Keyed> step = list;
    for (Keyed& k : step)
      k.w.cost = ra::visit_tiles(pb.layout, N, s_n, pb.causal, (k.w.shard - t + N) % N, k.w.maxq);
    const std::vector<ra::WorkItem> ordered = schedule(step, pb.heads_q, G);
    pl->step_items.insert(pl->step_items.end(), ordered.begin(), ordered.end());
    pl->step_off.push_back((int64_t)pl->step_items.size());
  }
}

// The planner of a windowed plan (ra_plan_window).
int32_t win_pos(const ra_problem& pb, int64_t s_n, int p, int64_t row) {
  return (int32_t)ra::pos_of(pb.layout, pb.n_shards, s_n, p, row);
}

// Key ranges of the queries of shard p at positions [minpos, maxpos], appended to the plan's
// list; returns the number of key tiles.
int32_t add_ranges(ra_plan_s* pl, const ra::WinView& k, int p, int32_t minpos, int32_t maxpos) {
  const int N = k.shards;
  int32_t tiles = 0;
  auto add = [&](int step, int r, int32_t from, int32_t to) {
    while (from < to) {  // (a range stays within a run of equally spaced positions)
      const int32_t end = std::min(to, ra::run_end(k.layout, k.s_n, from)), row0 = from / k.stripe * k.stripe;
      pl->win_ranges.push_back({(int16_t)step, (int16_t)r, row0, end, (int32_t)ra::pos_of(k.layout, N, k.s_n, r, row0)});
      tiles += ra::range_tiles(pl->win_ranges.back(), k.tile);
      from = end;
    }
  };
  for (int t = 0; t < N; ++t) {
    const int r = N == 1 ? 0 : (p - t + N) % N;
    ra::WinSpan sp = ra::win_span(k.layout, N, k.s_n, pl->window, pl->sinks, r, minpos, maxpos);
    // A range begins with a whole stripe: where the window's first stripe holds sinks, the two
    // are one range, or these sinks would be in both.
    if (sp.lo / k.stripe * k.stripe < sp.first) sp.first = sp.lo = 0;
    add(t, r, 0, sp.first);
    add(t, r, sp.lo, sp.hi);
  }
  return tiles;
}

// A forward work list over the views q and k.
ra_plan_s::WinList add_win_list(ra_plan_s* pl, const ra::WinView& q, const ra::WinView& k) {
  const ra_problem& pb = pl->prob;
  const int G = pb.heads_q / pb.heads_kv;
  const bool head_pairs = G % 2 == 0;
  // The query rows of an item, each with its key ranges: one tile for two heads of a
  // key/value head's group, or (odd group) two consecutive tiles of one head.
  struct Rows {
    ra::WinItem item;
    int32_t tiles;
  };
  std::vector<Rows> rows;
  auto pos = [&](int p, int32_t row) { return (int32_t)ra::pos_of(q.layout, q.shards, q.s_n, p, row); };
  for (int p = 0; p < q.shards; ++p)
    for (int32_t row = 0; row < q.s_n;) {
      Rows x{};
      x.item.shard = p;
      x.item.row0 = row;
      x.item.row_end = ra::run_end(q.layout, q.s_n, row);
      x.item.row1 = head_pairs ? row : (row + q.tile < x.item.row_end ? row + q.tile : -1);
      const int32_t end = std::min((x.item.row1 < 0 ? row : x.item.row1) + q.tile, x.item.row_end);
      x.item.pos0 = pos(p, row);
      x.item.pos1 = x.item.row1 < 0 ? 0 : pos(p, x.item.row1);
      x.item.range0 = (int32_t)pl->win_ranges.size();
      x.tiles = x.item.n_tiles = add_ranges(pl, k, p, pos(p, row), pos(p, end - 1));
      x.item.n_ranges = (int32_t)pl->win_ranges.size() - x.item.range0;
      rows.push_back(x);
      row = end;
    }
  // Longest first with key/value heads grouped (the order of ra::schedule_before).
  std::vector<Keyed> list;
  for (size_t g = 0; g < rows.size(); ++g)
    for (int64_t b = 0; b < pb.batch; ++b)
      for (int h = 0; h < pb.heads_q; h += head_pairs ? 2 : 1) {
        ra::WorkItem w{};
        w.bh0 = (int32_t)(b * pb.heads_q + h);
        w.bh1 = head_pairs ? w.bh0 + 1 : (rows[g].item.row1 >= 0 ? w.bh0 : -1);
        w.shard = (int32_t)g;
        w.cost = rows[g].tiles;
        list.push_back({w, (int64_t)list.size()});
      }
  const ra_plan_s::WinList out{q, k, (int64_t)pl->win_items.size(), (int64_t)list.size()};
  for (const ra::WorkItem& w : schedule(list, pb.heads_q, G)) {
    pl->win_items.push_back(rows[w.shard].item);
    pl->win_items.back().bh0 = w.bh0;
    pl->win_items.back().bh1 = w.bh1;
  }
  return out;
}

// FULL / PARTIAL / SKIP counts of a windowed plan: a 128-row key tile is visited when
// it holds a row of the span of the query tile, and FULL when every query of the tile
// sees every key of it.
void win_tile_counts(ra_plan_s* pl) {
  const ra_problem& pb = pl->prob;
  const int N = pb.n_shards;
  const int32_t s_n = (int32_t)pl->s_n, T = ra::kTileRows;
  pl->full.assign(N, 0);
  pl->partial.assign(N, 0);
  pl->skip.assign(N, 0);
  for (int p = 0; p < N; ++p)
    for (int qt = 0; qt < pl->n_qtiles; ++qt) {
      const int32_t qmin = win_pos(pb, s_n, p, (int64_t)qt * T);
      const int32_t qmax = (int32_t)last_row_pos(pb, s_n, p, (int64_t)qt * T);
      for (int t = 0; t < N; ++t) {
        const int r = (p - t + N) % N;
        const ra::WinSpan sp = ra::win_span(pb.layout, N, s_n, pl->window, pl->sinks, r, qmin, qmax);
        const int32_t a = (sp.first + T - 1) / T, b = sp.hi > sp.lo ? (sp.hi + T - 1) / T : 0;
        const int32_t from = sp.hi > sp.lo ? std::max(a, sp.lo / T) : 0;
        const int32_t visited = a + std::max(0, b - from);
        // rows every query of the tile sees: below `all` and from `win` on or below `sink`
        const int32_t all = ra::rows_le(pb.layout, N, s_n, r, qmin);
        const int32_t win = ra::rows_le(pb.layout, N, s_n, r, qmax - pl->window);
        const int32_t sink = std::min(all, ra::rows_le(pb.layout, N, s_n, r, pl->sinks - 1));
        // tiles [0, x) end at or below row x*T (the last tile at s_n)
        auto ended = [&](int32_t row) { return row >= s_n ? pl->n_ktiles : row / T; };
        int32_t full;
        if (sink >= win) {
          full = ended(all);
        } else {
          const int32_t lo = (win + T - 1) / T;
          full = ended(sink) + std::max(0, ended(all) - std::max(lo, ended(sink)));
        }
        pl->full[p] += full;
        pl->partial[p] += visited - full;
        pl->skip[p] += pl->n_ktiles - visited;
      }
    }
}

constexpr int32_t kMostTiles = 1 << 19;  // streamed tiles of a backward item: about half a second

// Backward work lists of a windowed plan (win_internal.h), walked by position or shard by
// shard as the forward's.
void build_win_bwd(ra_plan_s* pl, const ra::WinView& own, const ra::WinView& str) {
  const ra_problem& pb = pl->prob;
  const int N = own.shards;
  const int G = pb.heads_q / pb.heads_kv;
  const int32_t last_pos = (int32_t)pb.seq - 1;
  pl->win_own = own;
  pl->win_str = str;
  pl->win_scalars = pb.batch * (int64_t)pb.heads_q * N * ((str.s_n + str.tile - 1) / str.tile) * 128;

  // Ranges are gathered in `now`, then appended to the plan's list with an item.
  std::vector<ra::WinBwdRange> now;
  auto tiles_now = [&] {
    int32_t n = 0;
    for (const ra::WinBwdRange& x : now) n += ra::range_tiles64(x, str.tile);
    return n;
  };
  auto add = [&](int r, int32_t from, int32_t to) {
    if (to > from) now.push_back({r, from / str.tile * str.tile, to, from});
  };
  // Queries at positions [from, to], shard by shard from the one the key block sits on.
  auto queries = [&](int shard, int32_t from, int32_t to) {
    now.clear();
    for (int t = 0; t < N; ++t) {
      const int p = (shard + t) % N;
      add(p, ra::view_rows_le(str, p, from - 1), ra::view_rows_le(str, p, to));
    }
  };
  auto put_ranges = [&](ra::WinBwdItem* it, const std::vector<ra::WinBwdRange>& list) {
    it->range0 = (int32_t)pl->win_bwd_ranges.size();
    it->n_ranges = (int32_t)list.size();
    pl->win_bwd_ranges.insert(pl->win_bwd_ranges.end(), list.begin(), list.end());
  };
  auto tile_at = [&](int p, int32_t row) {
    ra::WinBwdItem it{};
    it.shard = p;
    it.row0 = row;
    it.row_end = std::min(row + own.tile, ra::run_end(own.layout, own.s_n, row));
    it.pos0 = (int32_t)ra::pos_of(own.layout, N, own.s_n, p, row);
    it.g1 = 1;
    it.part = -1;
    return it;
  };
  auto last_of = [&](const ra::WinBwdItem& it) {
    return (int32_t)ra::pos_of(own.layout, N, own.s_n, it.shard, it.row_end - 1);
  };
  // Items of one tile for every (batch, head), in the order of ra::schedule_before.
  auto emit = [&](std::vector<ra::WinBwdItem>& tiles, bool kv) {
    std::vector<Keyed> list;
    for (size_t x = 0; x < tiles.size(); ++x)
      for (int64_t b = 0; b < pb.batch; ++b)
        for (int h = 0; h < pb.heads_q; h += kv ? G : 1) {
          ra::WorkItem w{};
          w.bh0 = (int32_t)(b * pb.heads_q + h);
          w.shard = (int32_t)x;
          w.cost = tiles[x].n_tiles;
          list.push_back({w, (int64_t)list.size()});
        }
    for (const ra::WorkItem& w : schedule(list, pb.heads_q, G)) {
      ra::WinBwdItem it = tiles[w.shard];
      it.bh = kv ? w.bh0 / pb.heads_q * pb.heads_kv + w.bh0 % pb.heads_q / G : w.bh0;
      if (it.part >= 0) it.part += (int64_t)it.bh * it.pad2;  // the parts of a head
      pl->win_bwd_items.push_back(it);
    }
  };

  // Pass 0: first the tiles without a sink (their size bounds the pieces), then the others.
  std::vector<ra::WinBwdItem> tiles, sink_tiles;
  int32_t normal = 8;
  for (int p = 0; p < N; ++p)
    for (int32_t row = 0; row < own.s_n;) {
      ra::WinBwdItem it = tile_at(p, row);
      row = it.row_end;
      it.g1 = G;
      if (it.pos0 < pl->sinks) {
        sink_tiles.push_back(it);
        continue;
      }
      queries(p, it.pos0, (int32_t)std::min<int64_t>((int64_t)last_of(it) + pl->window - 1, last_pos));
      it.n_tiles = tiles_now() * G;
      normal = std::max(normal, it.n_tiles);
      put_ranges(&it, now);
      tiles.push_back(it);
    }
  // Pieces no smaller than a ten-thousandth of the whole pass: with many tiles of sinks they
  // balance without being cut finely, and their sums would take more memory than the tensors.
  // And none beyond a quarter second, the longest that a record is waited for being one.
  int64_t total = 0;
  for (const ra::WinBwdItem& it : tiles) total += it.n_tiles;
  for (ra::WinBwdItem& it : sink_tiles) {
    queries(it.shard, it.pos0, last_pos);
    it.n_tiles = tiles_now() * G;
    total += it.n_tiles;
  }
  total *= pb.batch * pb.heads_kv;
  normal = std::max(normal, (int32_t)std::min<int64_t>(total / 10000, kMostTiles / 2));
  const int32_t whole = std::max(normal, std::min(2 * normal, kMostTiles));  // tiles of a sink tile left as it is
  // Where the tiles are too few for the SMs (37, a quarter of 148, or less: the lists are built
  // before a device is known) the chain of streamed tiles of one is the pass: those of more than one and a half times an SM's share (8
  // tiles at least) are cut too.  Whole and cut: 1024 tokens of 8 query heads for 2, window 512,
  // 65 and 23 us; 810 of 4 for 1, 36 and 25; 4096 of 4 for 1 under a window of as many 225 and
  // 105.  With 64 tiles and more there is nothing to gain, and the parts have to be written and
  // added: 4096 tokens of 8 for 2 in zigzag shards 54 and 72.
  const int32_t share = (int32_t)std::clamp<int64_t>(total / 148, 8, kMostTiles / 2);
  const bool small = share < normal &&
                     (int64_t)(tiles.size() + sink_tiles.size()) * pb.batch * pb.heads_kv <= 37;
  int64_t parts = 0;  // floats per key/value head
  std::vector<ra::WinBwdSplit> splits;
  // The heads' queries `now` of a tile in pieces of up to `limit` streamed tiles, each with a
  // part of `rows` rows: of several heads while these have few.  Returns the number of pieces.
  std::vector<ra::WinBwdItem> pieces;
  auto cut = [&](const ra::WinBwdItem& it, int32_t limit, int32_t rows) {
    const int32_t per_head = tiles_now();
    const int heads = std::max(1, std::min(G, limit / std::max(per_head, 1)));
    std::vector<ra::WinBwdRange> piece;
    int32_t count = 0;
    auto flush = [&](int g0, int g1) {
      ra::WinBwdItem x = it;
      x.g0 = g0;
      x.g1 = g1;
      x.part = parts;
      x.part_rows = rows;
      x.n_tiles = 0;
      for (const ra::WinBwdRange& y : piece) x.n_tiles += ra::range_tiles64(y, str.tile) * (g1 - g0);
      put_ranges(&x, piece);
      pieces.push_back(x);
      parts += 2 * (int64_t)rows * 128;
      ++count;
      piece.clear();
    };
    for (int g0 = 0; g0 < G; g0 += heads) {
      const int g1 = std::min(G, g0 + heads);
      const int32_t most = std::max(1, limit / (g1 - g0));  // tiles of a piece, per head
      int32_t have = 0;
      for (ra::WinBwdRange x : now)
        while (x.first < x.end) {
          ra::WinBwdRange part = x;
          part.end = std::min<int64_t>(x.end, (int64_t)x.row0 + (int64_t)(most - have) * str.tile);
          piece.push_back(part);
          have += ra::range_tiles64(part, str.tile);
          x.first = x.row0 = part.end;
          if (have == most) {
            flush(g0, g1);
            have = 0;
          }
        }
      if (!piece.empty()) flush(g0, g1);
    }
    return count;
  };
  std::vector<ra::WinBwdItem> all;
  all.swap(tiles);
  for (ra::WinBwdItem it : all) {
    if (!small || it.n_tiles <= share + share / 2) {
      tiles.push_back(it);
      continue;
    }
    queries(it.shard, it.pos0, (int32_t)std::min<int64_t>((int64_t)last_of(it) + pl->window - 1, last_pos));
    ra::WinBwdSplit sp{0, it.shard, it.row0, it.row_end, parts, 0, 0, 0, 0, 0};
    sp.n_near = cut(it, share, 128);
    sp.far = parts;
    splits.push_back(sp);
  }
  for (ra::WinBwdItem it : sink_tiles) {
    const int32_t reach = (int32_t)std::min<int64_t>((int64_t)last_of(it) + pl->window - 1, last_pos);
    queries(it.shard, it.pos0, last_pos);
    it.n_tiles = tiles_now() * G;
    const bool far = it.n_tiles > whole && reach < last_pos;
    if (!far && (!small || it.n_tiles <= share + share / 2)) {
      put_ranges(&it, now);
      tiles.push_back(it);
      continue;
    }
    // The near queries in parts of all rows (one, unless the problem is small), the far ones,
    // which see the sinks alone, in pieces of up to `normal` tiles.
    const int32_t first_not = (pl->sinks - it.pos0 + own.apart - 1) / own.apart;  // rows that are sinks
    ra::WinBwdSplit sp{0, it.shard, it.row0, it.row_end, parts, 0, 0, std::min(first_not, it.row_end - it.row0), 0, 0};
    if (far) queries(it.shard, it.pos0, reach);
    sp.n_near = cut(it, small ? share : INT32_MAX, 128);
    sp.far = parts;
    if (far) {
      queries(it.shard, reach + 1, last_pos);
      sp.n_far = cut(it, small ? share : normal, sp.far_rows);
    }
    splits.push_back(sp);
  }
  tiles.insert(tiles.end(), pieces.begin(), pieces.end());
  for (ra::WinBwdItem& it : tiles) it.pad2 = parts;
  emit(tiles, true);
  pl->n_win_bwd_kv = (int64_t)pl->win_bwd_items.size();
  pl->win_parts = parts * pb.batch * pb.heads_kv;
  for (int64_t bh = 0; bh < pb.batch * pb.heads_kv; ++bh)
    for (ra::WinBwdSplit sp : splits) {
      sp.bh = (int32_t)bh;
      sp.near += bh * parts;
      sp.far += bh * parts;
      pl->win_splits.push_back(sp);
    }

  // Pass 1
  tiles.clear();
  for (int p = 0; p < N; ++p)
    for (int32_t row = 0; row < own.s_n;) {
      ra::WinBwdItem it = tile_at(p, row);
      row = it.row_end;
      now.clear();
      for (int t = 0; t < N; ++t) {
        const int r = (p - t + N) % N;
        const ra::WinSpan sp = ra::win_span(str.layout, N, str.s_n, pl->window, pl->sinks, r, it.pos0, last_of(it));
        add(r, 0, sp.first);
        add(r, sp.lo, sp.hi);
      }
      it.n_tiles = tiles_now();
      put_ranges(&it, now);
      tiles.push_back(it);
    }
  emit(tiles, false);
}

// CTAs of the backward's passes.  They do not depend on each other: where one alone leaves SMs
// idle, or ends in a wave that does, they run side by side in one launch.  Times are estimated
// in streamed tiles (a pass 0 tile takes 1.4 of pass 1's, an item 4 more for its beginning and
// end, a launch 6); side by side has to promise 5%.  Measured, one after the other and side by
// side, under a window of 512: 900 tokens of 4 heads 31 and 21 us, 1024 of 32 heads 91 and 68,
// 4096 of 8 heads 78 and 55, of 32 heads 196 and 178; no difference from 8192 of 32 heads on.
void choose_win_bwd_grids(ra_plan_s* pl, int sms) {
  struct Pass {
    int64_t n, sum, longest;
    double time(int g) const {
      return std::max<double>(longest, (double)((n + g - 1) / g) * ((double)sum / (double)n));
    }
  } pass[2] = {};
  for (size_t x = 0; x < pl->win_bwd_items.size(); ++x) {
    Pass& p = pass[(int64_t)x < pl->n_win_bwd_kv ? 0 : 1];
    const int64_t cost = pl->win_bwd_items[x].n_tiles + 4;
    ++p.n;
    p.sum += cost;
    p.longest = std::max(p.longest, cost);
  }
  constexpr double kTile0 = 1.4, kLaunch = 6;
  double best = 0.95 * (kTile0 * pass[0].time(sms) + pass[1].time(sms) + kLaunch);
  for (int x = 0; x < 2; ++x) pl->win_bwd_grid[x] = (int)std::min<int64_t>(pass[x].n, sms);
  pl->win_bwd_both = false;
  for (int g = 1; g < sms; ++g) {
    const double t = std::max(kTile0 * pass[0].time(g), pass[1].time(sms - g));
    if (t < best) {
      best = t;
      pl->win_bwd_both = true;
      pl->win_bwd_grid[0] = (int)std::min<int64_t>(pass[0].n, g);
      pl->win_bwd_grid[1] = (int)std::min<int64_t>(pass[1].n, sms - g);
    }
  }
}

void build_win_schedule(ra_plan_s* pl) {
  const ra_problem& pb = pl->prob;
  const int N = pb.n_shards;
  const int32_t s_n = (int32_t)pl->s_n;
  pl->n_qtiles = (int)((s_n + ra::kTileRows - 1) / ra::kTileRows);
  pl->n_ktiles = pl->n_qtiles;
  win_tile_counts(pl);
  if (pb.dtype != RA_DTYPE_BF16) return;  // the SIMT kernels walk rows, not items
  // Walked shard by shard, as the ring steps and the partials need it, and in the order of
  // positions, where a key tile then holds consecutive positions and the window's edges fall
  // into as few tiles as they can: the fused forward of contiguous shards (which are one
  // run of rows) and of striped ones.  A stripe of more than 128 shards exceeds a tile, and
  // zigzag chunks are runs of consecutive positions as they are.
  const ra::WinView ring{pb.layout, N, s_n, 1, ra::kTileRows, pb.layout == RA_LAYOUT_STRIPED ? N : 1};
  const ra::WinView natural{RA_LAYOUT_CONTIGUOUS, 1, (int32_t)pb.seq, 1, ra::kTileRows, 1};
  ra::WinView rows = natural;
  if (pb.layout == RA_LAYOUT_STRIPED && N > 1 && N <= ra::kTileRows) {
    rows.stripe = N;
    rows.tile = ra::kTileRows / N * N;
  }
  const bool by_position = pb.layout == RA_LAYOUT_CONTIGUOUS || (pb.layout == RA_LAYOUT_STRIPED && N <= ra::kTileRows);
  pl->win_lists[0] = add_win_list(pl, ring, ring);
  pl->win_lists[1] = N == 1 || !by_position ? pl->win_lists[0] : add_win_list(pl, rows, rows);
  pl->win_lists[2] = N == 1 ? pl->win_lists[0]
                     : pb.layout == RA_LAYOUT_CONTIGUOUS && by_position
                         ? pl->win_lists[1]
                         : add_win_list(pl, by_position ? rows : ring, natural);
  // (a streamed tile of the backward holds 64 rows)
  ra::WinView own = ring, str = ring;
  if (pb.layout != RA_LAYOUT_ZIGZAG && (N <= 64 || pb.layout == RA_LAYOUT_CONTIGUOUS)) own = str = rows;
  str.tile = 64 / str.stripe * str.stripe;
  build_win_bwd(pl, own, str);
}

ra_status upload(ra_plan_s* pl) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    pl->device = -1;
    return RA_OK;  // host-only plan
  }
  int count = 0;
  if (cudaGetDeviceCount(&count) != cudaSuccess || count == 0) {
    cudaGetLastError();
    pl->device = -1;
    return RA_OK;
  }
  pl->device = dev;
  cudaDeviceGetAttribute(&pl->sm_count, cudaDevAttrMultiProcessorCount, dev);
  cudaError_t e = cudaStreamCreateWithFlags(&pl->mem_stream, cudaStreamNonBlocking);
  if (e != cudaSuccess) {
    pl->mem_stream = nullptr;
    return fail(RA_ERR_CUDA, "plan stream: %s", cudaGetErrorString(e));
  }
  cudaStream_t ms = pl->mem_stream;
  e = cudaMallocAsync(reinterpret_cast<void**>(&pl->d_status), 256, ms);
  if (e == cudaSuccess) e = cudaMemsetAsync(pl->d_status, 0, 256, ms);
  auto put = [&](const auto& host, auto** dev) {
    if (e != cudaSuccess || host.empty()) return;
    const size_t bytes = host.size() * sizeof(host[0]);
    e = cudaMallocAsync(reinterpret_cast<void**>(dev), bytes, ms);
    if (e == cudaSuccess) e = cudaMemcpyAsync(*dev, host.data(), bytes, cudaMemcpyHostToDevice, ms);
  };
  put(pl->items, &pl->d_items);
  put(pl->step_items, &pl->d_step_items);
  put(pl->bwd_items, &pl->d_bwd_items);
  put(pl->gather_items, &pl->d_gather_items);
  put(pl->win_items, &pl->d_win_items);
  put(pl->win_ranges, &pl->d_win_ranges);
  put(pl->win_bwd_items, &pl->d_win_bwd_items);
  put(pl->win_bwd_ranges, &pl->d_win_bwd_ranges);
  put(pl->win_splits, &pl->d_win_splits);
  // the tables are in place before any launch on another stream reads them
  if (e == cudaSuccess) e = cudaStreamSynchronize(ms);
  if (e == cudaSuccess) e = cudaEventCreateWithFlags(&pl->ev_entry, cudaEventDisableTiming);
  if (e == cudaSuccess) e = cudaEventCreateWithFlags(&pl->ev_rot, cudaEventDisableTiming);
  if (e == cudaSuccess) e = cudaEventCreateWithFlags(&pl->ev_step, cudaEventDisableTiming);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "plan upload failed: %s", cudaGetErrorString(e));
  return RA_OK;
}


// Kernel parameters common to every forward launch of a plan: the whole ring, K/V
// read in place; callers set items, outputs and, for per-step launches, the range.
ra::FwdParams fwd_params(const ra_plan_s* plan) {
  const ra_problem& pb = plan->prob;
  ra::FwdParams prm{};
  prm.batch = (int32_t)pb.batch;
  prm.heads_q = pb.heads_q;
  prm.heads_kv = pb.heads_kv;
  prm.group = pb.heads_q / pb.heads_kv;
  prm.head_dim = pb.head_dim;
  prm.n_shards = pb.n_shards;
  prm.layout = (int16_t)pb.layout;
  prm.causal = (int16_t)pb.causal;
  prm.seq = pb.seq;
  prm.s_n = plan->s_n;
  prm.scale = pb.scale;
  prm.scale_log2 = pb.scale * 1.4426950408889634f;
  prm.status = plan->d_status;
  prm.item_counter = plan->d_status + 1;
  prm.step_lo = 0;
  prm.step_hi = (int16_t)pb.n_shards;
  prm.kv_rotated = 0;
  prm.round_sync = plan->round_sync ? 1 : 0;
  prm.gathered = 0;
  return prm;
}

ra_status mark_use(ra_plan_s* plan, cudaStream_t st);

// Launch a windowed plan's forward kernel: the steps and outputs of prm, on the items of
// the plan (those of the gathered forward when prm.gathered).
ra_status launch_win(ra_plan_s* plan, const ra::FwdParams& prm, const void* q, const void* k, const void* v,
                     cudaStream_t st) {
  const ra_problem& pb = plan->prob;
  ra::WinParams w{};
  w.batch = prm.batch;
  w.heads_q = prm.heads_q;
  w.heads_kv = prm.heads_kv;
  w.group = prm.group;
  w.head_dim = prm.head_dim;
  const int which = prm.gathered ? 2 : (prm.o_parts != nullptr ? 0 : 1);
  const ra_plan_s::WinList& list = plan->win_lists[which];
  w.q = list.q;
  w.k = list.k;
  if (pb.dtype != RA_DTYPE_BF16) {  // rows, not items
    w.q = {pb.layout, pb.n_shards, (int32_t)plan->s_n, 1, 0, 0};
    w.k = prm.gathered ? ra::WinView{RA_LAYOUT_CONTIGUOUS, 1, (int32_t)pb.seq, 1, 0, 0} : w.q;
  }
  w.window = plan->window;
  w.sinks = plan->sinks;
  w.seq = (int32_t)pb.seq;
  w.scale = prm.scale;
  w.scale_log2 = prm.scale_log2;
  w.step_lo = prm.step_lo;
  w.step_hi = std::min<int32_t>(prm.step_hi, w.k.shards);
  w.kv_rotated = prm.kv_rotated;
  w.n_items = (int32_t)list.count;
  w.items = plan->d_win_items + list.first;
  w.ranges = plan->d_win_ranges;
  w.o = prm.o;
  w.lse = prm.lse;
  w.o_parts = prm.o_parts;
  w.lse_parts = prm.lse_parts;
  w.status = prm.status;
  cudaError_t e;
  const char* why = "windowed f32 forward launch failed";
  if (pb.dtype == RA_DTYPE_BF16)
    e = ra::launch_win_fwd_bf16(w, q, k, v, (int)std::min<int64_t>(list.count, plan->sm_count > 0 ? plan->sm_count : 148), st, &why);
  else
    e = ra::launch_win_fwd_f32(w, static_cast<const float*>(q), static_cast<const float*>(k),
                               static_cast<const float*>(v), st);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "%s: %s", why, cudaGetErrorString(e));
  const ra_status s = mark_use(plan, st);
  return s != RA_OK ? s : ok();
}

// The bf16 backward of a windowed plan: scalars of the rows, dK and dV, dQ, and the sums of
// the key tiles that were cut.
ra_status launch_win_bwd(ra_plan_s* plan, const void* q, const void* k, const void* v, const void* o, const float* lse,
                         const void* dout, void* dq, void* dk, void* dv, float* scratch, cudaStream_t st) {
  const ra_problem& pb = plan->prob;
  ra::WinBwdParams w{};
  w.batch = (int32_t)pb.batch;
  w.heads_q = pb.heads_q;
  w.heads_kv = pb.heads_kv;
  w.group = pb.heads_q / pb.heads_kv;
  w.own = plan->win_own;
  w.str = plan->win_str;
  w.window = plan->window;
  w.sinks = plan->sinks;
  w.seq = (int32_t)pb.seq;
  w.blocks = (w.str.s_n + w.str.tile - 1) / w.str.tile;
  w.scale = pb.scale;
  w.scale_log2 = pb.scale * 1.4426950408889634f;
  w.lse2d = scratch;
  w.n_scalars = plan->win_scalars;
  w.parts = scratch + plan->win_scalars;
  w.dq = dq;
  w.dk = dk;
  w.dv = dv;
  w.q = q;
  w.dout = dout;
  w.ranges = plan->d_win_bwd_ranges;
  w.status = plan->d_status;
  const int sms = plan->sm_count > 0 ? plan->sm_count : 148;
  const char* why = "backward preparation launch failed";
  cudaError_t e = ra::launch_win_bwd_prep(w, o, lse, scratch, sms, st);
  ra::WinBwdParams prm[2] = {w, w};
  for (int pass = 0; pass < 2; ++pass) {
    const int64_t n = pass == 0 ? plan->n_win_bwd_kv : (int64_t)plan->win_bwd_items.size() - plan->n_win_bwd_kv;
    prm[pass].items = plan->d_win_bwd_items + (pass == 0 ? 0 : plan->n_win_bwd_kv);
    prm[pass].n_items = (int32_t)n;
  }
  if (e == cudaSuccess)
    e = ra::launch_win_bwd_bf16(prm, q, k, v, dout, plan->win_bwd_grid, plan->win_bwd_both, st, &why);
  if (e == cudaSuccess && !plan->win_splits.empty()) {
    why = "sum of the parts: launch failed";
    e = ra::launch_win_bwd_join(w, plan->d_win_splits, (int)plan->win_splits.size(), st);
  }
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "%s: %s", why, cudaGetErrorString(e));
  const ra_status s = mark_use(plan, st);
  return s != RA_OK ? s : ok();
}

// Launch the plan's forward kernel (tensor-core for bf16, SIMT for f32) on stream.
ra_status launch(ra_plan_s* plan, const ra::FwdParams& prm, const void* q, const void* k,
                 const void* v, cudaStream_t st) {
  if (plan->window > 0) return launch_win(plan, prm, q, k, v, st);
  cudaError_t e;
  if (plan->prob.dtype == RA_DTYPE_BF16) {
    if (prm.n_items == 0) return ok();
    const int grid = std::min(prm.n_items, plan->sm_count > 0 ? plan->sm_count : 148);
    const char* why = "";
    // The kernel hands out work items from a counter that starts at zero.
    e = cudaMemsetAsync(prm.item_counter, 0, sizeof(uint32_t), st);
    if (e != cudaSuccess) return fail(RA_ERR_CUDA, "counter reset: %s", cudaGetErrorString(e));
    e = ra::launch_fwd_bf16(prm, q, k, v, grid, st, &why);
    if (e == cudaErrorCooperativeLaunchTooLarge) {
      // Not every CTA can be resident (the GPU is shared): the dynamic schedule
      // needs no co-residency and computes the same result.
      cudaGetLastError();
      ra::FwdParams dyn = prm;
      dyn.round_sync = 0;
      e = ra::launch_fwd_bf16(dyn, q, k, v, grid, st, &why);
    }
    if (e != cudaSuccess) return fail(RA_ERR_CUDA, "%s: %s", why, cudaGetErrorString(e));
  } else {
    e = ra::launch_fwd_f32(prm, static_cast<const float*>(q), static_cast<const float*>(k),
                           static_cast<const float*>(v), st);
    if (e != cudaSuccess) return fail(RA_ERR_CUDA, "f32 forward launch failed: %s", cudaGetErrorString(e));
  }
  const ra_status s = mark_use(plan, st);
  return s != RA_OK ? s : ok();
}

ra_status check_device(const ra_plan_s* plan) {
  if (plan->device < 0) return fail(RA_ERR_NO_DEVICE, "plan was built without a CUDA device");
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess || cur != plan->device)
    return fail(RA_ERR_INVALID_ARG, "current device %d differs from the plan's device %d", cur, plan->device);
  return RA_OK;
}

ra_status mark_use(ra_plan_s* plan, cudaStream_t st) { return ra::mark_use(&plan->marks, st); }

size_t elem_bytes(const ra_problem& pb) { return pb.dtype == RA_DTYPE_BF16 ? 2 : 4; }

bool overlap(const void* a, const void* b, size_t bytes) {
  const char* x = static_cast<const char*>(a);
  const char* y = static_cast<const char*>(b);
  return x < y + bytes && y < x + bytes;
}

// The exchange: dst slot (p + 1) mod N <- src slot p for every [S, d] matrix of a
// [B, Hkv, S, d] tensor.  Two strided copy-engine transfers: slots 0..N-2 move up
// by one shard, slot N-1 wraps to slot 0.
cudaError_t rotate_one(const ra_plan_s* plan, const void* src, void* dst, cudaStream_t st) {
  const ra_problem& pb = plan->prob;
  const size_t row = (size_t)pb.head_dim * elem_bytes(pb);
  const size_t pitch = (size_t)pb.seq * row;
  const size_t shard = (size_t)plan->s_n * row;
  const size_t height = (size_t)pb.batch * pb.heads_kv;
  const int N = pb.n_shards;
  const char* s = static_cast<const char*>(src);
  char* d = static_cast<char*>(dst);
  if (N == 1) return cudaMemcpyAsync(d, s, pitch * height, cudaMemcpyDeviceToDevice, st);
  cudaError_t e = cudaMemcpy2DAsync(d + shard, pitch, s, pitch, (size_t)(N - 1) * shard, height,
                                    cudaMemcpyDeviceToDevice, st);
  if (e != cudaSuccess) return e;
  return cudaMemcpy2DAsync(d, pitch, s + (size_t)(N - 1) * shard, pitch, shard, height,
                           cudaMemcpyDeviceToDevice, st);
}

}  // namespace

void ra::set_last_error(const char* msg) { snprintf(g_err, sizeof(g_err), "%s", msg); }

ra_status ra::mark_use(std::vector<StreamMark>* marks, cudaStream_t st) {
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(st, &cap) != cudaSuccess) cudaGetLastError();
  if (cap != cudaStreamCaptureStatusNone) return RA_OK;  // queued into a graph, not run yet
  StreamMark* slot = nullptr;
  for (StreamMark& m : *marks)
    if (m.stream == st) slot = &m;
  if (slot == nullptr)
    for (StreamMark& m : *marks)
      if (cudaEventQuery(m.done) == cudaSuccess) {  // that stream's use has ended
        m.stream = st;
        slot = &m;
        break;
      }
  cudaGetLastError();  // a not-ready query is not an error
  if (slot == nullptr) {
    cudaEvent_t ev = nullptr;
    const cudaError_t e = cudaEventCreateWithFlags(&ev, cudaEventDisableTiming);
    if (e != cudaSuccess) return fail(RA_ERR_CUDA, "use event: %s", cudaGetErrorString(e));
    try {
      marks->push_back({st, ev});
    } catch (const std::exception&) {
      cudaEventDestroy(ev);
      return fail(RA_ERR_UNSUPPORTED, "out of host memory");
    }
    slot = &marks->back();
  }
  const cudaError_t e = cudaEventRecord(slot->done, st);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "use event record: %s", cudaGetErrorString(e));
  return RA_OK;
}

ra_status ra::check_on_current_device(const void* const* ptrs, int n, cudaStream_t stream) {
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) {
    cudaGetLastError();
    return fail(RA_ERR_NO_DEVICE, "no CUDA device");
  }
  for (int i = 0; i < n; ++i) {
    if (ptrs[i] == nullptr) continue;
    cudaPointerAttributes a{};
    const cudaError_t e = cudaPointerGetAttributes(&a, ptrs[i]);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return fail(RA_ERR_INVALID_ARG, "pointer %p: %s", ptrs[i], cudaGetErrorString(e));
    }
    if (a.type == cudaMemoryTypeDevice) {
      if (a.device != cur)
        return fail(RA_ERR_INVALID_ARG, "pointer %p is memory of device %d, the current device is %d", ptrs[i],
                    a.device, cur);
    } else if (a.type != cudaMemoryTypeManaged) {
      return fail(RA_ERR_INVALID_ARG, "pointer %p is not device memory", ptrs[i]);
    }
  }
  // A capturing stream may not be asked for its device (the question would end the
  // capture); a launch on a stream of another device fails by itself.
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess) cudaGetLastError();
  if (cap == cudaStreamCaptureStatusActive) return RA_OK;
  int sd = -1;
  const cudaError_t e = cudaStreamGetDevice(stream, &sd);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(RA_ERR_INVALID_ARG, "stream: %s", cudaGetErrorString(e));
  }
  if (sd != cur) return fail(RA_ERR_INVALID_ARG, "the stream belongs to device %d, the current device is %d", sd, cur);
  return RA_OK;
}

// A plan of a validated problem; window 0 is the whole (causal or full) prefix.
static ra_status make_plan(const ra_problem* prob, int64_t window, int64_t sinks, ra_plan_t* out) {
  ra_plan_s* pl = new (std::nothrow) ra_plan_s();
  if (pl == nullptr) return fail(RA_ERR_UNSUPPORTED, "out of host memory");
  pl->prob = *prob;
  if (pl->prob.scale == 0.f) pl->prob.scale = 1.0f / std::sqrt((float)prob->head_dim);
  pl->s_n = prob->seq / prob->n_shards;
  pl->window = (int32_t)std::min(window, prob->seq);  // (seq fits in 32 bits)
  pl->sinks = (int32_t)std::min(sinks, prob->seq);
  try {
    if (window > 0) build_win_schedule(pl);
    else build_schedule(pl);
  } catch (const std::exception& ex) {  // host allocation of the work lists failed
    delete pl;
    return fail(RA_ERR_UNSUPPORTED, "planning failed on the host: %s", ex.what());
  }
  const ra_status s = upload(pl);
  if (!pl->win_bwd_items.empty()) choose_win_bwd_grids(pl, pl->sm_count > 0 ? pl->sm_count : 148);
  if (s != RA_OK) {
    ra_plan_destroy(pl);
    return s;
  }
  *out = pl;
  return ok();
}

extern "C" {

ra_status ra_plan(const ra_problem* prob, ra_plan_t* out) {
  if (prob == nullptr || out == nullptr) return fail(RA_ERR_INVALID_ARG, "null argument");
  *out = nullptr;
  const ra_status s = validate(prob);
  return s != RA_OK ? s : make_plan(prob, 0, 0, out);
}

ra_status ra_plan_window(const ra_problem* prob, int64_t window, int64_t sinks, ra_plan_t* out) {
  if (prob == nullptr || out == nullptr) return fail(RA_ERR_INVALID_ARG, "null argument");
  *out = nullptr;
  const ra_status s = validate(prob);
  if (s != RA_OK) return s;
  if (prob->causal != 1) return fail(RA_ERR_INVALID_ARG, "a windowed plan is causal: causal must be 1");
  if (window < 1) return fail(RA_ERR_INVALID_ARG, "window must be >= 1");
  if (sinks < 0) return fail(RA_ERR_INVALID_ARG, "sinks must be >= 0");
  // Positions, and their differences of a window, stay in 32 bits; and a work item ends well
  // within the kernels' wait budget (its record is waited for until then): 2^24 keys are
  // 131072 tiles, a fifth of a second.  The backward's items hold a group's heads.
  if (prob->seq > (int64_t(1) << 30)) return fail(RA_ERR_UNSUPPORTED, "seq above 2^30 under a window");
  const int64_t reach = std::min(prob->seq, std::min(window, prob->seq) + std::min(sinks, prob->seq));
  if (prob->dtype == RA_DTYPE_BF16 && reach > (int64_t(1) << 24) / std::max(1, prob->heads_q / prob->heads_kv / 2))
    return fail(RA_ERR_UNSUPPORTED, "window + sinks above 2^24 / max(1, heads_q / heads_kv / 2) keys (bf16)");
  return make_plan(prob, window, sinks, out);
}

ra_status ra_plan_destroy(ra_plan_t plan) {
  if (plan == nullptr) return ok();
  if (plan->device >= 0) {
    int cur = -1;
    cudaGetDevice(&cur);
    if (cur != plan->device) cudaSetDevice(plan->device);
    // Kernels of this plan queued earlier may still read its work tables or its
    // status word: the frees are queued behind them (and only them), in stream
    // order, and the host does not wait.
    if (plan->mem_stream != nullptr) {
      for (const ra::StreamMark& m : plan->marks) cudaStreamWaitEvent(plan->mem_stream, m.done, 0);
      void* mem[] = {plan->d_items,      plan->d_step_items,    plan->d_bwd_items,      plan->d_gather_items,
                     plan->d_win_items,  plan->d_win_ranges,    plan->d_win_bwd_items,  plan->d_win_bwd_ranges,
                     plan->d_win_splits, plan->d_status};
      for (void* p : mem)
        if (p != nullptr) cudaFreeAsync(p, plan->mem_stream);
      cudaStreamDestroy(plan->mem_stream);  // released once its queued frees have run
    }
    for (const ra::StreamMark& m : plan->marks) cudaEventDestroy(m.done);
    cudaGetLastError();
    if (plan->ev_entry) cudaEventDestroy(plan->ev_entry);
    if (plan->ev_rot) cudaEventDestroy(plan->ev_rot);
    if (plan->ev_step) cudaEventDestroy(plan->ev_step);
    if (cur >= 0 && cur != plan->device) cudaSetDevice(cur);
  }
  delete plan;
  return ok();
}

ra_status ra_plan_tile_counts(ra_plan_t plan, int64_t* full, int64_t* partial, int64_t* skip) {
  if (plan == nullptr) return fail(RA_ERR_INVALID_ARG, "null plan");
  const size_t n = (size_t)plan->prob.n_shards;
  if (full) std::memcpy(full, plan->full.data(), n * sizeof(int64_t));
  if (partial) std::memcpy(partial, plan->partial.data(), n * sizeof(int64_t));
  if (skip) std::memcpy(skip, plan->skip.data(), n * sizeof(int64_t));
  return ok();
}

ra_status ra_fwd(ra_plan_t plan, const void* q, const void* k, const void* v, void* o, float* lse,
                 float* o_parts, float* lse_parts, void* stream) {
  if (plan == nullptr) return fail(RA_ERR_INVALID_ARG, "null plan");
  if (q == nullptr || k == nullptr || v == nullptr) return fail(RA_ERR_INVALID_ARG, "null q/k/v");
  const bool partials = o_parts != nullptr || lse_parts != nullptr;
  if (partials) {
    if (o_parts == nullptr || lse_parts == nullptr)
      return fail(RA_ERR_INVALID_ARG, "partials mode needs both o_parts and lse_parts");
    if (o != nullptr || lse != nullptr)
      return fail(RA_ERR_INVALID_ARG, "pass either o/lse (fused) or o_parts/lse_parts (partials), not both");
  } else if (o == nullptr) {
    return fail(RA_ERR_INVALID_ARG, "null o");
  }
  const void* ptrs[] = {q, k, v, o, lse, o_parts, lse_parts};
  for (const void* p : ptrs)
    if (p != nullptr && !aligned16(p)) return fail(RA_ERR_INVALID_ARG, "pointer %p is not 16-byte aligned", p);
  ra_status s = check_device(plan);
  if (s == RA_OK) s = ra::check_on_current_device(ptrs, 7, static_cast<cudaStream_t>(stream));
  if (s != RA_OK) return s;
  ra::FwdParams prm = fwd_params(plan);
  prm.items = plan->d_items;
  prm.n_items = (int32_t)plan->items.size();
  prm.o = o;
  prm.lse = lse;
  prm.o_parts = o_parts;
  prm.lse_parts = lse_parts;
  return launch(plan, prm, q, k, v, static_cast<cudaStream_t>(stream));
}

ra_status ra_merge_partials(int32_t n_parts, int64_t rows, int32_t d, const float* o_parts,
                            const float* lse_parts, void* o, int32_t o_dtype, float* lse, void* stream) {
  if (n_parts < 1 || rows < 1 || d < 1 || d > 1024)
    return fail(RA_ERR_INVALID_ARG, "n_parts, rows >= 1 and 1 <= d <= 1024 required");
  if (o_dtype != RA_DTYPE_F32 && o_dtype != RA_DTYPE_BF16) return fail(RA_ERR_INVALID_ARG, "bad o_dtype");
  if (o_parts == nullptr || lse_parts == nullptr || o == nullptr)
    return fail(RA_ERR_INVALID_ARG, "null pointer");
  const void* ptrs[] = {o_parts, lse_parts, o, lse};
  for (const void* p : ptrs)
    if (p != nullptr && !aligned16(p)) return fail(RA_ERR_INVALID_ARG, "pointer %p is not 16-byte aligned", p);
  const ra_status s = ra::check_on_current_device(ptrs, 4, static_cast<cudaStream_t>(stream));
  if (s != RA_OK) return s;
  cudaError_t e = ra::launch_merge(n_parts, rows, d, o_parts, lse_parts, o, o_dtype, lse,
                                   static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "merge launch failed: %s", cudaGetErrorString(e));
  return ok();
}

ra_status ra_layout_perm(int32_t layout, int64_t seq, int32_t n_shards, int32_t inverse,
                         int64_t rows_outer, int32_t row_bytes, const void* src, void* dst, void* stream) {
  ra_status s = check_layout(layout, seq, n_shards);
  if (s != RA_OK) return s;
  if (rows_outer < 1 || row_bytes < 4 || row_bytes % 4)
    return fail(RA_ERR_INVALID_ARG, "rows_outer >= 1 and row_bytes a positive multiple of 4 required");
  if (rows_outer > INT64_MAX / seq / row_bytes) return fail(RA_ERR_UNSUPPORTED, "tensor above 2^63-1 bytes");
  if (src == nullptr || dst == nullptr) return fail(RA_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(src) || !aligned16(dst)) return fail(RA_ERR_INVALID_ARG, "src/dst must be 16-byte aligned");
  const int64_t bytes = rows_outer * seq * (int64_t)row_bytes;
  const char* a = static_cast<const char*>(src);
  const char* b = static_cast<const char*>(dst);
  if (a < b + bytes && b < a + bytes) return fail(RA_ERR_INVALID_ARG, "src and dst overlap");
  const void* ptrs[] = {src, dst};
  s = ra::check_on_current_device(ptrs, 2, static_cast<cudaStream_t>(stream));
  if (s != RA_OK) return s;
  cudaError_t e = ra::launch_layout_perm(layout, seq, n_shards, inverse ? 1 : 0, rows_outer, row_bytes,
                                         src, dst, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "layout permute launch failed: %s", cudaGetErrorString(e));
  return ok();
}

ra_status ra_layout_index(int32_t layout, int64_t seq, int32_t n_shards, int64_t* pos_out) {
  ra_status s = check_layout(layout, seq, n_shards);
  if (s != RA_OK) return s;
  if (pos_out == nullptr) return fail(RA_ERR_INVALID_ARG, "null pos_out");
  const int64_t s_n = seq / n_shards;
  for (int p = 0; p < n_shards; ++p)
    for (int64_t i = 0; i < s_n; ++i) pos_out[p * s_n + i] = ra::pos_of(layout, n_shards, s_n, p, i);
  return ok();
}

ra_status ra_fwd_step(ra_plan_t plan, int32_t step, const void* q, const void* k_blk, const void* v_blk,
                      float* o_part, float* lse_part, void* stream) {
  if (plan == nullptr) return fail(RA_ERR_INVALID_ARG, "null plan");
  const ra_problem& pb = plan->prob;
  if (step < 0 || step >= pb.n_shards)
    return fail(RA_ERR_INVALID_ARG, "step %d outside 0..%d", step, pb.n_shards - 1);
  if (q == nullptr || k_blk == nullptr || v_blk == nullptr || o_part == nullptr || lse_part == nullptr)
    return fail(RA_ERR_INVALID_ARG, "null pointer");
  const void* ptrs[] = {q, k_blk, v_blk, o_part, lse_part};
  for (const void* p : ptrs)
    if (!aligned16(p)) return fail(RA_ERR_INVALID_ARG, "pointer %p is not 16-byte aligned", p);
  ra_status s = check_device(plan);
  if (s == RA_OK) s = ra::check_on_current_device(ptrs, 5, static_cast<cudaStream_t>(stream));
  if (s != RA_OK) return s;
  ra::FwdParams prm = fwd_params(plan);
  prm.step_lo = (int16_t)step;
  prm.step_hi = (int16_t)(step + 1);
  prm.kv_rotated = 1;
  if (!plan->step_off.empty()) {
    prm.items = plan->d_step_items + plan->step_off[step];
    prm.n_items = (int32_t)(plan->step_off[step + 1] - plan->step_off[step]);
  }
  prm.o_parts = o_part;
  prm.lse_parts = lse_part;
  return launch(plan, prm, q, k_blk, v_blk, static_cast<cudaStream_t>(stream));
}

ra_status ra_ring_rotate(ra_plan_t plan, const void* k_src, const void* v_src, void* k_dst, void* v_dst,
                         void* stream) {
  if (plan == nullptr) return fail(RA_ERR_INVALID_ARG, "null plan");
  if (k_src == nullptr || v_src == nullptr || k_dst == nullptr || v_dst == nullptr)
    return fail(RA_ERR_INVALID_ARG, "null pointer");
  const ra_problem& pb = plan->prob;
  const size_t bytes = (size_t)pb.batch * pb.heads_kv * pb.seq * pb.head_dim * elem_bytes(pb);
  if (overlap(k_src, k_dst, bytes) || overlap(v_src, v_dst, bytes) || overlap(k_dst, v_dst, bytes))
    return fail(RA_ERR_INVALID_ARG, "a destination overlaps its source or the other destination");
  ra_status s = check_device(plan);
  const void* ptrs[] = {k_src, v_src, k_dst, v_dst};
  if (s == RA_OK) s = ra::check_on_current_device(ptrs, 4, static_cast<cudaStream_t>(stream));
  if (s != RA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = rotate_one(plan, k_src, k_dst, st);
  if (e == cudaSuccess) e = rotate_one(plan, v_src, v_dst, st);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "rotation copy failed: %s", cudaGetErrorString(e));
  return ok();
}

ra_status ra_ring_fwd(ra_plan_t plan, const void* q, const void* k, const void* v, void* o, float* lse,
                      void* k_buf, void* v_buf, float* o_parts, float* lse_parts, void* stream,
                      void* comm_stream) {
  if (plan == nullptr) return fail(RA_ERR_INVALID_ARG, "null plan");
  const ra_problem& pb = plan->prob;
  const int N = pb.n_shards;
  if (q == nullptr || k == nullptr || v == nullptr || o == nullptr || o_parts == nullptr ||
      lse_parts == nullptr || (N > 1 && (k_buf == nullptr || v_buf == nullptr)))
    return fail(RA_ERR_INVALID_ARG, "null pointer");
  const void* ptrs[] = {q, k, v, o, lse, k_buf, v_buf, o_parts, lse_parts};
  for (const void* p : ptrs)
    if (p != nullptr && !aligned16(p)) return fail(RA_ERR_INVALID_ARG, "pointer %p is not 16-byte aligned", p);
  const size_t kv_bytes = (size_t)pb.batch * pb.heads_kv * pb.seq * pb.head_dim * elem_bytes(pb);
  if (N > 1 && (overlap(k_buf, v_buf, 2 * kv_bytes) || overlap(k_buf, k, kv_bytes) ||
                overlap(k_buf, v, kv_bytes) || overlap(v_buf, k, kv_bytes) || overlap(v_buf, v, kv_bytes)))
    return fail(RA_ERR_INVALID_ARG, "receive buffers overlap each other or K/V");
  ra_status s = check_device(plan);
  if (s == RA_OK) s = ra::check_on_current_device(ptrs, 9, static_cast<cudaStream_t>(stream));
  if (s == RA_OK) s = ra::check_on_current_device(nullptr, 0, static_cast<cudaStream_t>(comm_stream));
  if (s != RA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaStream_t cs = static_cast<cudaStream_t>(comm_stream);
  const int64_t rows = pb.batch * (int64_t)pb.heads_q * pb.seq;
  char* kb = static_cast<char*>(k_buf);
  char* vb = static_cast<char*>(v_buf);
  cudaError_t e = cudaSuccess;
  auto cuda_fail = [&](const char* what) { return fail(RA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e)); };

  // The communication stream starts after everything already queued on stream
  // (the caller's writes of K and V, earlier users of the receive buffers).
  if ((e = cudaEventRecord(plan->ev_entry, st)) != cudaSuccess) return cuda_fail("event record");
  if ((e = cudaStreamWaitEvent(cs, plan->ev_entry, 0)) != cudaSuccess) return cuda_fail("stream wait");
  for (int t = 0; t < N; ++t) {
    // Block held at step t: K/V themselves at step 0, then receive buffer (t - 1) % 2.
    const void* kt = t == 0 ? k : kb + (size_t)((t - 1) % 2) * kv_bytes;
    const void* vt = t == 0 ? v : vb + (size_t)((t - 1) % 2) * kv_bytes;
    if (t >= 1 && (e = cudaStreamWaitEvent(st, plan->ev_rot, 0)) != cudaSuccess) return cuda_fail("stream wait");
    if (t + 1 < N) {
      // Pass the block on while step t computes.  Its destination was last read
      // by step t - 1.
      if (t >= 2 && (e = cudaStreamWaitEvent(cs, plan->ev_step, 0)) != cudaSuccess) return cuda_fail("stream wait");
      s = ra_ring_rotate(plan, kt, vt, kb + (size_t)(t % 2) * kv_bytes, vb + (size_t)(t % 2) * kv_bytes, cs);
      if (s != RA_OK) return s;
      if ((e = cudaEventRecord(plan->ev_rot, cs)) != cudaSuccess) return cuda_fail("event record");
    }
    s = ra_fwd_step(plan, t, q, kt, vt, o_parts + (size_t)t * rows * pb.head_dim, lse_parts + (size_t)t * rows, st);
    if (s != RA_OK) return s;
    if ((e = cudaEventRecord(plan->ev_step, st)) != cudaSuccess) return cuda_fail("event record");
  }
  return ra_merge_partials(N, rows, pb.head_dim, o_parts, lse_parts, o, pb.dtype, lse, st);
}

ra_status ra_bwd_scratch_size(ra_plan_t plan, int64_t* bytes) {
  if (plan == nullptr || bytes == nullptr) return fail(RA_ERR_INVALID_ARG, "null argument");
  const ra_problem& pb = plan->prob;
  if (plan->window > 0 && pb.dtype == RA_DTYPE_BF16) {
    *bytes = (plan->win_scalars + plan->win_parts) * (int64_t)sizeof(float);
    return ok();
  }
  const int64_t n64 = (plan->s_n + 63) / 64;
  *bytes = pb.batch * (int64_t)pb.heads_q * pb.n_shards * n64 * 128 * (int64_t)sizeof(float);
  return ok();
}

ra_status ra_bwd(ra_plan_t plan, const void* q, const void* k, const void* v, const void* o, const float* lse,
                 const void* dout, void* dq, void* dk, void* dv, float* scratch, void* stream) {
  if (plan == nullptr) return fail(RA_ERR_INVALID_ARG, "null plan");
  const ra_problem& pb = plan->prob;
  const void* ptrs[] = {q, k, v, o, lse, dout, dq, dk, dv, scratch};
  for (const void* p : ptrs) {
    if (p == nullptr) return fail(RA_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(p)) return fail(RA_ERR_INVALID_ARG, "pointer %p is not 16-byte aligned", p);
  }
  ra_status s = check_device(plan);
  if (s == RA_OK) s = ra::check_on_current_device(ptrs, 10, static_cast<cudaStream_t>(stream));
  if (s != RA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (plan->window > 0 && pb.dtype == RA_DTYPE_BF16)
    return launch_win_bwd(plan, q, k, v, o, lse, dout, dq, dk, dv, scratch, st);
  const int64_t n64 = (plan->s_n + 63) / 64;
  cudaError_t e = ra::launch_bwd_prep(pb.dtype, pb.batch * (int64_t)pb.heads_q, pb.seq, pb.n_shards, pb.head_dim, o,
                                      dout, lse, scratch, st);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "backward preparation launch failed: %s", cudaGetErrorString(e));

  ra::BwdParams prm{};
  prm.batch = (int32_t)pb.batch;
  prm.heads_q = pb.heads_q;
  prm.heads_kv = pb.heads_kv;
  prm.group = pb.heads_q / pb.heads_kv;
  prm.head_dim = pb.head_dim;
  prm.n_shards = pb.n_shards;
  prm.layout = (int16_t)pb.layout;
  prm.causal = (int16_t)pb.causal;
  prm.seq = pb.seq;
  prm.s_n = plan->s_n;
  prm.scale = pb.scale;
  prm.scale_log2 = pb.scale * 1.4426950408889634f;
  prm.lse2d = scratch;
  prm.n64 = n64;
  prm.dq = dq;
  prm.dk = dk;
  prm.dv = dv;
  prm.q = q;
  prm.dout = dout;
  prm.status = plan->d_status;
  prm.item_counter = plan->d_status + 1;
  if (pb.dtype != RA_DTYPE_BF16) {
    const float *qf = static_cast<const float*>(q), *kf = static_cast<const float*>(k), *vf = static_cast<const float*>(v),
                *df = static_cast<const float*>(dout);
    e = plan->window > 0 ? ra::launch_win_bwd_f32(prm, plan->window, plan->sinks, qf, kf, vf, df, st)
                         : ra::launch_bwd_f32(prm, qf, kf, vf, df, st);
    if (e != cudaSuccess) return fail(RA_ERR_CUDA, "f32 backward launch failed: %s", cudaGetErrorString(e));
    s = mark_use(plan, st);
    return s != RA_OK ? s : ok();
  }
  const int sms = plan->sm_count > 0 ? plan->sm_count : 148;
  for (int pass = 0; pass < 2; ++pass) {
    const int64_t n = pass == 0 ? plan->n_bwd_kv : (int64_t)plan->bwd_items.size() - plan->n_bwd_kv;
    prm.items = plan->d_bwd_items + (pass == 0 ? 0 : plan->n_bwd_kv);
    prm.n_items = (int32_t)n;
    if (n == 0) continue;
    // each pass hands out work items from a counter that starts at zero
    e = cudaMemsetAsync(prm.item_counter, 0, sizeof(uint32_t), st);
    if (e != cudaSuccess) return fail(RA_ERR_CUDA, "counter reset: %s", cudaGetErrorString(e));
    const char* why = "";
    prm.round_sync = plan->bwd_round_sync[pass] ? 1 : 0;
    e = ra::launch_bwd_bf16(pass, prm, q, k, v, dout, (int)std::min<int64_t>(n, sms), st, &why);
    if (e == cudaErrorCooperativeLaunchTooLarge) {  // not every CTA resident: dynamic schedule
      cudaGetLastError();
      prm.round_sync = 0;
      e = ra::launch_bwd_bf16(pass, prm, q, k, v, dout, (int)std::min<int64_t>(n, sms), st, &why);
    }
    if (e != cudaSuccess) return fail(RA_ERR_CUDA, "%s: %s", why, cudaGetErrorString(e));
  }
  s = mark_use(plan, st);
  return s != RA_OK ? s : ok();
}

ra_status ra_allgather_kv(ra_plan_t plan, const void* k, const void* v, void* k_all, void* v_all, void* stream) {
  if (plan == nullptr) return fail(RA_ERR_INVALID_ARG, "null plan");
  const ra_problem& pb = plan->prob;
  const void* ptrs[] = {k, v, k_all, v_all};
  for (const void* p : ptrs) {
    if (p == nullptr) return fail(RA_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(p)) return fail(RA_ERR_INVALID_ARG, "pointer %p is not 16-byte aligned", p);
  }
  const size_t bytes = (size_t)pb.batch * pb.heads_kv * pb.seq * pb.head_dim * elem_bytes(pb);
  if (overlap(k, k_all, bytes) || overlap(v, v_all, bytes) || overlap(k_all, v_all, bytes))
    return fail(RA_ERR_INVALID_ARG, "a destination overlaps its source or the other destination");
  ra_status s = check_device(plan);
  if (s == RA_OK) s = ra::check_on_current_device(ptrs, 4, static_cast<cudaStream_t>(stream));
  if (s != RA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int row_bytes = pb.head_dim * (int)elem_bytes(pb);
  const int64_t outer = pb.batch * (int64_t)pb.heads_kv;
  // layout order -> natural order: every shard's rows land at their positions
  cudaError_t e = ra::launch_layout_perm(pb.layout, pb.seq, pb.n_shards, 1, outer, row_bytes, k, k_all, st);
  if (e == cudaSuccess) e = ra::launch_layout_perm(pb.layout, pb.seq, pb.n_shards, 1, outer, row_bytes, v, v_all, st);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "gather launch failed: %s", cudaGetErrorString(e));
  return ok();
}

ra_status ra_fwd_gathered(ra_plan_t plan, const void* q, const void* k_all, const void* v_all, void* o, float* lse,
                          void* stream) {
  if (plan == nullptr) return fail(RA_ERR_INVALID_ARG, "null plan");
  if (q == nullptr || k_all == nullptr || v_all == nullptr || o == nullptr)
    return fail(RA_ERR_INVALID_ARG, "null pointer");
  const void* ptrs[] = {q, k_all, v_all, o, lse};
  for (const void* p : ptrs)
    if (p != nullptr && !aligned16(p)) return fail(RA_ERR_INVALID_ARG, "pointer %p is not 16-byte aligned", p);
  ra_status s = check_device(plan);
  if (s == RA_OK) s = ra::check_on_current_device(ptrs, 5, static_cast<cudaStream_t>(stream));
  if (s != RA_OK) return s;
  ra::FwdParams prm = fwd_params(plan);
  prm.gathered = 1;
  prm.step_lo = 0;
  prm.step_hi = 1;
  prm.items = plan->d_gather_items;
  prm.n_items = (int32_t)plan->gather_items.size();
  prm.round_sync = plan->gather_round_sync ? 1 : 0;
  prm.o = o;
  prm.lse = lse;
  return launch(plan, prm, q, k_all, v_all, static_cast<cudaStream_t>(stream));
}

ra_status ra_ulysses_a2a(int32_t direction, int32_t layout, int64_t seq, int32_t n_shards, int64_t batch,
                          int32_t heads, int32_t row_bytes, const void* src, void* dst, void* stream) {
  ra_status s = check_layout(layout, seq, n_shards);
  if (s != RA_OK) return s;
  if (direction != 0 && direction != 1) return fail(RA_ERR_INVALID_ARG, "direction must be 0 or 1");
  if (batch < 1 || heads < 1 || heads % n_shards)
    return fail(RA_ERR_INVALID_ARG, "batch >= 1 and heads a positive multiple of n_shards required");
  if (row_bytes != 256 && row_bytes != 4)
    return fail(RA_ERR_UNSUPPORTED, "row_bytes must be 256 (d = 128 bf16) or 4 (one float)");
  if (batch > INT32_MAX || batch * (int64_t)heads * seq > INT32_MAX)
    return fail(RA_ERR_UNSUPPORTED, "B*H*S above 2^31-1 rows");
  if (src == nullptr || dst == nullptr) return fail(RA_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(src) || !aligned16(dst)) return fail(RA_ERR_INVALID_ARG, "src/dst must be 16-byte aligned");
  if (overlap(src, dst, (size_t)(batch * heads * seq) * row_bytes))
    return fail(RA_ERR_INVALID_ARG, "src and dst overlap");
  const void* ptrs[] = {src, dst};
  s = ra::check_on_current_device(ptrs, 2, static_cast<cudaStream_t>(stream));
  if (s != RA_OK) return s;
  cudaError_t e = ra::launch_ulysses_a2a(direction, layout, n_shards, (int)batch, heads, seq, row_bytes, src, dst,
                                         static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "exchange launch failed: %s", cudaGetErrorString(e));
  return ok();
}

ra_status ra_wait_selftest(uint32_t* status_out) {
  if (status_out == nullptr) return fail(RA_ERR_INVALID_ARG, "null status_out");
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return fail(RA_ERR_NO_DEVICE, "no CUDA device");
  }
  uint32_t* d_word = nullptr;
  cudaError_t e = cudaMalloc(&d_word, sizeof(uint32_t));
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "status word: %s", cudaGetErrorString(e));
  e = cudaMemset(d_word, 0, sizeof(uint32_t));
  if (e == cudaSuccess) e = ra::launch_wait_selftest(d_word, nullptr);
  if (e == cudaSuccess) e = cudaMemcpy(status_out, d_word, sizeof(uint32_t), cudaMemcpyDeviceToHost);
  cudaFree(d_word);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "wait self-test: %s", cudaGetErrorString(e));
  return ok();
}

ra_status ra_sync_status(ra_plan_t plan, void* stream) {
  if (plan == nullptr) return fail(RA_ERR_INVALID_ARG, "null plan");
  if (plan->device < 0) return fail(RA_ERR_NO_DEVICE, "plan was built without a CUDA device");
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "stream synchronize: %s", cudaGetErrorString(e));
  uint32_t word = 0;
  e = cudaMemcpy(&word, plan->d_status, sizeof(word), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return fail(RA_ERR_CUDA, "status read: %s", cudaGetErrorString(e));
  if (word != 0) {
    // cleared before a launch on a stream that does not wait for the default one can set it
    e = cudaMemset(plan->d_status, 0, sizeof(word));
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) return fail(RA_ERR_CUDA, "status clear: %s", cudaGetErrorString(e));
    char msg[200];
    const ra_status code = ra::status_word_error(word, msg, sizeof(msg));
    return fail(code, "%s", msg);
  }
  return ok();
}

const char* ra_last_error(void) { return g_err; }

}  // extern "C"
