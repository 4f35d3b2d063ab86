// Every work list of a windowed plan against the mask, pair by pair (test_window_lists_host.py).
//
// Built from the planner's own source, without a device: expands each list as the kernels
// do -- items, ranges, tiles, the columns that a row sees (win_internal.h) -- down to rows of
// the tensors, and counts how often each (query, key) pair enters a sum.  A pair that is seen
// has to enter once, any other not at all; the backward's parts of a cut tile have to be those
// that the last kernel adds.  One line of input is a case:
//   batch seq heads_q heads_kv n_shards layout window sinks
// and one line of output is a fault ("ok N" at the end: cases looked at).
#include "ra_api.cu"

#include <cinttypes>
#include <map>
#include <string>

namespace {

struct Case {
  ra_problem pb;
  int window, sinks;
  std::string name;
};

int faults = 0;
void fault(const Case& c, const char* what, int64_t a, int64_t b, int64_t got) {
  if (++faults <= 40) printf("%s: %s (%" PRId64 ", %" PRId64 "): %" PRId64 "\n", c.name.c_str(), what, a, b, got);
}

// Position of row m of a head in the plan's layout.
int64_t position(const ra_problem& pb, int64_t m) {
  const int64_t s_n = pb.seq / pb.n_shards;
  return ra::pos_of(pb.layout, pb.n_shards, s_n, (int)(m / s_n), m % s_n);
}
// Row of a head that column x of a tensor-map box beginning at row0 of a view's shard holds.
int64_t box_row(const ra::WinView& v, int64_t seq, int shard, int64_t row0, int64_t x) {
  const int64_t i = ((int64_t)shard * v.s_n + row0) / v.stripe;
  return x % v.stripe * (seq / v.stripe) + i + x / v.stripe;
}
// Row of a head at which the kernels write own row `row` of a view's shard.
int64_t out_row(const ra::WinView& v, int64_t seq, int shard, int64_t row) {
  const int64_t head_row = (int64_t)shard * v.s_n + row;
  return v.stripe == 1 ? head_row : head_row % v.stripe * (seq / v.stripe) + head_row / v.stripe;
}

struct Counts {
  int64_t seq;
  std::vector<int> n;
  Counts(int64_t heads, int64_t seq) : seq(seq), n((size_t)(heads * seq * seq), 0) {}
  int& at(int64_t head, int64_t i, int64_t j) { return n[(size_t)((head * seq + i) * seq + j)]; }
};
void check(const Case& c, Counts& got, int64_t heads, const char* what) {
  for (int64_t h = 0; h < heads; ++h)
    for (int64_t i = 0; i < c.pb.seq; ++i)
      for (int64_t j = 0; j < c.pb.seq; ++j) {
        const bool seen = j <= i && (j > i - c.window || j < c.sinks);
        if (got.at(h, i, j) != (int)seen) {
          fault(c, what, i, j, got.at(h, i, j));
          return;
        }
      }
}

void forward(const Case& c, ra_plan_s* pl, int which) {
  const ra_problem& pb = c.pb;
  const ra_plan_s::WinList& list = pl->win_lists[which];
  const bool gathered = which == 2;
  const int64_t heads = pb.batch * pb.heads_q;
  Counts got(heads, pb.seq);
  for (int64_t x = list.first; x < list.first + list.count; ++x) {
    const ra::WinItem& it = pl->win_items[(size_t)x];
    int32_t tiles = 0;
    for (int k = 0; k < it.n_ranges; ++k) {
      const ra::WinRange& rg = pl->win_ranges[(size_t)(it.range0 + k)];
      const int n = ra::range_tiles(rg, list.k.tile);
      tiles += n;
      if (rg.row0 < 0 || rg.row0 >= rg.end || rg.end > list.k.s_n || rg.row0 % list.k.stripe)
        fault(c, "range", rg.row0, rg.end, x);
      if (k > 0 && pl->win_ranges[(size_t)(it.range0 + k - 1)].step > rg.step) fault(c, "steps in order", x, k, rg.step);
      if (list.k.shards > 1 && rg.r != ((it.shard - rg.step) % pb.n_shards + pb.n_shards) % pb.n_shards)
        fault(c, "shard of a step", x, k, rg.r);
      for (int g = 0; g < (it.bh1 >= 0 ? 2 : 1); ++g)
        for (int row = 0; row < list.q.tile; ++row) {
          const int i = (g ? it.row1 : it.row0) + row;
          if (i >= it.row_end) break;
          const int64_t m = out_row(list.q, pb.seq, it.shard, i);
          const int64_t pos = position(pb, m);
          const int64_t own = (g ? it.pos1 : it.pos0) + (int64_t)row * list.q.apart;
          if (own != pos) fault(c, "position of a query", m, own, pos);
          const ra::WinColumns seen = ra::range_columns(rg, list.k.apart, c.window, c.sinks, (int32_t)own);
          for (int kt = 0; kt < n; ++kt)
            for (int col = 0; col < list.k.tile; ++col) {
              const int y = kt * list.k.tile + col;
              if (y >= seen.hi || !(y >= seen.lo || y < seen.sk)) continue;
              const int64_t key = box_row(list.k, pb.seq, rg.r, rg.row0 + kt * list.k.tile, col);
              if (key < 0 || key >= pb.seq) fault(c, "key row", x, y, key);
              else ++got.at(g ? it.bh1 : it.bh0, pos, gathered ? key : position(pb, key));
            }
        }
    }
    if (tiles != it.n_tiles) fault(c, "tiles of an item", x, tiles, it.n_tiles);
  }
  const char* names[] = {"ring list", "fused list", "gathered list"};
  check(c, got, heads, names[which]);
}

template <int kPass>
void backward(const Case& c, ra_plan_s* pl) {
  const ra_problem& pb = c.pb;
  const int G = pb.heads_q / pb.heads_kv;
  ra::WinBwdParams P{};
  P.own = pl->win_own;
  P.str = pl->win_str;
  P.window = pl->window;
  P.sinks = pl->sinks;
  P.seq = (int32_t)pb.seq;
  const int64_t heads = pb.batch * pb.heads_q;
  Counts got(heads, pb.seq);
  std::map<int64_t, int> parts;  // first float -> rows
  const int64_t first = kPass == 0 ? 0 : pl->n_win_bwd_kv;
  const int64_t last = kPass == 0 ? pl->n_win_bwd_kv : (int64_t)pl->win_bwd_items.size();
  for (int64_t x = first; x < last; ++x) {
    const ra::WinBwdItem& it = pl->win_bwd_items[(size_t)x];
    if (kPass == 0 && it.part >= 0) {
      if (!parts.emplace(it.part, it.part_rows).second) fault(c, "part written twice", x, it.part, it.part_rows);
      if (it.part + 2 * (int64_t)it.part_rows * 128 > pl->win_parts) fault(c, "part beyond the scratch", x, it.part, pl->win_parts);
    }
    int32_t tiles = 0;
    for (int head = it.g0; head < it.g1; ++head) {
      const int64_t bh = kPass == 0 ? (int64_t)it.bh / pb.heads_kv * pb.heads_q + it.bh % pb.heads_kv * G + head : it.bh;
      for (int k = 0; k < it.n_ranges; ++k) {
        const ra::WinBwdRange& rg = pl->win_bwd_ranges[(size_t)(it.range0 + k)];
        const int n = ra::range_tiles64(rg, P.str.tile);
        tiles += n;
        if (rg.row0 < 0 || rg.row0 >= rg.end || rg.end > P.str.s_n || rg.row0 % P.str.tile)
          fault(c, "range", rg.row0, rg.end, x);
        for (int row = 0; row < P.own.tile; ++row) {
          const int i = it.row0 + row;
          if (i >= it.row_end) break;
          if (kPass == 0 && it.part >= 0 && row >= it.part_rows) break;  // (not written)
          const int64_t m = out_row(P.own, pb.seq, it.shard, i);
          const int64_t pos = position(pb, m), own = it.pos0 + (int64_t)row * P.own.apart;
          if (own != pos) fault(c, "position of an own row", m, own, pos);
          const ra::WinBwdColumns live = ra::range_columns<kPass>(P, rg, (int32_t)own);
          for (int kt = 0; kt < n; ++kt)
            for (int col = 0; col < P.str.tile; ++col) {
              const int y = kt * P.str.tile + col;
              if (!((y >= live.lo && y < live.hi) || (y >= live.from && y < live.sk))) continue;
              const int64_t other = box_row(P.str, pb.seq, rg.r, rg.row0 + kt * P.str.tile, col);
              if (other < 0 || other >= pb.seq) fault(c, "streamed row", x, y, other);
              else if (kPass == 0) ++got.at(bh, position(pb, other), pos);
              else ++got.at(bh, pos, position(pb, other));
            }
        }
      }
    }
    if (tiles != it.n_tiles) fault(c, "tiles of an item", x, tiles, it.n_tiles);
  }
  check(c, got, heads, kPass == 0 ? "dK, dV list" : "dQ list");
  if (kPass != 0) return;
  // What the last kernel adds is what the items left.
  for (const ra::WinBwdSplit& sp : pl->win_splits) {
    for (int n = 0; n < sp.n_near; ++n)
      if (parts.count(sp.near + n * 2 * 128 * 128) == 0 || parts[sp.near + n * 2 * 128 * 128] != 128) fault(c, "near part", sp.near, n, 0);
      else parts.erase(sp.near + n * 2 * 128 * 128);
    for (int n = 0; n < sp.n_far; ++n) {
      const int64_t at = sp.far + (int64_t)n * 2 * sp.far_rows * 128;
      if (parts.count(at) == 0 || parts[at] != sp.far_rows) fault(c, "far part", sp.far, n, 0);
      else parts.erase(at);
    }
  }
  if (!parts.empty()) fault(c, "parts that nobody adds", (int64_t)parts.size(), parts.begin()->first, 0);
}

}  // namespace

int main() {
  char line[256];
  int cases = 0;
  while (fgets(line, sizeof(line), stdin) != nullptr) {
    Case c{};
    long long batch, seq;
    if (sscanf(line, "%lld %lld %d %d %d %d %d %d", &batch, &seq, &c.pb.heads_q, &c.pb.heads_kv, &c.pb.n_shards,
               &c.pb.layout, &c.window, &c.sinks) != 8)
      return 2;
    c.pb.batch = batch;
    c.pb.seq = seq;
    c.pb.head_dim = 128;
    c.pb.causal = 1;
    c.pb.dtype = RA_DTYPE_BF16;
    c.name = std::string(line, strcspn(line, "\n"));
    if (validate(&c.pb) != RA_OK) {
      printf("%s: %s\n", c.name.c_str(), g_err);
      return 3;
    }
    ra_plan_s pl;
    pl.prob = c.pb;
    pl.s_n = seq / c.pb.n_shards;
    pl.window = (int32_t)std::min<int64_t>(c.window, seq);
    pl.sinks = (int32_t)std::min<int64_t>(c.sinks, seq);
    build_win_schedule(&pl);
    for (int which = 0; which < 3; ++which) forward(c, &pl, which);
    backward<0>(c, &pl);
    backward<1>(c, &pl);
    ++cases;
  }
  printf("ok %d\n", cases);
  return faults != 0;
}
