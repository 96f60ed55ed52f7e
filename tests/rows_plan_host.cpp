// Host check of the row planner (csrc/serving/rows_plan.cuh, rows_chunks.cuh) that
// gdattn_decode_sink and gdattn_decode_prefix walk by, on random ragged batches:
// - the tiles of a unit hold each position that some row of the block sees, once,
//   in slots inside the cache, the right slot for each position, and no tile
//   crosses the pinned slots' end of a run or the ring's;
// - a row's visible positions are the definition's, and all are in its unit's tiles;
// - chunks are equal and cover all tiles; segments cover every unit's tiles once;
// - no two partials share a slot, all slots are inside the array, and the merge
//   finds exactly the pieces of every unit that was cut (or, with a prefix, of
//   every unit).
// Prints "ok <cases>", or the first failure, and exits non-zero on failure.
#include "warp_emulation.h"

#include <map>
#include <set>
#include <utility>

#define GDATTN_HD inline
#include "rows_chunks.cuh"

using namespace gdattn;

namespace {

void fail(const char *what, int k) {
  fprintf(stderr, "case %d: %s\n", k, what);
  exit(1);
}

struct PlanCall {
  const RowsGeom *g;
  int32_t c, workers;
  RowsPlan plan;
};
PlanCall g_call;

RowsPlan plan_of(const RowsGeom &g, int32_t c, int32_t workers) {
  g_call.g = &g;
  g_call.c = c;
  g_call.workers = workers;
  run_warp(
      [](void *) {
        const RowsPlan p = plan_rows(*g_call.g, g_call.c, g_call.workers);
        if ((threadIdx.x & 31) == 0) g_call.plan = p;
      },
      nullptr);
  return g_call.plan;
}

// Positions that a token sees, by the definition.
bool sees_own(const RowsGeom &g, int32_t L, int32_t t, int32_t j) {
  const int64_t p = static_cast<int64_t>(L) - g.tokens + t;
  if (L <= 0 || p < 0 || j > p || j < 0) return false;
  return g.window == 0 || j > p - g.window || j < g.sinks;
}
bool sees_prefix(const RowsGeom &g, int32_t L, int32_t t, int32_t P, int32_t j) {
  const int64_t p = static_cast<int64_t>(L) - g.tokens + t;
  if (L <= 0 || p < 0 || j >= P || j < 0) return false;
  return g.window == 0 || j > P + p - g.window;
}

std::map<int32_t, int32_t> positions(const UnitTiles &u, int32_t capacity, int k) {
  std::map<int32_t, int32_t> slot_of_pos;
  for (int32_t t = 0; t < u.n; ++t) {
    const RowTile tile = unit_tile(u, t);
    if (tile.ntok < 0 || tile.ntok > kRowTile) fail("tile size", k);
    if (tile.slot < 0 || tile.slot + tile.ntok > capacity) fail("tile leaves the cache", k);
    if (tile.ntok == 0 && u.n != 1) fail("empty tile in a unit of several", k);
    for (int32_t i = 0; i < tile.ntok; ++i)
      if (!slot_of_pos.emplace(tile.pos + i, tile.slot + i).second) fail("position twice", k);
  }
  return slot_of_pos;
}

void check_case(std::mt19937_64 &rng, int k) {
  auto pick = [&](int32_t lo, int32_t hi) {
    return std::uniform_int_distribution<int32_t>(lo, hi)(rng);
  };
  RowsGeom g = {};
  const bool with_prefix = pick(0, 1) == 1;
  g.batch = pick(1, pick(0, 3) ? 6 : 40);
  g.tokens = pick(0, 1) ? 1 : pick(1, pick(0, 1) ? 9 : 150);
  g.group = (int[]){1, 2, 3, 16, 128}[pick(0, 4)];
  g.n_kv_heads = pick(1, 3);
  g.window = (with_prefix && pick(0, 1)) ? 0 : pick(1, 200);
  g.sinks = with_prefix ? 0 : (int[]){0, 1, 4, 70}[pick(0, 3)];
  const bool wraps = g.window > 0 && pick(0, 1);
  g.capacity = wraps ? g.sinks + g.window + g.tokens - 1 + pick(0, 30) : 700;
  g.prefix_rows = with_prefix ? pick(1, 300) : 0;
  std::vector<int32_t> lens(g.batch);
  bool expect_bad = false;
  for (int32_t &L : lens) {
    const int kind = pick(0, 9);
    L = kind == 0 ? 0 : kind == 1 ? g.tokens : pick(g.tokens, wraps ? 2000 : 700);
    if (pick(0, 60) == 0) {  // lengths a call cannot serve
      L = pick(0, 1) ? -pick(1, 5) : (wraps || g.window == 0 ? 100000 : 0);
      if (g.window == 0 && L > 0) expect_bad = true;
      if (L < 0) expect_bad = true;
    }
    if (L > 0 && L < g.tokens) expect_bad = true;
  }
  int32_t P = with_prefix ? pick(0, g.prefix_rows) : 0;
  int32_t P_device = P;
  if (with_prefix && pick(0, 30) == 0) {
    P_device = pick(0, 1) ? -3 : g.prefix_rows + 5;
    P = P_device < 0 ? 0 : g.prefix_rows;
    expect_bad = true;
  }
  g.seqlens = lens.data();
  g.prefix_len = with_prefix ? &P_device : nullptr;
  const int32_t per_block = 128 / g.group;
  g.qt_seq = std::min(g.tokens, per_block);
  g.nqb = (g.tokens + g.qt_seq - 1) / g.qt_seq;
  const int32_t pairs = g.batch * g.tokens;
  g.qt_pre = std::min(pairs, per_block);
  g.npb = (pairs + g.qt_pre - 1) / g.qt_pre;
  g.unit_cost = pick(0, 4);
  const int32_t workers = pick(0, 2) ? pick(1, 20) : 148;

  // Rows against their units' tiles.
  for (int32_t b = 0; b < g.batch; ++b)
    for (int32_t qb = 0; qb < g.nqb; ++qb) {
      bool bad = false;
      const UnitTiles u = own_unit(g, lens[b], qb, bad);
      const auto at = positions(u, g.capacity, k);
      if (bad) continue;  // rows are invalid; the slots were checked
      std::set<int32_t> seen;
      for (int32_t t = qb * g.qt_seq; t < std::min(g.tokens, (qb + 1) * g.qt_seq); ++t) {
        const RowRange r = own_row_range(g, lens[b], t);
        const int32_t p = lens[b] - g.tokens + t;
        for (int32_t j = std::max(0, std::min(p - g.window - 3, p - 3)); j <= p + 3; ++j) {
          const bool in = ((j >= r.lo && j < r.hi) || (j < r.pin && j < r.hi)) && j >= 0;
          if (in != sees_own(g, lens[b], t, j)) fail("own row range", k);
        }
        for (int32_t j = 0; j < r.hi; ++j)
          if (sees_own(g, lens[b], t, j)) seen.insert(j);
      }
      for (int32_t j : seen)
        if (!at.count(j)) fail("a visible position has no tile", k);
      for (const auto &e : at) {
        if (!seen.count(e.first)) fail("a tile holds a position nobody sees", k);
        if (e.second != (e.first < g.sinks ? e.first
                                           : g.sinks + (e.first - g.sinks) %
                                                           (g.capacity - g.sinks)))
          fail("wrong slot", k);
      }
    }

  // Chunks, segments, partials.
  std::map<std::pair<bool, int32_t>, std::vector<std::pair<int32_t, int32_t>>> pieces;
  std::map<std::pair<bool, int64_t>, std::pair<std::pair<bool, int32_t>, int32_t>> slots;
  std::map<std::pair<bool, int32_t>, RowSegment> unit_of;
  RowsPlan pl = {};
  std::vector<RowSegment> first_of(workers + 1);
  std::vector<bool> has_first(workers + 1, false);
  int64_t steps_done = 0;
  for (int32_t c = 0; c < workers; ++c) {
    pl = plan_of(g, c, workers);
    if (expect_bad && !pl.bad) fail("impossible lengths went unnoticed", k);
    if (pl.cs != steps_done) fail("chunks do not follow one another", k);
    const int32_t busy = std::min(workers, pl.total);
    if (pl.ce - pl.cs > pl.total / busy + 1 || (c < busy && pl.ce - pl.cs < pl.total / busy))
      fail("uneven chunks", k);
    for (int32_t f = pl.cs; f < pl.ce; ++f)
      if (chunk_of(pl.total, workers, f) != c) fail("chunk_of", k);
    steps_done = pl.ce;
    RowSegments it;
    it.init(pl);
    RowSegment s;
    int64_t last = -1;
    int segments = 0;
    while (it.next(g, s)) {
      if (s.t0 < 0 || s.t1 <= s.t0 || s.t1 > s.u.n) fail("segment range", k);
      const int64_t from = s.start + g.unit_cost + s.t0, to = s.start + g.unit_cost + s.t1;
      if (from < pl.cs || to > pl.ce || from <= last) fail("a segment outside its chunk", k);
      last = from;
      if (s.opens != (segments == 0)) fail("opens", k);
      int32_t words[kSegmentWords];
      pack_segment(s, words);
      RowSegment w = {};
      unpack_segment(g, words, w);
      if (w.x != s.x || w.b != s.b || w.qb != s.qb || w.unit != s.unit || w.L != s.L ||
          w.start != s.start || w.t0 != s.t0 || w.t1 != s.t1 || w.prefix != s.prefix ||
          w.opens != s.opens || w.u.n != s.u.n)
        fail("a packed segment", k);
      for (int32_t t = s.t0; t < s.t1; ++t) {
        const RowTile x = unit_tile(s.u, t), y = unit_tile(w.u, t);
        if (x.pos != y.pos || x.slot != y.slot || x.ntok != y.ntok) fail("a packed tile", k);
      }
      if (segments++ == 0) {
        first_of[c] = s;
        has_first[c] = true;
      }
      const std::pair<bool, int32_t> id(s.prefix, s.unit);
      pieces[id].emplace_back(s.t0, s.t1);
      if (unit_of.count(id) && unit_of[id].start != s.start) fail("a unit's start moves", k);
      unit_of[id] = s;
      if (with_prefix || !s.whole()) {
        const int32_t slot = partial_slot(with_prefix, c, s.unit, s.opens);
        const int64_t units = s.prefix ? static_cast<int64_t>(g.npb) * g.n_kv_heads
                                       : static_cast<int64_t>(g.batch) * g.nqb * g.n_kv_heads;
        if (slot < 0 || slot >= (with_prefix ? workers + units : 2 * workers))
          fail("slot outside the workspace", k);
        if (!slots.emplace(std::make_pair(s.prefix, slot), std::make_pair(id, s.t0)).second)
          fail("two partials in one slot", k);
      }
    }
  }
  if (steps_done != pl.total) fail("steps left out", k);
  // (no windows: the unit covers [lo, P) with lo from the batch's shortest sequence)
  const UnitTiles pu = prefix_unit(g, P, pl.least_own);
  if (with_prefix) {
    const auto tiles = positions(pu, g.prefix_rows, k);
    for (int32_t b = 0; b < g.batch; ++b)
      for (int32_t t = 0; t < g.tokens; ++t) {
        const RowRange r = prefix_row_range(g, lens[b], t, P);
        for (int32_t j = 0; j < P + 2; ++j) {
          const bool in = j >= r.lo && j < r.hi;
          if (in != sees_prefix(g, lens[b], t, P, j)) fail("prefix row range", k);
          if (in && !tiles.count(j)) fail("a visible prefix position has no tile", k);
        }
      }
    for (const auto &e : tiles)
      if (e.first != e.second || e.first >= P) fail("prefix tile", k);
  }
  const int64_t units = (pu.n > 0 ? static_cast<int64_t>(g.npb) * g.n_kv_heads : 0) +
                        static_cast<int64_t>(g.batch) * g.nqb * g.n_kv_heads;
  if (static_cast<int64_t>(pieces.size()) != units) fail("units left out", k);
  std::set<std::pair<bool, int32_t>> merged;
  auto expect_parts = [&](const std::pair<bool, int32_t> &id, const PartSlots &ps) {
    const auto &want = pieces[id];
    if (ps.n != static_cast<int32_t>(want.size())) fail("number of pieces", k);
    for (int32_t i = 0; i < ps.n; ++i) {
      const int64_t slot = i == 0 ? ps.first : ps.next + (i - 1) * ps.step;
      const auto f = slots.find(std::make_pair(id.first, slot));
      if (f == slots.end() || f->second.first != id || f->second.second != want[i].first)
        fail("the merge reads another piece", k);
    }
    merged.insert(id);
  };
  if (with_prefix) {
    for (const auto &e : pieces)
      expect_parts(e.first, unit_parts(pl.total, workers, unit_of[e.first].start + g.unit_cost,
                                       unit_of[e.first].u.n, e.first.second));
  } else {
    for (int32_t c = 0; c + 1 < workers; ++c) {
      if (!has_first[c + 1]) continue;
      const RowSegment &s = first_of[c + 1];
      PartSlots ps;
      if (cut_parts(pl.total, workers, c, s.start, g.unit_cost, s.u.n, ps)) {
        const std::pair<bool, int32_t> id(false, s.unit);
        if (merged.count(id)) fail("a unit is merged twice", k);
        expect_parts(id, ps);
      }
    }
    for (const auto &e : pieces)
      if ((e.second.size() > 1) != (merged.count(e.first) > 0)) fail("a cut unit is not merged", k);
  }
  for (const auto &e : pieces) {
    int32_t t = 0;
    for (const auto &pc : e.second) {
      if (pc.first != t) fail("a unit's pieces do not follow one another", k);
      t = pc.second;
    }
    if (t != unit_of[e.first].u.n) fail("a unit's tiles are not covered", k);
  }
}

}  // namespace

int main(int argc, char **argv) {
  const int cases = argc > 1 ? atoi(argv[1]) : 100;
  std::mt19937_64 rng(11);
  for (int k = 0; k < cases; ++k) check_case(rng, k);
  printf("ok %d\n", cases);
  return 0;
}
