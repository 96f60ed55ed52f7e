// Host check of the row planner's arithmetic (csrc/serving/rows_plan.cuh) at the ends of
// 32 bits: windows up to 2^31 - 1, lengths from -2^31 to 2^31 - 1, sequences shorter than
// the step.  Compiled with traps on signed overflow.  Prints "ok", or the first failure.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#define GDATTN_HD inline
#include "rows_plan.cuh"

using namespace gdattn;

static void fail(const char *what, const RowsGeom &g, int32_t L, int32_t qb) {
  fprintf(stderr, "%s: T %d, window %d, sinks %d, C %d, L %d, block %d\n", what, g.tokens,
          g.window, g.sinks, g.capacity, L, qb);
  exit(1);
}

static void check(const RowsGeom &g, int32_t L, int32_t qb) {
  bool bad = false;
  const UnitTiles u = own_unit(g, L, qb, bad);
  if ((L < 0 || (L > 0 && L < g.tokens)) && !bad) fail("a bad length went unnoticed", g, L, qb);
  // What the block's tokens see, by the definition, in 64 bits.
  const int64_t first = static_cast<int64_t>(L) - g.tokens + static_cast<int64_t>(qb) * g.qt_seq;
  const int64_t toks = g.tokens - qb * g.qt_seq < g.qt_seq ? g.tokens - qb * g.qt_seq : g.qt_seq;
  const int64_t hi = first + toks;
  int64_t want = 0;  // rows
  if (L > 0 && hi > 0) {
    int64_t lo = g.window > 0 && first + 1 > g.window ? first + 1 - g.window : 0;
    const int64_t oldest = static_cast<int64_t>(L) - (g.capacity - g.sinks);
    if ((lo > g.sinks ? lo : g.sinks) < oldest) lo = oldest < hi ? oldest : hi;  // (reported)
    want = hi - lo + (g.sinks < lo ? g.sinks : lo);
  }
  int64_t got = 0;
  if (u.n < 1) fail("a unit without a tile", g, L, qb);
  // All tiles, or those at both ends of a long unit.
  for (int32_t t = 0; t < u.n; t = t == 999 && u.n > 2000 ? u.n - 1000 : t + 1) {
    const RowTile r = unit_tile(u, t);
    if (r.ntok < 0 || r.ntok > kRowTile) fail("rows of a tile", g, L, qb);
    if (r.ntok > 0 && (r.pos < 0 || r.pos + (r.ntok - 1) >= hi || r.slot < 0 ||
                       r.slot > g.capacity - r.ntok ||
                       r.slot != slot_of(r.pos, g.sinks, g.capacity)))
      fail("a tile's place", g, L, qb);
    got += r.ntok;
  }
  if (u.n <= 2000 && got != want) fail("rows of a unit", g, L, qb);
  for (int32_t t = qb * g.qt_seq; t < qb * g.qt_seq + toks; ++t) {
    const RowRange r = own_row_range(g, L, t), q = prefix_row_range(g, L, t, 1000);
    const int64_t p = static_cast<int64_t>(L) - g.tokens + t;
    const bool there = L > 0 && p >= 0;
    const int64_t lo = g.window > 0 && p + 1 > g.window ? p + 1 - g.window : 0;
    if (there ? r.lo != lo || r.hi != p + 1 : r.hi != 0) fail("a row's range", g, L, qb);
    if (!there && q.hi != 0) fail("a row's prefix range", g, L, qb);
  }
}

int main() {
  const int32_t top = INT32_MAX;
  for (int32_t window : {0, 1, 64, 1000, 1 << 30, top - 300, top - 2, top - 1, top})
    for (int32_t tokens : {1, 2, 4, 9, 65, 300})
      for (int32_t sinks : {0, 4, 70})
        for (int32_t capacity : {71, 500, 1 << 20, 1 << 30})
          for (int32_t qt : {1, 64}) {
            RowsGeom g = {};
            g.batch = 1;
            g.tokens = tokens;
            g.n_kv_heads = g.group = 1;
            g.window = window;
            g.sinks = sinks;
            g.capacity = capacity;
            g.qt_seq = qt < tokens ? qt : tokens;
            g.nqb = (tokens + g.qt_seq - 1) / g.qt_seq;
            for (int32_t qb = 0; qb < g.nqb; ++qb) {
              for (int32_t L = -3; L <= tokens + 3; ++L) check(g, L, qb);
              for (int32_t L : {INT32_MIN, INT32_MIN + 1, -(1 << 30), capacity, capacity + 1,
                                1 << 30, top - 300, top - 1, top})
                check(g, L, qb);
            }
          }
  printf("ok\n");
  return 0;
}
