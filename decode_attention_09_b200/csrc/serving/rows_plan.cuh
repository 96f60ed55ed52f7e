// Which cache rows the query rows of a call attend, and in which tiles a block
// of query rows walks them: the arithmetic that the kernels of gdattn_decode_sink
// and gdattn_decode_prefix share.  Plain integer code, compiled for the CPU too
// (tests/rows_plan_host.cpp).
//
// A sequence's cache holds S pinned rows and a ring: position j lives in slot j
// below S and in slot S + (j - S) mod (C - S) from there on (S = 0: a plain
// ring).  Token t of T of sequence b sits at position p = L_b - T + t of its own
// tokens and attends [max(0, p + 1 - w), p + 1) and the pinned positions below
// that; of a shared prefix of P rows in front of them it attends
// [max(0, P + p + 1 - w), P)  (w = 0: everything).
#pragma once

#include <cstdint>

#ifndef GDATTN_HD
#define GDATTN_HD __host__ __device__ __forceinline__
#endif

namespace gdattn {

struct RowsGeom {
  const int32_t *seqlens;     // [batch], device
  const int32_t *prefix_len;  // device scalar, or null: no prefix
  int32_t batch;
  int32_t tokens;             // T
  int32_t n_kv_heads;
  int32_t group;              // query heads per KV head, G
  int32_t window;             // w, 0: none
  int32_t sinks;              // S
  int32_t capacity;           // C
  int32_t prefix_rows;        // rows of the prefix tensors
  int32_t qt_seq, nqb;        // tokens per block of a sequence, blocks per sequence
  int32_t qt_pre, npb;        // (token, sequence) pairs per prefix block, blocks
  int32_t unit_cost;          // what a unit costs besides its tiles, in tiles
};

GDATTN_HD int32_t imin32(int32_t a, int32_t b) { return a < b ? a : b; }
GDATTN_HD int32_t imax32(int32_t a, int32_t b) { return a > b ? a : b; }

// The prefix length the call uses; `bad` when the device scalar is out of range.
GDATTN_HD int32_t clamp_prefix(const RowsGeom &g, int32_t p, bool &bad) {
  if (p < 0 || p > g.prefix_rows) bad = true;
  return imax32(0, imin32(p, g.prefix_rows));
}

// Positions a query row sees: [lo, hi) and those below min(pin, hi).
struct RowRange {
  int32_t lo, hi, pin;
};

GDATTN_HD RowRange own_row_range(const RowsGeom &g, int32_t L, int32_t t) {
  RowRange r = {0, 0, 0};
  if (L <= 0) return r;  // a padding entry
  const int32_t p = L - g.tokens + t;
  if (p < 0) return r;  // a token in front of the sequence
  r.hi = p + 1;
  r.lo = g.window > 0 ? imax32(0, p + 1 - g.window) : 0;
  r.pin = g.sinks;
  return r;
}

GDATTN_HD RowRange prefix_row_range(const RowsGeom &g, int32_t L, int32_t t, int32_t P) {
  RowRange r = {0, 0, 0};
  if (L <= 0) return r;
  const int32_t p = L - g.tokens + t;
  if (p < 0) return r;
  r.hi = P;
  const int64_t lo = g.window > 0 ? static_cast<int64_t>(P) + p + 1 - g.window : 0;
  r.lo = lo <= 0 ? 0 : (lo < P ? static_cast<int32_t>(lo) : P);
  return r;
}

GDATTN_HD int32_t slot_of(int32_t pos, int32_t sinks, int32_t capacity) {
  return pos < sinks ? pos : sinks + (pos - sinks) % (capacity - sinks);
}

// A sequence length the call cannot serve: negative, shorter than the step, or
// (checked where the range is known) reaching behind the ring.
GDATTN_HD bool bad_length(const RowsGeom &g, int32_t L) { return L < 0 || (L > 0 && L < g.tokens); }

// First position of the ring still in the cache of a sequence of length L.
GDATTN_HD int32_t oldest_in_ring(const RowsGeom &g, int32_t L) {
  return L - (g.capacity - g.sinks);
}

// ------------------------------------------------------------------- tiles
// A unit is what one block of query rows of one KV head attends: a block of
// consecutive tokens of one sequence over that sequence's cache ("own"), or a
// block of (token, sequence) pairs of the batch over the prefix.  Its positions
// are walked in tiles of at most kRowTile rows that sit in consecutive slots:
// first the pinned positions in front of the main range, then the main range,
// cut where the ring wraps.
constexpr int32_t kRowTile = 64;

struct UnitTiles {
  int32_t pin;         // [0, pin): pinned positions below the main range
  int32_t lo;          // the main range's first position, in slot0
  int32_t slot0;
  int32_t run0, run1;  // its positions before the ring's wrap and behind it
  int32_t slot1;       // slot of the first position behind the wrap
  int32_t npin, n0, n; // tiles of pin, tiles of run0, all tiles
};

struct RowTile {
  int32_t pos, slot, ntok;
};

GDATTN_HD int32_t tiles_of(int32_t rows) { return (rows + kRowTile - 1) / kRowTile; }

GDATTN_HD RowTile unit_tile(const UnitTiles &u, int32_t t) {
  RowTile r;
  if (t < u.npin) {
    r.pos = r.slot = t * kRowTile;
    r.ntok = imin32(kRowTile, u.pin - r.pos);
  } else if (t < u.npin + u.n0) {
    const int32_t off = (t - u.npin) * kRowTile;
    r.pos = u.lo + off;
    r.slot = u.slot0 + off;
    r.ntok = imin32(kRowTile, u.run0 - off);
  } else {
    const int32_t off = (t - u.npin - u.n0) * kRowTile;
    r.pos = u.lo + u.run0 + off;
    r.slot = u.slot1 + off;
    r.ntok = imin32(kRowTile, u.run1 - off);
  }
  return r;
}

// Tiles of block qb of a sequence of length L.  A block without any position
// still has one tile, of no rows, so that its output rows are written.
GDATTN_HD UnitTiles own_unit(const RowsGeom &g, int32_t L, int32_t qb, bool &bad) {
  UnitTiles u = {0, 0, 0, 0, 0, g.sinks, 0, 0, 1};
  if (bad_length(g, L)) bad = true;
  if (L <= 0) return u;
  const int32_t first = L - g.tokens + qb * g.qt_seq;
  const int32_t hi = first + imin32(g.qt_seq, g.tokens - qb * g.qt_seq);
  if (hi <= 0) return u;
  // (compared first: with a window near 2^31 and a sequence shorter than the step the
  // difference leaves 32 bits)
  int32_t lo = g.window > 0 && first + 1 > g.window ? first + 1 - g.window : 0;
  const int32_t oldest = oldest_in_ring(g, L);
  if (imax32(lo, g.sinks) < oldest) {  // positions that later ones overwrote
    bad = true;
    lo = imin32(oldest, hi);
  }
  u.pin = imin32(g.sinks, lo);
  u.lo = lo;
  u.slot0 = slot_of(lo, g.sinks, g.capacity);
  u.run0 = imin32(hi - lo, g.capacity - u.slot0);
  u.run1 = hi - lo - u.run0;
  u.npin = tiles_of(u.pin);
  u.n0 = tiles_of(u.run0);
  u.n = imax32(1, u.npin + u.n0 + tiles_of(u.run1));
  return u;
}

// Tiles of every prefix block: the positions that some sequence's tokens reach,
// least_own being the fewest own positions in front of a query token.
GDATTN_HD UnitTiles prefix_unit(const RowsGeom &g, int32_t P, int32_t least_own) {
  UnitTiles u = {0, 0, 0, 0, 0, 0, 0, 0, 0};
  const int64_t lo = g.window > 0 ? static_cast<int64_t>(P) + least_own + 1 - g.window : 0;
  u.lo = u.slot0 = lo <= 0 ? 0 : (lo < P ? static_cast<int32_t>(lo) : P);
  u.run0 = P - u.lo;
  u.n0 = u.n = tiles_of(u.run0);
  return u;
}

}  // namespace gdattn
