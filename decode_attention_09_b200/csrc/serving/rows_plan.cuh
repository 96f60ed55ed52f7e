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
  const int32_t p = L - g.tokens + t;
  if (L <= 0 || p < 0) return r;  // a padding entry, or a token in front of the sequence
  r.hi = p + 1;
  r.lo = g.window > 0 ? imax32(0, p + 1 - g.window) : 0;
  r.pin = g.sinks;
  return r;
}

GDATTN_HD RowRange prefix_row_range(const RowsGeom &g, int32_t L, int32_t t, int32_t P) {
  RowRange r = {0, 0, 0};
  const int32_t p = L - g.tokens + t;
  if (L <= 0 || p < 0) return r;
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

}  // namespace gdattn
