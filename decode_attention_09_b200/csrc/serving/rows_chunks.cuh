// Split of a call's work over the CTAs (or CTA pairs) of the grid.
//
// A unit takes unit_cost steps (starting a block, writing its rows) and then one step
// per tile.  All units' steps are laid end to end: first the prefix units, unit
// u = x * npb + pb (KV head x, prefix block pb), then the own units, unit
// y * Hkv + x for pair y = b * nqb + qb (sequence b, its block qb).  The whole is
// cut into equal chunks, one per worker (a CTA or a CTA pair), whatever the mix
// of lengths: the lengths are read on the device, so a captured graph follows
// them and the host never waits.  The tiles of a unit in a chunk are a segment.
#pragma once

#include <cstdint>

#include "../ptx.cuh"
#include "rows_plan.cuh"

namespace gdattn {

// Chunk c of n steps cut for `workers`: [chunk_begin(c), chunk_begin(c + 1)), sizes that
// differ by at most one (equal ones rounded up leave the last workers without any:
// 1216 steps over 148 workers used 136 of them).
// With fewer steps than workers the first workers get one each, so that the pieces of
// a unit sit in consecutive chunks.
// (All steps of a call fit 32 bits: the host refuses others.)
GDATTN_HD int32_t chunk_begin(int32_t steps, int32_t workers, int32_t c) {
  const int32_t n = imin32(steps, workers);
  return c < n ? static_cast<int32_t>(static_cast<int64_t>(c) * steps / n) : steps;
}
GDATTN_HD int32_t chunk_of(int32_t steps, int32_t workers, int32_t step) {
  const int32_t n = imin32(steps, workers);
  return static_cast<int32_t>(((static_cast<int64_t>(step) + 1) * n - 1) / steps);
}

struct RowsPlan {
  int32_t total;      // steps
  int32_t cs, ce;     // this worker's steps
  int32_t prefix_all; // steps of all prefix units
  int32_t y_start;    // first step of pair y
  int32_t y;          // the own pair that step max(cs, prefix_all) is in
  int32_t prefix_len; // P
  int32_t least_own;
  int32_t bad;
  UnitTiles pu;       // of every prefix unit
};

__device__ __forceinline__ int32_t warp_sum32(int32_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Steps of a unit of pair y.
__device__ __forceinline__ int32_t pair_steps(const RowsGeom &g, int32_t y, bool &bad) {
  const int32_t b = y / g.nqb;
  return own_unit(g, __ldg(g.seqlens + b), y - b * g.nqb, bad).n + g.unit_cost;
}

// And of a prefix unit (none when there is nothing to read).
GDATTN_HD int32_t prefix_steps(const RowsGeom &g, const UnitTiles &pu) {
  return pu.n > 0 ? pu.n + g.unit_cost : 0;
}

// The plan of worker c of `workers`; run by one whole warp, every lane gets it.
__device__ __forceinline__ RowsPlan plan_rows(const RowsGeom &g, int32_t c, int32_t workers) {
  const int lane = threadIdx.x & 31;
  const int32_t pairs = g.batch * g.nqb;
  RowsPlan p;
  bool bad = false;
  int32_t own = 0;
  for (int32_t y = lane; y < pairs; y += 32) own += pair_steps(g, y, bad);
  own = warp_sum32(own) * g.n_kv_heads;
  p.prefix_len = 0;
  p.least_own = 0;
  if (g.prefix_len != nullptr) {
    p.prefix_len = clamp_prefix(g, __ldg(g.prefix_len), bad);
    int32_t least = INT32_MAX;
    if (g.window > 0) {
      for (int32_t b = lane; b < g.batch; b += 32) {
        const int32_t L = __ldg(g.seqlens + b);
        if (L > 0) least = imin32(least, imax32(0, L - g.tokens));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        least = imin32(least, __shfl_xor_sync(0xffffffffu, least, o));
    }
    p.least_own = least == INT32_MAX ? 0 : least;
  }
  p.pu = prefix_unit(g, p.prefix_len, p.least_own);  // without a prefix: no tiles
  p.prefix_all = prefix_steps(g, p.pu) * g.n_kv_heads * g.npb;
  p.bad = __any_sync(0xffffffffu, bad);
  p.total = p.prefix_all + own;
  p.cs = chunk_begin(p.total, workers, c);
  p.ce = chunk_begin(p.total, workers, c + 1);
  // The own pair whose steps reach past the chunk's start.
  p.y = 0;
  p.y_start = p.prefix_all;
  if (p.cs > p.prefix_all) {
    int32_t base = p.prefix_all;
    p.y = pairs;
    for (int32_t y0 = 0; y0 < pairs; y0 += 32) {
      const int32_t y = y0 + lane;
      bool dummy = false;
      const int32_t span = y < pairs ? pair_steps(g, y, dummy) * g.n_kv_heads : 0;
      int32_t incl = span;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      incl += base;
      const unsigned hit = __ballot_sync(0xffffffffu, y < pairs && incl > p.cs);
      if (hit) {
        const int first = __ffs(hit) - 1;
        p.y = y0 + first;
        p.y_start = __shfl_sync(0xffffffffu, incl - span, first);
        break;
      }
      base = __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  return p;
}

// One (chunk, unit) piece of work: tiles [t0, t1) of the unit, at least one.
struct RowSegment {
  UnitTiles u;
  int32_t t0, t1;
  int32_t x;       // KV head
  int32_t b, qb;   // own: sequence and block; prefix: qb is the prefix block
  int32_t unit;    // index among the prefix units, or among the own units
  int32_t L;       // own: the sequence's length
  int32_t start;   // the unit's first step
  bool prefix;
  bool opens;      // first segment of its chunk
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == u.n; }
};

// Walks the segments of a chunk in order; every warp that needs them runs its own.
struct RowSegments {
  const RowsPlan *plan;  // in shared memory, in the row kernel
  int32_t pos, y_start, y;

  __device__ __forceinline__ void init(const RowsPlan &p) {
    plan = &p;
    pos = p.cs;
    y_start = p.y_start;
    y = p.y;
  }

  __device__ __forceinline__ bool next(const RowsGeom &g, RowSegment &s) {
    const int32_t pairs = g.batch * g.nqb, ce = plan->ce;
    while (pos < ce) {
      if (pos < plan->prefix_all) {
        const int32_t steps = prefix_steps(g, plan->pu);
        s.prefix = true;
        s.u = plan->pu;
        s.unit = pos / steps;
        s.x = s.unit / g.npb;
        s.qb = s.unit - s.x * g.npb;
        s.b = 0;
        s.L = 0;
        s.start = s.unit * steps;
      } else {
        for (; y < pairs; ++y) {
          bool dummy = false;
          s.b = y / g.nqb;
          s.qb = y - s.b * g.nqb;
          s.L = __ldg(g.seqlens + s.b);
          s.u = own_unit(g, s.L, s.qb, dummy);
          const int32_t span = (s.u.n + g.unit_cost) * g.n_kv_heads;
          if (y_start + span > pos) break;
          y_start += span;
        }
        if (y >= pairs) return false;
        s.prefix = false;
        s.x = (pos - y_start) / (s.u.n + g.unit_cost);
        s.unit = y * g.n_kv_heads + s.x;
        s.start = y_start + s.x * (s.u.n + g.unit_cost);
      }
      const int32_t first = s.start + g.unit_cost;  // its first tile's step
      s.opens = s.start <= plan->cs;
      s.t0 = imax32(0, pos - first);
      s.t1 = imin32(ce - first, s.u.n);  // (negative: none)
      pos = imin32(first + s.u.n, ce);
      if (s.t1 > s.t0) return true;  // (else the chunk ends in front of the first tile)
    }
    return false;
  }
};

// A segment as it passes between the warps of the row kernel, which find it once:
// eight warps that each walked the units spent 5000 cycles a segment on it.
constexpr int kSegmentWords = 11;

GDATTN_HD void pack_segment(const RowSegment &s, int32_t *w) {
  w[0] = s.x | (s.prefix ? 1 << 30 : 0) | (s.opens ? 1 << 29 : 0);  // (x is below 2^23)
  w[1] = s.u.lo;
  w[2] = s.u.slot0;
  w[3] = s.u.run0;
  w[4] = s.u.run1;
  w[5] = s.t0;
  w[6] = s.t1;
  w[7] = s.b;
  w[8] = s.qb;
  w[9] = s.L;
  w[10] = s.start;
}

GDATTN_HD void unpack_segment(const RowsGeom &g, const int32_t *w, RowSegment &s) {
  s.x = w[0] & ((1 << 29) - 1);
  s.prefix = (w[0] >> 30 & 1) != 0;
  s.opens = (w[0] >> 29 & 1) != 0;
  s.u.lo = w[1];
  s.u.slot0 = w[2];
  s.u.run0 = w[3];
  s.u.run1 = w[4];
  s.t0 = w[5];
  s.t1 = w[6];
  s.b = w[7];
  s.qb = w[8];
  s.L = w[9];
  s.start = w[10];
  s.u.pin = s.prefix ? 0 : imin32(g.sinks, s.u.lo);
  s.u.slot1 = s.prefix ? 0 : g.sinks;
  s.u.npin = tiles_of(s.u.pin);
  s.u.n0 = tiles_of(s.u.run0);
  s.u.n = s.prefix ? s.u.n0 : imax32(1, s.u.npin + s.u.n0 + tiles_of(s.u.run1));
  s.unit = s.prefix ? s.x * g.npb + s.qb : (s.b * g.nqb + s.qb) * g.n_kv_heads + s.x;
}

// ---------------------------------------------------------------- partials
// Slot of a segment's partial.  With a prefix every segment leaves one: chunk c
// touching unit u of its kind writes slot c + u (if a later chunk touches unit u',
// then u' >= u, so no two pieces share a slot).  Without one only pieces of split
// units do, at most two a chunk: its first segment and its last.
GDATTN_HD int32_t partial_slot(bool prefix_call, int32_t c, int32_t unit, bool opens) {
  return prefix_call ? c + unit : 2 * c + (opens ? 0 : 1);
}

// The slots of a unit's pieces: the first one's, then next, next + step, ...
struct PartSlots {
  int32_t first, next, step, n;
};

// Call with a prefix: a unit of its kind whose n > 0 tiles start at step `first`.
GDATTN_HD PartSlots unit_parts(int32_t steps, int32_t workers, int32_t first, int32_t n,
                               int32_t unit) {
  const int32_t cf = chunk_of(steps, workers, first);
  PartSlots s;
  s.n = chunk_of(steps, workers, first + n - 1) - cf + 1;
  s.step = 1;
  s.first = partial_slot(true, cf, unit, false);
  s.next = s.first + 1;
  return s;
}

// Call without a prefix: whether the boundary behind chunk c is the first one among
// the tiles of the unit that starts at step `start` and has n tiles, and its pieces.
GDATTN_HD bool cut_parts(int32_t steps, int32_t workers, int32_t c, int32_t start,
                         int32_t unit_cost, int32_t n, PartSlots &s) {
  const int32_t first = start + unit_cost, here = chunk_begin(steps, workers, c + 1);
  if (first >= here || here >= first + n) return false;        // not among its tiles
  const int32_t begin = chunk_begin(steps, workers, c);
  if (first < begin) return false;                             // cut by an earlier boundary
  s.n = chunk_of(steps, workers, first + n - 1) - c + 1;
  s.first = partial_slot(false, c, 0, start <= begin);
  s.next = partial_slot(false, c + 1, 0, true);
  s.step = 2;
  return true;
}

// What the row kernel leaves for the merge, so that the merge plans nothing again (its
// many CTAs doing so took 40 us behind an 8192-token prompt).
// Without a prefix: entry c, written by worker c + 1, says whether the boundary behind
// chunk c is a unit's first one (parts.n > 0), which unit and where its pieces are.
struct CutEntry {
  PartSlots parts;
  int32_t b, qb, x, pad;
};
// With a prefix, written by worker 0: all steps, a prefix unit's steps and tiles and the
// first steps of the own pairs.
struct PrefixEntry {
  int32_t steps, prefix_steps, prefix_tiles;
};

// Run by one whole warp, for worker 0 of a call with a prefix.
__device__ __forceinline__ void write_pair_starts(const RowsGeom &g, const RowsPlan &p,
                                                  PrefixEntry *entry, int32_t *pair_start) {
  const int lane = threadIdx.x & 31;
  const int32_t pairs = g.batch * g.nqb;
  if (lane == 0) {
    entry->steps = p.total;
    entry->prefix_steps = prefix_steps(g, p.pu);
    entry->prefix_tiles = p.pu.n;
  }
  int32_t base = p.prefix_all;
  for (int32_t y0 = 0; y0 < pairs; y0 += 32) {
    const int32_t y = y0 + lane;
    bool dummy = false;
    const int32_t span = y < pairs ? pair_steps(g, y, dummy) * g.n_kv_heads : 0;
    int32_t incl = span;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (y < pairs) pair_start[y] = base + incl - span;
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) pair_start[pairs] = base;
}

}  // namespace gdattn
