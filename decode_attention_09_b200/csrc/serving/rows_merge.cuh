// Joins the partials that rows_attn.cuh leaves:
//   lse = log sum_i exp(lse_i),  out = sum_i exp(lse_i - lse) o_i.
// One warp per output row, a lane owning D / 32 of its dims; the parts' log-sum-exps
// are read first (one per lane and step), then the parts' rows, eight in flight.
// Where the parts are is worked out from the lengths before the wait on the kernel
// in front.  Bound by latency: a few L2 round trips.
#pragma once

#include <cstdint>

#include "../ptx.cuh"
#include "rows_attn.cuh"
#include "rows_chunks.cuh"

namespace gdattn {

// Parts of one row: row r of the slots `at` of a slot array with `rows` rows a slot.
struct RowParts {
  const float *o, *lse;
  PartSlots at;
  int32_t rows, r;
  __device__ __forceinline__ int64_t row(int32_t i) const {
    return (i == 0 ? at.first : at.next + (i - 1) * at.step) * rows + r;
  }
};

template <int D>
__device__ __forceinline__ void merge_row(const RowParts (&src)[2], uint16_t *out, float *lse) {
  constexpr int V = D / 128;  // float4 per lane
  const int lane = threadIdx.x & 31;
  const int32_t n0 = src[0].at.n, n = n0 + src[1].at.n;
  float m = -INFINITY;
  for (int32_t i = lane; i < n; i += 32) {
    const RowParts &s = i < n0 ? src[0] : src[1];
    m = fmaxf(m, __ldcg(s.lse + s.row(i < n0 ? i : i - n0)));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float4 acc[V];
#pragma unroll
  for (int c = 0; c < V; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  float z = 0.f;
  if (m != -INFINITY) {
    constexpr int kFlight = 8 / V;
    for (int32_t i0 = 0; i0 < n; i0 += kFlight) {
      float w[kFlight];
      float4 v[kFlight][V];
#pragma unroll
      for (int q = 0; q < kFlight; ++q) {
        const int32_t i = i0 + q;
        if (i < n) {
          const RowParts &s = i < n0 ? src[0] : src[1];
          const int64_t row = s.row(i < n0 ? i : i - n0);
          w[q] = __ldcg(s.lse + row);
#pragma unroll
          for (int c = 0; c < V; ++c)
            v[q][c] = __ldcg(reinterpret_cast<const float4 *>(s.o + row * D) + c * 32 + lane);
        } else {
          w[q] = -INFINITY;
        }
      }
#pragma unroll
      for (int q = 0; q < kFlight; ++q) {
        if (w[q] == -INFINITY) continue;  // an empty part adds nothing
        const float f = exp2f(w[q] - m);
        z += f;
#pragma unroll
        for (int c = 0; c < V; ++c) {
          acc[c].x = fmaf(f, v[q][c].x, acc[c].x);
          acc[c].y = fmaf(f, v[q][c].y, acc[c].y);
          acc[c].z = fmaf(f, v[q][c].z, acc[c].z);
          acc[c].w = fmaf(f, v[q][c].w, acc[c].w);
        }
      }
    }
  }
  const float inv = z > 0.f ? __fdividef(1.f, z) : 0.f;
#pragma unroll
  for (int c = 0; c < V; ++c) {
    uint2 pk;
    pk.x = pack_bf16x2(acc[c].x * inv, acc[c].y * inv);
    pk.y = pack_bf16x2(acc[c].z * inv, acc[c].w * inv);
    *reinterpret_cast<uint2 *>(out + (c * 32 + lane) * 4) = pk;
  }
  if (lane == 0 && lse != nullptr) *lse = z > 0.f ? (m + log2f(z)) * kLn2 : -INFINITY;
}

constexpr int kMergeThreads = 256;

// Sinks: units that a chunk boundary cuts.  CTA x looks at the boundary behind
// chunk x and joins the unit there if this is the unit's first boundary.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_cut_units_kernel(const RowsParams p) {
  const RowsGeom &g = p.g;
  const int32_t c = blockIdx.x;
  const RowsPlan pl = plan_rows(g, c + 1, p.workers);  // every warp: no exchange needed
  RowSegments segs;
  segs.init(g, pl);
  RowSegment seg;
  RowParts src[2] = {};
  const bool cut =
      segs.next(g, seg) && cut_parts(pl.chunk, c, pl.cs, seg.t0, seg.u.n, src[0].at);
  grid_launch_dependents();
  grid_dependency_wait();
  if (!cut) return;
  const int32_t nrow = imin32(g.qt_seq, g.tokens - seg.qb * g.qt_seq) * g.group;
  const int32_t r = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5);
  if (r >= nrow) return;
  src[0].o = p.own_o;
  src[0].lse = p.own_lse;
  src[0].rows = p.rs;
  src[0].r = r;
  const int32_t tq = r / g.group, h = r - tq * g.group;
  const int64_t row = (static_cast<int64_t>(seg.qb * g.qt_seq + tq) * g.batch + seg.b) *
                          (g.n_kv_heads * g.group) + seg.x * g.group + h;
  merge_row<D>(src, p.out + row * D, p.lse != nullptr ? p.lse + row : nullptr);
}

// Prefix: every output row has parts of its prefix unit and of its own unit.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_prefix_kernel(const RowsParams p) {
  const RowsGeom &g = p.g;
  const int lane = threadIdx.x & 31;
  const int32_t Hq = g.n_kv_heads * g.group;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kMergeThreads / 32) + (threadIdx.x >> 5);
  const bool real = row < static_cast<int64_t>(g.tokens) * g.batch * Hq;
  const int64_t safe = real ? row : 0;
  const int32_t a = static_cast<int32_t>(safe / Hq), hq = static_cast<int32_t>(safe % Hq);
  const int32_t x = hq / g.group, h = hq - x * g.group;
  const int32_t tok = a / g.batch, b = a - tok * g.batch;
  const RowsPlan pl = plan_rows(g, 0, p.workers);
  const UnitTiles pu = prefix_unit(g, pl.prefix_len, pl.least_own);
  RowParts src[2] = {};
  src[0].o = p.pre_o;
  src[0].lse = p.pre_lse;
  src[1].o = p.own_o;
  src[1].lse = p.own_lse;
  if (pu.n > 0) {
    const int32_t pb = a / g.qt_pre;
    const int32_t unit = x * g.npb + pb;
    src[0].at = unit_parts(pl.chunk, static_cast<int64_t>(unit) * pu.n, pu.n, unit);
    src[0].rows = p.rp;
    src[0].r = (a - pb * g.qt_pre) * g.group + h;
  }
  const int32_t qb = tok / g.qt_seq, y = b * g.nqb + qb;
  bool dummy = false;
  int64_t before = 0;
  for (int32_t yy = lane; yy < y; yy += 32) before += pair_tiles(g, yy, dummy);
  before = warp_sum64(before) * g.n_kv_heads;
  const int32_t n = pair_tiles(g, y, dummy);
  src[1].at = unit_parts(pl.chunk, pl.prefix_all + before + static_cast<int64_t>(x) * n, n,
                         y * g.n_kv_heads + x);
  src[1].rows = p.rs;
  src[1].r = (tok - qb * g.qt_seq) * g.group + h;
  grid_launch_dependents();
  grid_dependency_wait();
  if (real) merge_row<D>(src, p.out + row * D, p.lse != nullptr ? p.lse + row : nullptr);
}

}  // namespace gdattn
