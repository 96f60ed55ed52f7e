// Joins the partials that rows_attn.cuh leaves:
//   lse = log sum_i exp(lse_i),  out = sum_i exp(lse_i - lse) o_i.
// One to eight warps share an output row (more where there are few rows, whose parts
// would otherwise be read one after the other: 64 rows of 65 parts at head_dim 512 took
// 36 us with one warp a row), a lane owning D / 32 of its dims, sixteen 16-byte loads
// in flight.  The row kernel says where the parts are.  Bound by latency: a few L2 round
// trips.
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
    return static_cast<int64_t>(i == 0 ? at.first : at.next + (i - 1) * at.step) * rows + r;
  }
};

constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;

// What a warp knows of a row after its share of the parts.
template <int D>
struct RowSum {
  float4 acc[D / 128];
  float m, z;
};

template <int D>
__device__ __forceinline__ void add_part(RowSum<D> &s, float lse, const float4 (&v)[D / 128]) {
  if (lse == -INFINITY) return;  // an empty part adds nothing, whatever its row holds
  const float m = fmaxf(s.m, lse);
  const float a = exp2f(s.m - m), f = exp2f(lse - m);
  s.m = m;
  s.z = fmaf(s.z, a, f);
#pragma unroll
  for (int c = 0; c < D / 128; ++c) {
    s.acc[c].x = fmaf(f, v[c].x, s.acc[c].x * a);
    s.acc[c].y = fmaf(f, v[c].y, s.acc[c].y * a);
    s.acc[c].z = fmaf(f, v[c].z, s.acc[c].z * a);
    s.acc[c].w = fmaf(f, v[c].w, s.acc[c].w * a);
  }
}

// Parts share, share + shares, ... of a row.
template <int D>
__device__ __forceinline__ RowSum<D> sum_parts(const RowParts (&src)[2], int share, int shares) {
  constexpr int V = D / 128;       // float4 per lane
  constexpr int kFlight = 16 / V;  // parts in flight
  const int lane = threadIdx.x & 31;
  const int32_t n0 = src[0].at.n, n = n0 + src[1].at.n;
  RowSum<D> s;
  s.m = -INFINITY;
  s.z = 0.f;
#pragma unroll
  for (int c = 0; c < V; ++c) s.acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int32_t i0 = share; i0 < n; i0 += kFlight * shares) {
    float lse[kFlight];
    float4 v[kFlight][V];
#pragma unroll
    for (int q = 0; q < kFlight; ++q) {
      const int32_t i = i0 + q * shares;
      lse[q] = -INFINITY;
      if (i < n) {
        const RowParts &from = i < n0 ? src[0] : src[1];
        const int64_t row = from.row(i < n0 ? i : i - n0);
        lse[q] = __ldcg(from.lse + row);
#pragma unroll
        for (int c = 0; c < V; ++c)
          v[q][c] = __ldcg(reinterpret_cast<const float4 *>(from.o + row * D) + c * 32 + lane);
      }
    }
#pragma unroll
    for (int q = 0; q < kFlight; ++q) add_part<D>(s, lse[q], v[q]);
  }
  return s;
}

// The row's output, by the warps of a CTA that share it (1, 2, 4 or 8 of them, next to
// one another; every warp of the CTA calls this).
template <int D>
__device__ __forceinline__ void merge_row(const RowParts (&src)[2], bool real, int shares,
                                          uint16_t *out, float *lse) {
  constexpr int V = D / 128;
  __shared__ float4 sh_acc[kMergeWarps][D / 4];
  __shared__ float sh_m[kMergeWarps], sh_z[kMergeWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int share = warp % shares;
  RowSum<D> s = {};
  if (real) s = sum_parts<D>(src, share, shares);
  if (shares > 1) {  // of the whole CTA
    if (share > 0) {
#pragma unroll
      for (int c = 0; c < V; ++c) sh_acc[warp][c * 32 + lane] = s.acc[c];
      if (lane == 0) {
        sh_m[warp] = s.m;
        sh_z[warp] = s.z;
      }
    }
    __syncthreads();
    if (share > 0) return;
    for (int w = warp + 1; w < warp + shares; ++w) {
      // (a share of one part or more: its rows, weighted by its sum)
      const float mw = sh_m[w], zw = sh_z[w];
      if (!real || zw == 0.f) continue;
      const float m = fmaxf(s.m, mw);
      const float a = exp2f(s.m - m), f = exp2f(mw - m);
      s.m = m;
      s.z = s.z * a + zw * f;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float4 v = sh_acc[w][c * 32 + lane];
        s.acc[c].x = fmaf(f, v.x, s.acc[c].x * a);
        s.acc[c].y = fmaf(f, v.y, s.acc[c].y * a);
        s.acc[c].z = fmaf(f, v.z, s.acc[c].z * a);
        s.acc[c].w = fmaf(f, v.w, s.acc[c].w * a);
      }
    }
  }
  if (!real) return;
  const float inv = s.z > 0.f ? __fdividef(1.f, s.z) : 0.f;
#pragma unroll
  for (int c = 0; c < V; ++c) {
    uint2 pk;
    pk.x = pack_bf16x2(s.acc[c].x * inv, s.acc[c].y * inv);
    pk.y = pack_bf16x2(s.acc[c].z * inv, s.acc[c].w * inv);
    *reinterpret_cast<uint2 *>(out + (c * 32 + lane) * 4) = pk;
  }
  if (lane == 0 && lse != nullptr) *lse = s.z > 0.f ? (s.m + log2f(s.z)) * kLn2 : -INFINITY;
}

// Sinks: units that a chunk boundary cuts.  CTA x joins the unit whose first boundary
// is the one behind chunk x, if there is one.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_cut_units_kernel(const RowsParams p) {
  const RowsGeom &g = p.g;
  grid_launch_dependents();
  grid_dependency_wait();
  const CutEntry cut = p.cuts[blockIdx.x];
  if (cut.parts.n == 0) return;
  const int32_t nrow = imin32(g.qt_seq, g.tokens - cut.qb * g.qt_seq) * g.group;
  const int32_t r = blockIdx.y * (kMergeWarps / p.merge_shares) + (threadIdx.x >> 5) / p.merge_shares;
  RowParts src[2] = {};
  src[0].at = cut.parts;
  src[0].o = p.own_o;
  src[0].lse = p.own_lse;
  src[0].rows = p.rs;
  src[0].r = r;
  const int32_t tq = r / g.group, h = r - tq * g.group;
  const int64_t row = (static_cast<int64_t>(cut.qb * g.qt_seq + tq) * g.batch + cut.b) *
                          (g.n_kv_heads * g.group) + cut.x * g.group + h;
  merge_row<D>(src, r < nrow, p.merge_shares, p.out + row * D,
               p.lse != nullptr ? p.lse + row : nullptr);
}

// Prefix: every output row has parts of its prefix unit and of its own unit.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_prefix_kernel(const RowsParams p) {
  const RowsGeom &g = p.g;
  const int32_t Hq = g.n_kv_heads * g.group;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kMergeWarps / p.merge_shares) +
                      (threadIdx.x >> 5) / p.merge_shares;
  const bool real = row < static_cast<int64_t>(g.tokens) * g.batch * Hq;
  const int64_t safe = real ? row : 0;
  const int32_t a = static_cast<int32_t>(safe / Hq), hq = static_cast<int32_t>(safe % Hq);
  const int32_t x = hq / g.group, h = hq - x * g.group;
  const int32_t tok = a / g.batch, b = a - tok * g.batch;
  const int32_t pb = a / g.qt_pre, qb = tok / g.qt_seq, y = b * g.nqb + qb;
  RowParts src[2] = {};
  src[0].o = p.pre_o;
  src[0].lse = p.pre_lse;
  src[0].rows = p.rp;
  src[0].r = (a - pb * g.qt_pre) * g.group + h;
  src[1].o = p.own_o;
  src[1].lse = p.own_lse;
  src[1].rows = p.rs;
  src[1].r = (tok - qb * g.qt_seq) * g.group + h;
  grid_launch_dependents();
  grid_dependency_wait();
  const PrefixEntry entry = *p.prefix_entry;
  const int32_t start = p.pair_start[y];
  const int32_t steps = (p.pair_start[y + 1] - start) / g.n_kv_heads;
  if (entry.prefix_tiles > 0) {
    const int32_t unit = x * g.npb + pb;
    src[0].at = unit_parts(entry.steps, p.workers,
                           unit * entry.prefix_steps + g.unit_cost,
                           entry.prefix_tiles, unit);
  }
  src[1].at = unit_parts(entry.steps, p.workers,
                         start + x * steps + g.unit_cost, steps - g.unit_cost, y * g.n_kv_heads + x);
  merge_row<D>(src, real, p.merge_shares, p.out + row * D,
               p.lse != nullptr ? p.lse + row : nullptr);
}

}  // namespace gdattn
