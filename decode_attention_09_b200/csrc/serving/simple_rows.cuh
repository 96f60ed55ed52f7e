// Attention of one query row per CTA, on the CUDA cores: the definition written
// down, for every geometry.
#pragma once

#include <cstdint>

#include "../ptx.cuh"
#include "rows_plan.cuh"

namespace gdattn {

struct SimpleRowsParams {
  RowsGeom g;
  const uint16_t *q, *k, *v, *pk, *pv;
  int64_t batch_stride;
  uint16_t *out;
  float *lse;
  uint32_t *status;
  float qscale, post;
};

constexpr int kSimpleWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kSimpleWarps) simple_rows_kernel(const SimpleRowsParams p) {
  constexpr int E = D / 32;
  const RowsGeom &g = p.g;
  const int32_t n = blockIdx.x, h = blockIdx.y, Hq = gridDim.y;
  const int32_t t = n / g.batch, b = n - t * g.batch, x = h / g.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t L = g.seqlens[b];
  bool bad = bad_length(g, L);
  const int32_t P = g.prefix_len != nullptr ? clamp_prefix(g, *g.prefix_len, bad) : 0;
  RowRange own = own_row_range(g, L, t);
  const int32_t oldest = oldest_in_ring(g, L);
  if (own.hi > 0 && imax32(own.lo, g.sinks) < oldest && oldest > g.sinks) {
    bad = true;
    own.lo = imin32(own.hi, imax32(own.lo, oldest));
  }
  const RowRange pre = prefix_row_range(g, L, t, P);
  if (bad && h == 0 && threadIdx.x == 0) atomicOr(p.status, kStatusSeqlen);
  const int32_t pin = imin32(imin32(own.pin, own.hi), own.lo);  // pinned rows below the window
  const int32_t n_pre = pre.hi - pre.lo, n_own = own.hi - own.lo;
  float q[E], o[E];
  const uint16_t *qr = p.q + (static_cast<int64_t>(n) * Hq + h) * D;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = bf16lo(qr[lane + 32 * e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int64_t row = static_cast<int64_t>(g.n_kv_heads) * D;
  for (int32_t i = warp; i < n_pre + pin + n_own; i += kSimpleWarps) {
    const uint16_t *kr, *vr;
    if (i < n_pre) {
      const int64_t off = (pre.lo + i) * row + x * D;
      kr = p.pk + off;
      vr = p.pv + off;
    } else {
      const int32_t j = i - n_pre;
      const int32_t pos = j < pin ? j : own.lo + j - pin;
      const int64_t off = b * p.batch_stride + slot_of(pos, g.sinks, g.capacity) * row + x * D;
      kr = p.k + off;
      vr = p.v + off;
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], bf16lo(kr[lane + 32 * e]), s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s = p.post != 0.f ? p.post * tanhf(s * p.qscale) : s * p.qscale;
    const float mn = fmaxf(m, s);
    const float a = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(w, bf16lo(vr[lane + 32 * e]), o[e] * a);
  }
  __shared__ float sm[kSimpleWarps], sl[kSimpleWarps], so[kSimpleWarps][D];
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = o[e];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float M = -INFINITY, Z = 0.f;
  for (int w = 0; w < kSimpleWarps; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < kSimpleWarps; ++w) Z += sl[w] > 0.f ? sl[w] * exp2f(sm[w] - M) : 0.f;
  for (int d = threadIdx.x; d < D; d += 32 * kSimpleWarps) {
    float acc = 0.f;
    for (int w = 0; w < kSimpleWarps; ++w)
      if (sl[w] > 0.f) acc += so[w][d] * exp2f(sm[w] - M);
    p.out[(static_cast<int64_t>(n) * Hq + h) * D + d] = f32_to_bf16_rn(Z > 0.f ? acc / Z : 0.f);
  }
  if (threadIdx.x == 0 && p.lse != nullptr)
    p.lse[static_cast<int64_t>(n) * Hq + h] =
        Z > 0.f ? (M + log2f(Z)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace gdattn
