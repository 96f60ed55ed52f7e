// Slots of a step's packed rows, and the writes of K and V rows that go by them.
#pragma once

#include <cstdint>

#include "../ptx.cuh"
#include "rows_plan.cuh"

namespace gdattn {

// ------------------------------------------------------------- slot maps
struct SlotMapParams {
  const int32_t *seqlens;   // [batch], with the step's tokens
  const int32_t *new_lens;  // [batch], tokens of this step
  int32_t *row_start;       // [batch + 1]
  int32_t *row_seq, *row_pos, *row_slot;  // [n_rows]
  int32_t batch, n_rows, capacity, sinks;
};

constexpr int kSlotMapThreads = 256;
constexpr int kSlotMapRows = 1024;  // rows per CTA

// Every CTA scans the step's lengths itself (one load per sequence; no second
// launch and no wait between CTAs), keeps the sequences that reach into its
// kSlotMapRows rows and then finds each row's sequence among them by bisection.
// At most kSlotMapRows non-empty sequences reach into a CTA's rows.  Bound by
// latency: the scan, one bisection and one store each.
__global__ void __launch_bounds__(kSlotMapThreads) slot_map_kernel(const SlotMapParams p) {
  __shared__ int32_t s_start[kSlotMapRows], s_seq[kSlotMapRows];
  __shared__ int64_t s_warp[kSlotMapThreads / 32];
  __shared__ int32_t s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kSlotMapRows;
  const int64_t r1 = r0 + kSlotMapRows;
  const bool first_cta = blockIdx.x == 0;
  if (tid == 0) s_count = 0;
  int64_t base = 0;
  __syncthreads();
  for (int32_t b0 = 0; b0 < p.batch; b0 += kSlotMapThreads) {
    const int32_t b = b0 + tid;
    const int32_t n = b < p.batch ? imax32(0, __ldg(p.new_lens + b)) : 0;
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int64_t before = base, sum = 0;
#pragma unroll
    for (int w = 0; w < kSlotMapThreads / 32; ++w) {
      if (w < warp) before += s_warp[w];
      sum += s_warp[w];
    }
    const int64_t start = before + incl - n;
    if (first_cta && b < p.batch) {
      if (b == 0) p.row_start[0] = 0;
      p.row_start[b + 1] = static_cast<int32_t>(start + n < INT32_MAX ? start + n : INT32_MAX);
    }
    // Sequences come in the order of their rows; within a group of threads the
    // list is ordered by counting the ones in front.
    const bool mine = n > 0 && start < r1 && start + n > r0;
    const unsigned ballot = __ballot_sync(0xffffffffu, mine);
    __shared__ int32_t s_hits[kSlotMapThreads / 32];
    if (lane == 0) s_hits[warp] = __popc(ballot);
    __syncthreads();
    int32_t at = s_count, hits = 0;
#pragma unroll
    for (int w = 0; w < kSlotMapThreads / 32; ++w) {
      if (w < warp) at += s_hits[w];
      hits += s_hits[w];
    }
    if (mine) {
      at += __popc(ballot & ((1u << lane) - 1));
      s_start[at] = static_cast<int32_t>(start - r0);  // may be negative
      s_seq[at] = b;
    }
    base += sum;
    __syncthreads();
    if (tid == 0) s_count += hits;
    __syncthreads();
    if (!first_cta && base >= r1) break;
  }
  const int32_t count = s_count;
  for (int32_t i = tid; i < kSlotMapRows && r0 + i < p.n_rows; i += kSlotMapThreads) {
    int32_t seq = -1, pos = -1, slot = -1;
    if (r0 + i < base && count > 0) {
      int32_t a = 0, z = count - 1;  // last entry that starts at or before row i
      while (a < z) {
        const int32_t mid = (a + z + 1) >> 1;
        if (s_start[mid] <= i) a = mid; else z = mid - 1;
      }
      seq = s_seq[a];
      const int32_t L = __ldg(p.seqlens + seq);
      pos = L - imax32(0, __ldg(p.new_lens + seq)) + (i - s_start[a]);
      // A row of the ring survives the step if no later position takes its slot.
      if (pos >= 0 && (pos < p.sinks || pos >= L - (p.capacity - p.sinks)))
        slot = slot_of(pos, p.sinks, p.capacity);
    }
    p.row_seq[r0 + i] = seq;
    p.row_pos[r0 + i] = pos;
    p.row_slot[r0 + i] = slot;
  }
}

// ------------------------------------------------------------ cache writes
struct CacheWriteParams {
  const uint16_t *rows[2];   // K, V rows (V null: K = V)
  uint8_t *cache[2];
  float *scale[2];           // fp8
  const int32_t *row_seq, *row_slot;
  int64_t row_stride;        // elements between rows
  int64_t batch_stride;      // elements between sequences of a cache
  int32_t n_rows, batch, capacity, n_kv_heads, head_dim;
};

constexpr int kCacheWriteThreads = 256;

// One 16-byte piece of one row per thread and step.
__global__ void __launch_bounds__(kCacheWriteThreads) cache_write_kernel(const CacheWriteParams p) {
  const int32_t pieces = p.n_kv_heads * p.head_dim / 8;  // of a row
  const int64_t total = static_cast<int64_t>(p.n_rows) * pieces;
  const int w = blockIdx.y;
  const int64_t row_elems = static_cast<int64_t>(p.n_kv_heads) * p.head_dim;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCacheWriteThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kCacheWriteThreads) {
    const int32_t r = static_cast<int32_t>(i / pieces), e = static_cast<int32_t>(i % pieces) * 8;
    const int32_t b = __ldg(p.row_seq + r), slot = __ldg(p.row_slot + r);
    if (b < 0 || b >= p.batch || slot < 0 || slot >= p.capacity) continue;
    const uint4 v = *reinterpret_cast<const uint4 *>(p.rows[w] + r * p.row_stride + e);
    *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(p.cache[w]) + b * p.batch_stride +
                               slot * row_elems + e) = v;
  }
}

// One warp per (row, KV head): the row's largest magnitude, then its codes.
template <int D>
__global__ void __launch_bounds__(kCacheWriteThreads)
    cache_write_fp8_kernel(const CacheWriteParams p) {
  constexpr int E = D / 32;  // elements per lane: 8 or 16
  const int lane = threadIdx.x & 31;
  const int w = blockIdx.y;
  const int64_t total = static_cast<int64_t>(p.n_rows) * p.n_kv_heads;
  const int64_t row_elems = static_cast<int64_t>(p.n_kv_heads) * D;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kCacheWriteThreads + threadIdx.x) >> 5;
       i < total; i += static_cast<int64_t>(gridDim.x) * kCacheWriteThreads / 32) {
    const int32_t r = static_cast<int32_t>(i / p.n_kv_heads);
    const int32_t h = static_cast<int32_t>(i % p.n_kv_heads);
    const int32_t b = __ldg(p.row_seq + r), slot = __ldg(p.row_slot + r);
    if (b < 0 || b >= p.batch || slot < 0 || slot >= p.capacity) continue;
    const uint16_t *src = p.rows[w] + r * p.row_stride + h * D + lane * E;
    uint32_t raw[E / 2];
#pragma unroll
    for (int c = 0; c < E / 8; ++c)
      *reinterpret_cast<uint4 *>(raw + 4 * c) = *reinterpret_cast<const uint4 *>(src + 8 * c);
    float x[E], amax = 0.f;
#pragma unroll
    for (int c = 0; c < E / 2; ++c) {
      x[2 * c] = bf16lo(raw[c]);
      x[2 * c + 1] = bf16hi(raw[c]);
      amax = fmaxf(amax, fmaxf(fabsf(x[2 * c]), fabsf(x[2 * c + 1])));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float scale = __fdiv_rn(amax, 448.f);
    uint16_t code[E / 2];
#pragma unroll
    for (int c = 0; c < E / 2; ++c)
      code[c] = scale > 0.f
                    ? e4m3x2_rn(__fdiv_rn(x[2 * c], scale), __fdiv_rn(x[2 * c + 1], scale))
                    : static_cast<uint16_t>(0);
    uint8_t *dst = p.cache[w] + b * p.batch_stride + slot * row_elems + h * D + lane * E;
#pragma unroll
    for (int c = 0; c < E / 8; ++c) {
      uint2 pk;
      pk.x = code[4 * c] | static_cast<uint32_t>(code[4 * c + 1]) << 16;
      pk.y = code[4 * c + 2] | static_cast<uint32_t>(code[4 * c + 3]) << 16;
      *reinterpret_cast<uint2 *>(dst + 8 * c) = pk;
    }
    if (lane == 0)
      p.scale[w][(static_cast<int64_t>(b) * p.n_kv_heads + h) * p.capacity + slot] = scale;
  }
}

}  // namespace gdattn
