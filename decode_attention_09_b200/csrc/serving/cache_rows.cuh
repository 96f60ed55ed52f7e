// Slots of a step's packed rows, and the writes of K and V rows that go by them.
#pragma once

#include <cstdint>

#include "../ptx.cuh"
#include "rows_plan.cuh"

namespace gdattn {

// 16 bytes that this kernel reads once, past the L1.
__device__ __forceinline__ uint4 ld_nc_v4(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

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
  const uint16_t *k_rows, *v_rows;  // v_rows null: K = V
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;         // fp8
  const int32_t *row_seq, *row_slot;
  int64_t row_stride;               // elements between rows
  int64_t batch_stride;             // elements between sequences of a cache
  int32_t n_rows, batch, capacity, n_kv_heads, head_dim;
};

constexpr int kCacheWriteThreads = 256;
constexpr int kCacheWritePieces = 4;  // 16-byte pieces per thread and tensor

// Where a row goes: the offset of its cache row in rows, or false.
__device__ __forceinline__ bool row_target(const CacheWriteParams &p, int32_t r, int32_t &b,
                                           int32_t &slot) {
  b = __ldg(p.row_seq + r);
  slot = __ldg(p.row_slot + r);
  return b >= 0 && b < p.batch && slot >= 0 && slot < p.capacity;
}

// A copy, bound by HBM: each thread moves kCacheWritePieces 16-byte pieces of K and
// as many of V, all loads in flight before the first store.  Rows are read once and
// never again here, so they pass the L1.
__global__ void __launch_bounds__(kCacheWriteThreads) cache_write_kernel(const CacheWriteParams p) {
  const uint32_t pieces = static_cast<uint32_t>(p.n_kv_heads) * p.head_dim / 8;  // of a row
  const int64_t row_elems = static_cast<int64_t>(pieces) * 8;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kCacheWriteThreads * kCacheWritePieces);
  const int32_t r0 = static_cast<int32_t>(first / pieces);
  const uint32_t e0 = static_cast<uint32_t>(first - static_cast<int64_t>(r0) * pieces);
  uint4 kx[kCacheWritePieces], vx[kCacheWritePieces];
  int64_t dst[kCacheWritePieces];
#pragma unroll
  for (int j = 0; j < kCacheWritePieces; ++j) {
    const uint32_t i = e0 + j * kCacheWriteThreads + threadIdx.x;
    const uint32_t row = i / pieces, e = (i - row * pieces) * 8;
    const int64_t r = static_cast<int64_t>(r0) + row;
    dst[j] = -1;
    int32_t b, slot;
    if (r < p.n_rows && row_target(p, static_cast<int32_t>(r), b, slot)) {
      dst[j] = b * p.batch_stride + slot * row_elems + e;
      kx[j] = ld_nc_v4(p.k_rows + r * p.row_stride + e);
      if (p.v_rows != nullptr) vx[j] = ld_nc_v4(p.v_rows + r * p.row_stride + e);
    }
  }
#pragma unroll
  for (int j = 0; j < kCacheWritePieces; ++j) {
    if (dst[j] < 0) continue;
    *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(p.k_cache) + dst[j]) = kx[j];
    if (p.v_rows != nullptr)
      *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(p.v_cache) + dst[j]) = vx[j];
  }
}

// x / s rounded to fp32, r being 1 / s rounded: Markstein's correction (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).
// The remainder of the first guess is exact in a fused multiply-add, and the sum is
// within 2^-47 of the quotient before its one rounding.  That rounding could only go
// the other way next to a midpoint of fp32, which a bf16 x over a scale that is itself
// x' / 448 never comes that close to; the tests go through every pair of mantissas.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}

// Scales that leave the reciprocal, the guess and its remainder (2^-46 of the product)
// normal, for every quotient that is not far below e4m3's smallest number.
__device__ __forceinline__ bool plain_scale(float s) { return s > 1e-18f && s < 1e30f; }

// Word w of four (w a constant), two bf16.
__device__ __forceinline__ uint32_t word(const uint4 &v, int w) {
  return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
}

// One warp per (row, KV head) at a time, kFp8Rows of them in flight: the row's largest
// magnitude, then its codes.  Bound by HBM (2 D bytes read, D + 4 written).
constexpr int kFp8Rows = 4;
template <int D>
__global__ void __launch_bounds__(kCacheWriteThreads)
    cache_write_fp8_kernel(const CacheWriteParams p) {
  constexpr int E = D / 32;  // elements per lane: 8 or 16
  const int lane = threadIdx.x & 31;
  const uint16_t *rows = blockIdx.y == 0 ? p.k_rows : p.v_rows;
  uint8_t *cache = blockIdx.y == 0 ? p.k_cache : p.v_cache;
  float *scales = blockIdx.y == 0 ? p.k_scale : p.v_scale;
  const uint32_t H = static_cast<uint32_t>(p.n_kv_heads);
  const int64_t row_elems = static_cast<int64_t>(H) * D;
  const int64_t first =
      (static_cast<int64_t>(blockIdx.x) * (kCacheWriteThreads / 32) + (threadIdx.x >> 5)) * kFp8Rows;
  const int64_t r0 = first / H;
  const uint32_t h0 = static_cast<uint32_t>(first - r0 * H);
  uint4 raw[kFp8Rows][E / 8];
  int64_t dst[kFp8Rows], sat[kFp8Rows];
#pragma unroll
  for (int j = 0; j < kFp8Rows; ++j) {
    const uint32_t row = (h0 + j) / H, h = h0 + j - row * H;
    const int64_t r = r0 + row;
    dst[j] = -1;
    int32_t b, slot;
    if (r < p.n_rows && row_target(p, static_cast<int32_t>(r), b, slot)) {
      dst[j] = b * p.batch_stride + slot * row_elems + h * D + lane * E;
      sat[j] = (static_cast<int64_t>(b) * H + h) * p.capacity + slot;
      const uint16_t *src = rows + r * p.row_stride + h * D + lane * E;
#pragma unroll
      for (int c = 0; c < E / 8; ++c) raw[j][c] = ld_nc_v4(src + 8 * c);
    }
  }
#pragma unroll
  for (int j = 0; j < kFp8Rows; ++j) {
    if (dst[j] < 0) continue;  // the whole warp
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < E / 2; ++c) {
      const uint32_t x = word(raw[j][c / 4], c % 4);
      amax = fmaxf(amax, fmaxf(fabsf(bf16lo(x)), fabsf(bf16hi(x))));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float scale = __fdiv_rn(amax, 448.f);
    const bool plain = plain_scale(scale);  // of the whole warp
    const float inv = plain ? __frcp_rn(scale) : 0.f;
    uint32_t code[E / 4] = {};
#pragma unroll
    for (int c = 0; c < E / 2; ++c) {
      const uint32_t x = word(raw[j][c / 4], c % 4);
      uint16_t two = 0;
      if (plain)
        two = e4m3x2_rn(quotient(bf16lo(x), scale, inv), quotient(bf16hi(x), scale, inv));
      else if (scale > 0.f)
        two = e4m3x2_rn(__fdiv_rn(bf16lo(x), scale), __fdiv_rn(bf16hi(x), scale));
      code[c / 2] |= static_cast<uint32_t>(two) << (16 * (c % 2));
    }
    if (E == 8)
      *reinterpret_cast<uint2 *>(cache + dst[j]) = make_uint2(code[0], code[1]);
    else
      *reinterpret_cast<uint4 *>(cache + dst[j]) =
          make_uint4(code[0], code[1], code[E / 4 - 2], code[E / 4 - 1]);
    if (lane == 0) scales[sat[j]] = scale;
  }
}

}  // namespace gdattn
