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
// latency: the scan, one bisection and one store each.  64 sequences of one token: 2.2 us
// a call in a replayed graph.
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
      // In 64 bits: a negative length under many new tokens leaves 32.
      const int64_t at = static_cast<int64_t>(L) - __ldg(p.new_lens + seq) + (i - s_start[a]);
      pos = static_cast<int32_t>(at > INT32_MIN ? at : INT32_MIN);
      // A row of the ring survives the step if no later position takes its slot.
      if (pos >= 0 && (pos < p.sinks || at >= static_cast<int64_t>(L) - (p.capacity - p.sinks)))
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
// never again here, so they pass the L1.  12000 rows of 8 x 256 in K and V: 35 us, 5.6
// TB/s, 87 % of a copy of the whole memory's rate.
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
// (The remainder is taken as q s - x and its product subtracted, so that a zero keeps
// its sign: x - q s is +0 for x = -0.)
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(q, s, -x), -r, q);
}

// Scales that leave the reciprocal, the guess and its remainder (2^-46 of the product)
// normal, for every quotient that is not far below e4m3's smallest number.
__device__ __forceinline__ bool plain_scale(float s) { return s > 1e-18f && s < 1e30f; }

__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b & 0x7FFF7FFFu));
  return r;
}

__device__ __forceinline__ uint32_t codes_of(uint32_t x, uint32_t y, float s, float r) {
  return e4m3x2_rn(quotient(bf16lo(x), s, r), quotient(bf16hi(x), s, r)) |
         static_cast<uint32_t>(e4m3x2_rn(quotient(bf16lo(y), s, r), quotient(bf16hi(y), s, r)))
             << 16;
}
__device__ __forceinline__ uint32_t codes_by_division(uint32_t x, uint32_t y, float s) {
  if (!(s > 0.f)) return 0;  // a row of zeros
  return e4m3x2_rn(__fdiv_rn(bf16lo(x), s), __fdiv_rn(bf16hi(x), s)) |
         static_cast<uint32_t>(e4m3x2_rn(__fdiv_rn(bf16lo(y), s), __fdiv_rn(bf16hi(y), s))) << 16;
}

// A row of one KV head: its largest magnitude, then its codes.  D / 32 lanes share a
// row, 32 elements each, so that what a row costs besides its elements is spread over
// four (D = 256) rows a warp: with a warp for each row the kernel was bound by
// instructions (51 us for 12000 rows of 8 heads; this way 32 us, 4.7 TB/s, 61 % of the
// issue slots: 2 D bytes read and D + 4 written).
template <int D>
__global__ void __launch_bounds__(kCacheWriteThreads)
    cache_write_fp8_kernel(const CacheWriteParams p) {
  constexpr int LANES = D / 32;              // of a row
  constexpr int ROWS = kCacheWriteThreads / LANES;
  const int l = threadIdx.x % LANES;
  const uint16_t *rows = blockIdx.y == 0 ? p.k_rows : p.v_rows;
  uint8_t *cache = blockIdx.y == 0 ? p.k_cache : p.v_cache;
  float *scales = blockIdx.y == 0 ? p.k_scale : p.v_scale;
  const uint32_t H = static_cast<uint32_t>(p.n_kv_heads);
  const int64_t row_elems = static_cast<int64_t>(H) * D;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS;
  const int64_t r0 = first / H;
  const uint32_t hh = static_cast<uint32_t>(first - r0 * H) + threadIdx.x / LANES;
  const uint32_t row = hh / H, h = hh - row * H;
  const int64_t r = r0 + row;
  int32_t b = 0, slot = 0;
  const bool there = r < p.n_rows && row_target(p, static_cast<int32_t>(r), b, slot);
  uint4 x[4] = {};
  if (there) {
    const uint16_t *src = rows + r * p.row_stride + h * D + l * 8;
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = ld_nc_v4(src + c * 8 * LANES);
  }
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    top = absmax_bf16x2(top, x[c].x);
    top = absmax_bf16x2(top, x[c].y);
    top = absmax_bf16x2(top, x[c].z);
    top = absmax_bf16x2(top, x[c].w);
  }
  float amax = fmaxf(bf16lo(top), bf16hi(top));
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float scale = __fdiv_rn(amax, 448.f);
  if (!there) return;
  uint8_t *dst = cache + b * p.batch_stride + slot * row_elems + h * D + l * 8;
  if (plain_scale(scale)) {
    const float inv = __frcp_rn(scale);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint2 *>(dst + c * 8 * LANES) =
          make_uint2(codes_of(x[c].x, x[c].y, scale, inv), codes_of(x[c].z, x[c].w, scale, inv));
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint2 *>(dst + c * 8 * LANES) = make_uint2(
          codes_by_division(x[c].x, x[c].y, scale), codes_by_division(x[c].z, x[c].w, scale));
  }
  if (l == 0) scales[(static_cast<int64_t>(b) * H + h) * p.capacity + slot] = scale;
}

}  // namespace gdattn
