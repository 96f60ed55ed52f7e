// Attention of blocks of query rows over cache rows, on the 5th-generation tensor
// cores: the kernel of gdattn_decode_sink and gdattn_decode_prefix.
//
// A block is up to 128 query rows of one KV head: tokens of one sequence times
// the query heads of the group, or (token, sequence) pairs of the batch times the
// group, over the shared prefix.  Per tile of 64 cache rows
//
//   S[128 x 64]   = Q[128 x D] . K_tile^T[D x 64]
//   O[128 x D]   += P_hi[128 x 64] . V_tile[64 x D] + P_lo[128 x 64] . V_tile[64 x D]
//
// with the running maximum and sum of a softmax in one pass.  Every TMEM lane is a
// query row, so a softmax thread owns a row.  Weights are stored as bf16 plus the
// bf16 remainder (truncated; 2^-14 relative).  A row's reference moves only when a
// score exceeds it by 2^24: floating point keeps weights above 1 as exact as those
// below, and 2^24 times 2^17 keys times the largest |V| of a model stays far from
// the largest fp32.  The thread then rescales its O row in TMEM.
//
// head_dim 512 (NH = 2): O alone would fill tensor memory, so a block runs on a
// cluster of two CTAs, each with 256 of the dims of Q, K, V and O.  Each computes
// the scores' partial sum over its dims and sends it to the other through
// distributed shared memory (32 KiB a tile and direction); both then add the two
// parts in the same way, so their softmax decisions agree bit for bit.  A cache
// row crosses HBM once and no product is computed twice.
//
// Work split: rows_chunks.cuh lays all tiles end to end and gives each worker (CTA
// or pair) an equal chunk; loads run ahead across units.  Whole units are written
// directly (sinks), pieces as normalised fp32 partials plus log2-sum-exp, which the
// CTA of the last piece joins where a block has few rows, and rows_merge.cuh elsewhere.
//
// Shared memory (1 CTA per SM): Q blocks (64 KiB; two buffers when a block's rows
// fill at most half), a ring of 32 KiB tiles (five for NH = 1; three for NH = 2 beside
// two 32 KiB score exchange buffers).  K and V tiles take turns in the ring; with
// K = V a tile serves both products.  Partial tiles are fetched in 16-row boxes.
//
// TMEM: O (256 columns) and four buffers of 64 columns, each first a tile's scores,
// then, written in place by 16 columns, its weights.
//
// Warps: 3 loads tiles, 0 loads Q, 1 issues Q.K and owns TMEM, 2 issues P.V, 4-7 and
// 8-11 run the softmax of even and of odd tiles.  (Warps 0, 4 and 8 share a scheduler:
// where a block has few rows, 4 and 8 have them all, and the tile loader beside them cost
// a verify step 2 to 3 percent.)  Every wait is bounded.
//
// What bounds it: a tile's softmax is a chain of some 4500 cycles (two reads of the
// scores from tensor memory, the exponentials, the stores of the weights), the same for
// one row and for 128, and two groups in turn give a tile every 2500 to 4000.  That comes
// with query rows in the lanes: a block of one token has two live lanes of 128.  The
// library's pair kernels, which put the cache rows there, take 17 us where this one takes
// 22.6 (8 sequences, one token, windows of 1024) and 82 where it takes 108 to 123 (64).
// With four tokens and up the two are even at 8 sequences (24), 89 to 125 at 64.  Its loops
// take 16 columns and stay rolled, because all of the L1 is in use as shared memory and a
// spilled register costs a trip to the L2: 32 or 64 columns at a time, or the next read in
// flight, spill 100 to 560 bytes and take 10 to 25 % longer.  Measured: 64 ragged sequences of 4
// tokens over windows of 1024 in 130 to 135 us (4.1 TB/s), an 8192-token prompt in 233 to
// 242 us (540 TFLOP/s of the formula's products, half as many again with the weights'
// second part), 64 sequences behind 8192 shared tokens at head_dim 512 in 75 to 78 us.
//
// A parity wait is sound only while its barrier is in the phase waited for or the
// next.  kfull, vfull: eight uses back, tile i - 8's products are done.  odone of tile
// j: Q.K of tile j waited for the use before it, and whoever waits has seen tile j's
// scores; it cannot complete again before tile j + 4, which needs the waiter's own
// weights.  refset: the two groups alternate inside a segment and meet at its end.
// oempty: a group arrives behind the segment's last P.V, whose first one waited for
// the phase before.
//
// Warp 3 finds the segments and passes them on in eight slots, without waiting for
// their readers: it writes segment n + 8 in front of loading that segment's first tile
// i, and to load tile i - 1 it waited for the products of tile i - 6 (or a later one).
// Tiles i - 7 and i - 6 come behind segment n's first tile, so both softmax groups,
// and with them every other warp, have read segment n.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "../ptx.cuh"
#include "rows_chunks.cuh"
#include "rows_plan.cuh"
#include "rows_ptx.cuh"

namespace gdattn {

template <int NH>
struct RowsConfig {
  static constexpr int DH = 256;                    // dims per CTA
  static constexpr int D = DH * NH;
  static constexpr int M = 128;                     // query rows per block
  static constexpr int TILE = kRowTile;
  static constexpr int CW = 16;                     // score columns a softmax loop takes at once
  static constexpr int BOXB = TILE * 128;           // 64 rows x 64 dims: 8 KiB
  static constexpr int TB = BOXB * (DH / 64);       // a tile: 32 KiB
  static constexpr int NST = NH == 1 ? 5 : 3;       // ring
  static constexpr uint32_t kAhead = NH == 1 ? 2 : 1;  // K tiles in front of V tiles
  static constexpr int QB = 64 * 1024;
  static constexpr int XB = M * TILE * 4;           // score exchange buffer: 32 KiB
  static constexpr int OFF_KV = QB;                 // Q first: its MMA reads run past short blocks
  static constexpr int OFF_X = OFF_KV + NST * TB;
  static constexpr int OFF_REF = OFF_X + (NH == 1 ? 0 : 2 * XB);  // [2][128] floats
  static constexpr int OFF_BAR = OFF_REF + 2 * M * 4;
  static constexpr int SMEM = OFF_BAR + 1024 + 1024;
  static constexpr int kThreads = 384;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t S_COL = 0;              // 4 buffers x 64, scores then weights
  static constexpr uint32_t O_COL = 256;            // 256
};
static_assert(RowsConfig<1>::SMEM <= 227 * 1024 && RowsConfig<2>::SMEM <= 227 * 1024,
              "shared memory budget");

struct RowsParams {
  RowsGeom g;
  uint16_t *out;       // bf16 [T][B][Hq][D]
  int32_t out_halves;  // out is on a 16-byte boundary only
  float *lse;          // [T][B][Hq] or null
  // (own_o and pre_o are on 32-byte boundaries)
  float *own_o, *own_lse;  // partials of own units, rs rows a slot; a CTA pair's two have
  int64_t lse_stride;      // a copy of own_lse each, lse_stride elements apart
  float *pre_o, *pre_lse;  // partials of prefix units, rp rows a slot
  CutEntry *cuts;          // [workers - 1], a call without a prefix (null: the last piece's
                           // CTA joins a cut unit here, no merge kernel follows), and
  uint32_t *counters;      // [workers * NH] pieces left so far, zero between calls
  PrefixEntry *prefix_entry;  // a call with one, and
  int32_t *pair_start;        // [batch * nqb + 1]
  uint32_t *status;
  int32_t workers;
  int32_t rs, rp;      // rows of a slot
  int32_t q_stride;    // bytes between the 64-dim chunks of a Q block (1 KiB multiple)
  int32_t q_bufs;      // Q buffers (1 or 2)
  int32_t q_bytes_own, q_bytes_pre;  // bytes of a 64-dim chunk that TMA writes
  float qscale;        // scale * log2(e), or scale / cap with a soft-cap
  float post;          // cap * log2(e), or 0
  int32_t test_withhold;
  int32_t merge_shares;  // warps that share a row of the merge
};

// The tensor maps of a call: caches and prefix in boxes of 64 rows and of 16,
// q by (token, sequence x head) and by (token x sequence, head).
struct RowsMaps {
  CUtensorMap k, v, k16, v16;
  CUtensorMap pk, pv, pk16, pv16;
  CUtensorMap q_own, q_pre;
};

// Ring entry of tile i's K: with separate tensors K_0 .. K_a are followed by V_0,
// K_(a+1), V_1 and so on (a = kAhead); with K = V there is one entry a tile.
template <int NH, bool SHARED>
__device__ __forceinline__ uint32_t k_entry(uint32_t i) {
  constexpr uint32_t a = RowsConfig<NH>::kAhead;
  return SHARED ? i : (i <= a ? i : 2 * i - a);
}
// And of its V: one behind K_(i + a).  Behind a chunk's last K the entries of the K
// that would follow stay unused; no later entry takes their slots.
template <int NH, bool SHARED>
__device__ __forceinline__ uint32_t v_entry(uint32_t i) {
  constexpr uint32_t a = RowsConfig<NH>::kAhead;
  return SHARED ? i : 2 * i + a + 1;
}

// Joins the pieces of one row of a cut unit, 256 dims of it, by one warp:
//   lse = log2 sum_i 2^lse_i,  out = sum_i 2^(lse_i - lse) o_i.
template <int D>
__device__ __forceinline__ void join_pieces(const float *o, const float *lse, const PartSlots &at,
                                            int32_t rows, int32_t r, uint16_t *out,
                                            float *out_lse) {
  constexpr int kFlight = 4;
  const int lane = threadIdx.x & 31;
  float4 acc[2] = {};
  float m = -INFINITY, z = 0.f;
  for (int32_t i0 = 0; i0 < at.n; i0 += kFlight) {
    float e[kFlight];
    float4 v[kFlight][2];
#pragma unroll
    for (int q = 0; q < kFlight; ++q) {
      const int32_t i = i0 + q;
      e[q] = -INFINITY;
      if (i < at.n) {
        const int64_t row =
            static_cast<int64_t>(i == 0 ? at.first : at.next + (i - 1) * at.step) * rows + r;
        e[q] = __ldcg(lse + row);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          v[q][c] = __ldcg(reinterpret_cast<const float4 *>(o + row * D) + c * 32 + lane);
      }
    }
#pragma unroll
    for (int q = 0; q < kFlight; ++q) {
      if (e[q] == -INFINITY) continue;  // an empty piece adds nothing
      const float top = fmaxf(m, e[q]);
      const float a = exp2f(m - top), f = exp2f(e[q] - top);
      m = top;
      z = fmaf(z, a, f);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        acc[c].x = fmaf(f, v[q][c].x, acc[c].x * a);
        acc[c].y = fmaf(f, v[q][c].y, acc[c].y * a);
        acc[c].z = fmaf(f, v[q][c].z, acc[c].z * a);
        acc[c].w = fmaf(f, v[q][c].w, acc[c].w * a);
      }
    }
  }
  const float inv = z > 0.f ? __fdividef(1.f, z) : 0.f;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint2 pk;
    pk.x = pack_bf16x2(acc[c].x * inv, acc[c].y * inv);
    pk.y = pack_bf16x2(acc[c].z * inv, acc[c].w * inv);
    *reinterpret_cast<uint2 *>(out + (c * 32 + lane) * 4) = pk;
  }
  if (lane == 0 && out_lse != nullptr) *out_lse = z > 0.f ? (m + log2f(z)) * kLn2 : -INFINITY;
}

// Segment n of a chunk, found again from its start; for a warp whose loader gave up.
__device__ __noinline__ bool nth_segment(const RowsGeom *g, const RowsPlan *plan, uint32_t n,
                                         RowSegment *s) {
  RowSegments it;
  it.init(*plan);
  for (uint32_t k = 0; k <= n; ++k)
    if (!it.next(*g, *s)) return false;
  return true;
}

template <int NH, bool SHARED, bool CAP>
__global__ void __launch_bounds__(RowsConfig<NH>::kThreads, 1)
    rows_attn_kernel(const __grid_constant__ RowsMaps maps, const __grid_constant__ RowsParams p) {
  using Cfg = RowsConfig<NH>;
  constexpr int DH = Cfg::DH, NST = Cfg::NST, TILE = Cfg::TILE, CW = Cfg::CW;

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // By an offset: the compiler then knows that these are shared addresses of 32 bits.
  uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  uint8_t *qs = smem;
  uint8_t *kv = smem + Cfg::OFF_KV;
  // [2 groups][16 column quads][128 rows]
  float4 *xs = reinterpret_cast<float4 *>(smem + Cfg::OFF_X);
  float *ref = reinterpret_cast<float *>(smem + Cfg::OFF_REF);  // [2 groups][128 rows]
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::OFF_BAR);
  uint64_t *kfull = bars;          // [8] K of tile i & 7: TMA -> Q.K (with K = V everyone)
  uint64_t *vfull = bars + 8;      // [8] V of tile i & 7: TMA -> P.V, softmax (partial tiles)
  uint64_t *empty = bars + 16;     // [5] ring slot: Q.K / P.V -> TMA
  uint64_t *sfull = bars + 21;     // [4] Q.K -> softmax
  uint64_t *pfull = bars + 25;     // [4] softmax -> P.V
  uint64_t *odone = bars + 29;     // [4] P.V -> Q.K (the buffer is free), softmax (O is current)
  uint64_t *qfull = bars + 33;     // [2] TMA -> Q.K
  uint64_t *qempty = bars + 35;    // [2] Q.K -> TMA
  uint64_t *oempty = bars + 37;    // softmax (O was read) -> P.V
  uint64_t *drain = bars + 38;     // [2] the MMA warps: all their MMAs are done
  uint64_t *refset = bars + 40;    // [2][4] softmax warp -> the other group's: its reference is set
  uint64_t *xfull = bars + 48;     // [2][4] peer's softmax warp -> this one: its scores are here
  uint64_t *xfree = bars + 56;     // [2][4] peer's softmax warp: read what this one sent
  uint32_t *tmem_base_smem = reinterpret_cast<uint32_t *>(bars + 64);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 65);
  RowsPlan *plan_smem = reinterpret_cast<RowsPlan *>(bars + 66);
  static_assert(sizeof(RowsPlan) <= 9 * 8, "the plan's place");
  volatile int *last_piece = reinterpret_cast<volatile int *>(bars + 75);  // [2 groups]
  uint64_t *seg_full = bars + 76;  // [8] warp 3 -> everyone: segment n & 7 is there
  constexpr uint32_t kSlots = 8;
  int32_t *seg_slots = reinterpret_cast<int32_t *>(bars + 84);  // [8][kSegmentWords]
  static_assert(84 * 8 + kSlots * kSegmentWords * 4 <= 1024, "barriers and segments");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const RowsGeom &g = p.g;
  const int32_t worker = static_cast<int32_t>(blockIdx.x) / NH;
  const int rank = NH == 1 ? 0 : static_cast<int>(blockIdx.x) % NH;  // this CTA's dims

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) mbar_init(&empty[s], 1);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&pfull[s], 4);
      mbar_init(&odone[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&qfull[s], 1);
      mbar_init(&qempty[s], 1);
      mbar_init(&drain[s], 1);
    }
    mbar_init(oempty, 4);
    for (int s = 0; s < 8; ++s) {
      mbar_init(&seg_full[s], 1);
      mbar_init(&kfull[s], 1);
      mbar_init(&vfull[s], 1);
      mbar_init(&refset[s], 1);
      mbar_init(&xfull[s], 1);
      mbar_init(&xfree[s], 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 3 && lane == 0) {
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.q_own);
    if (g.prefix_len != nullptr) {
      prefetch_tensormap(&maps.pk);
      prefetch_tensormap(&maps.q_pre);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_base_smem, Cfg::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 0) {
    const RowsPlan pl = plan_rows(g, worker, p.workers);
    if (lane == 0) *plan_smem = pl;
  }
  grid_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (NH == 2) cluster_sync();  // the peer's barriers are there
  tc_fence_after();
  const uint32_t tmem = *tmem_base_smem;
  const RowsPlan &plan = *plan_smem;
  RowSegment seg;
  // Segment n (false: there is none), by a whole warp.
  auto take = [&](uint32_t n) {
    const bool there =
        mbar_wait(&seg_full[n % kSlots], (n / kSlots) & 1, abort_flag, p.status);
    if (__all_sync(0xffffffffu, there)) {
      unpack_segment(g, seg_slots + n % kSlots * kSegmentWords, seg);
      return seg.t1 > seg.t0;
    }
    // Every warp walks all segments, whatever failed: the groups' barriers stay paired.
    RowSegment found = {};
    const bool any = nth_segment(&p.g, plan_smem, n, &found);
    seg = found;
    return any;
  };

  if (warp == 3) {
    // --------------------------------------------------------- tile loads
    // Tiles of a sequence's cache without any of the step's own rows hold what earlier
    // steps wrote and are loaded before the kernel in front has ended.  A prefix may be
    // another sequence's cache, to which the call in front appends: its tiles wait.
    bool waited = false;
    // Rows that several blocks read (a prompt's, a prefix under many query rows) stay in
    // the L2; those that are read once make room first.  (All evicted first, an 8192-token
    // prompt read 910 MB from HBM for its 202.)
    const uint64_t once = l2_evict_first_policy(), again = l2_evict_normal_policy();
    bool ok = true;
    uint32_t nk = 0, nv = 0;  // tiles whose K, V were loaded
    auto load = [&](const RowSegment &sg, int32_t t, bool is_v) {
      const RowTile tile = unit_tile(sg.u, t);
      const uint32_t e = is_v ? v_entry<NH, SHARED>(nv) : k_entry<NH, SHARED>(nk);
      const int st = e % NST;
      if (e >= NST) ok = mbar_wait(&empty[st], ((e / NST) - 1) & 1, abort_flag, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (!waited && (sg.prefix || tile.pos + tile.ntok > sg.L - g.tokens)) {
        grid_dependency_wait();
        waited = true;
      }
      uint64_t *bar = is_v ? &vfull[nv & 7] : &kfull[nk & 7];
      const uint64_t pol = (sg.prefix ? g.npb : g.nqb) > 1 ? again : once;
      if (!(p.test_withhold && e == 0) && elect_one()) {
        const bool big = tile.ntok > 48;
        const int boxes = big ? 1 : (tile.ntok + 15) / 16;
        const CUtensorMap *map =
            sg.prefix ? (big ? (is_v ? &maps.pv : &maps.pk) : (is_v ? &maps.pv16 : &maps.pk16))
                      : (big ? (is_v ? &maps.v : &maps.k) : (is_v ? &maps.v16 : &maps.k16));
        uint8_t *dst = kv + st * Cfg::TB;
        if (boxes == 0) {
          mbar_arrive(bar);  // a tile of no rows: nothing to load
        } else {
          mbar_arrive_expect_tx(bar, static_cast<uint32_t>((big ? TILE : 16 * boxes) * 2 * DH));
#pragma unroll 1
          for (int q = 0; q < boxes; ++q)
#pragma unroll 1
            for (int j = 0; j < DH / 64; ++j)
              tma_load_4d(dst + j * Cfg::BOXB + q * 2048, map, rank * DH + 64 * j, sg.x,
                          tile.slot + 16 * q, sg.b, bar, pol);
        }
      }
      __syncwarp();
      ++(is_v ? nv : nk);
    };
    RowSegments segs;
    segs.init(plan);
    uint32_t n = 0;  // segments passed on
    auto next = [&]() {
      if (!ok) return false;
      const bool any = segs.next(g, seg);
      if (!any) seg = RowSegment{};  // tells the end: a segment of no tiles
      if (lane == 0) {
        pack_segment(seg, seg_slots + n % kSlots * kSegmentWords);
        mbar_arrive(&seg_full[n % kSlots]);
      }
      __syncwarp();
      ++n;
      return any;
    };
    if (SHARED) {
      while (next())
        for (int32_t t = seg.t0; ok && t < seg.t1; ++t) load(seg, t, false);
    } else {
      // K tiles run kAhead tiles in front of V tiles: a V tile is needed only after
      // its scores' softmax, and its slot is better used by a K tile until then.
      RowSegment vseg = {};
      int32_t vt = 0;
      uint32_t vn = 0;
      auto load_v = [&]() {
        if (vt == vseg.t1) {  // (at most kAhead segments behind the K tiles')
          unpack_segment(g, seg_slots + vn++ % kSlots * kSegmentWords, vseg);
          vt = vseg.t0;
        }
        load(vseg, vt++, true);
      };
      while (next())
        for (int32_t t = seg.t0; ok && t < seg.t1; ++t) {
          load(seg, t, false);
          if (ok && nk > Cfg::kAhead) load_v();
        }
      while (ok && nv < nk) load_v();
    }
    // Never leave with copies in flight into shared memory.
    volatile int no_abort = 0;
    for (uint32_t f = nk > NST ? nk - NST : 0; f < nk; ++f)
      if (!(p.test_withhold && f == 0)) mbar_wait(&kfull[f & 7], (f >> 3) & 1, &no_abort, p.status);
    for (uint32_t f = nv > NST ? nv - NST : 0; f < nv; ++f)
      mbar_wait(&vfull[f & 7], (f >> 3) & 1, &no_abort, p.status);
  } else if (warp == 0) {
    // ------------------------------------------------------------ Q loads
    grid_dependency_wait();
    bool has = take(0);
    if (rank == 0) {
      if (plan.bad && worker == 0 && lane == 0) atomicOr(p.status, kStatusSeqlen);
      if (g.prefix_len != nullptr) {
        if (worker == 0) write_pair_starts(g, plan, p.prefix_entry, p.pair_start);
      } else if (p.cuts != nullptr && worker > 0 && lane == 0) {
        CutEntry cut = {};
        if (has &&
            cut_parts(plan.total, p.workers, worker - 1, seg.start, g.unit_cost, seg.u.n,
                      cut.parts)) {
          cut.b = seg.b;
          cut.qb = seg.qb;
          cut.x = seg.x;
        } else {
          cut.parts.n = 0;
        }
        p.cuts[worker - 1] = cut;
      }
      __syncwarp();
    }
    bool ok = true;
    uint32_t n = 0;  // blocks so far
    while (ok && has) {
      const uint32_t buf = n % p.q_bufs, use = n / p.q_bufs;
      if (use > 0) ok = mbar_wait(&qempty[buf], (use - 1) & 1, abort_flag, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (elect_one()) {
        uint8_t *dst = qs + buf * 4 * p.q_stride;
        mbar_arrive_expect_tx(&qfull[buf], 4 * (seg.prefix ? p.q_bytes_pre : p.q_bytes_own));
#pragma unroll 1
        for (int j = 0; j < DH / 64; ++j) {
          if (seg.prefix)
            tma_load_tokens(dst + j * p.q_stride, &maps.q_pre, rank * DH + 64 * j, seg.x * g.group,
                        seg.qb * g.qt_pre, &qfull[buf]);
          else
            tma_load_tokens(dst + j * p.q_stride, &maps.q_own, rank * DH + 64 * j,
                        (seg.b * g.n_kv_heads + seg.x) * g.group, seg.qb * g.qt_seq, &qfull[buf]);
        }
      }
      __syncwarp();
      has = take(++n);
    }
    volatile int no_abort = 0;
    const uint32_t bufs = static_cast<uint32_t>(p.q_bufs);
    for (uint32_t f = n > bufs ? n - bufs : 0; f < n; ++f)
      mbar_wait(&qfull[f % bufs], (f / bufs) & 1, &no_abort, p.status);
  } else if (warp == 1) {
    // --------------------------------------------------------- Q.K MMAs
    const uint32_t idesc = idesc_bf16_f32(128, TILE, false, false);
    const uint64_t qdesc = smem_desc_sw128(smem_u32(qs), 16, 1024);  // K-major
    const uint64_t kdesc = smem_desc_sw128(smem_u32(kv), 16, 1024);  // K-major
    bool ok = true;
    uint32_t i = 0, n = 0;
    while (ok && take(n)) {
      const uint32_t buf = n % p.q_bufs, use = n / p.q_bufs;
      ok = mbar_wait(&qfull[buf], use & 1, abort_flag, p.status);
      ok = __all_sync(0xffffffffu, ok);
      const uint32_t qoff = (buf * 4 * p.q_stride) >> 4, qstep = p.q_stride >> 4;
      for (int32_t t = seg.t0; ok && t < seg.t1; ++t) {
        const int st = k_entry<NH, SHARED>(i) % NST, sb = i & 3;
        ok = mbar_wait(&kfull[i & 7], (i >> 3) & 1, abort_flag, p.status);
        if (ok && i >= 4) ok = mbar_wait(&odone[sb], ((i >> 2) - 1) & 1, abort_flag, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll 1
          for (int j = 0; j < DH / 64; ++j)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_bf16(tmem + Cfg::S_COL + sb * TILE, qdesc + qoff + j * qstep + kk * 2,
                          kdesc + ((st * Cfg::TB + j * Cfg::BOXB + kk * 32) >> 4), idesc,
                          (j | kk) != 0);
          tc_commit(&sfull[sb]);
          if (!SHARED) tc_commit(&empty[st]);
          if (t + 1 == seg.t1) tc_commit(&qempty[buf]);
        }
        __syncwarp();
        ++i;
      }
      ++n;
    }
    if (elect_one()) tc_commit(&drain[0]);
    __syncwarp();
    volatile int no_abort = 0;
    mbar_wait(&drain[0], 0, &no_abort, p.status);
  } else if (warp == 2) {
    // --------------------------------------------------------- P.V MMAs
    const uint32_t idesc = idesc_bf16_f32(128, DH, false, true);
    // V tile as the MN-major B operand: 64-dim chunks BOXB apart, 8 rows per 1 KiB
    const uint64_t vdesc = smem_desc_sw128(smem_u32(kv), Cfg::BOXB, 1024);
    bool ok = true;
    uint32_t i = 0, n = 0;
    for (; ok && take(n); ++n) {
      for (int32_t t = seg.t0; ok && t < seg.t1; ++t) {
        const int st = v_entry<NH, SHARED>(i) % NST, pb = i & 3;
        // The first product of a block overwrites O: its last block was read.
        if (t == seg.t0 && n > 0) ok = mbar_wait(oempty, (n - 1) & 1, abort_flag, p.status);
        if (ok) ok = mbar_wait(&pfull[pb], (i >> 2) & 1, abort_flag, p.status);
        if (ok) ok = mbar_wait(SHARED ? &kfull[i & 7] : &vfull[i & 7], (i >> 3) & 1, abort_flag, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          // A = P from tensor memory: 16 rows' weights are 8 columns of bf16 pairs,
          // followed by the 8 columns of their remainders.
#pragma unroll 1
          for (int kk = 0; kk < TILE / 16; ++kk)
#pragma unroll
            for (int part = 0; part < 2; ++part)
              tc_mma_bf16_ta(tmem + Cfg::O_COL, tmem + Cfg::S_COL + pb * TILE + kk * 16 + part * 8,
                             vdesc + ((st * Cfg::TB + kk * 2048) >> 4), idesc,
                             !(t == seg.t0 && kk == 0 && part == 0));
          tc_commit(&odone[pb]);
          tc_commit(&empty[st]);
        }
        __syncwarp();
        ++i;
      }
    }
    if (elect_one()) tc_commit(&drain[1]);
    __syncwarp();
    volatile int no_abort = 0;
    mbar_wait(&drain[1], 0, &no_abort, p.status);
  } else {
    // --------------------------------------------------------- softmax
    // Two groups of four warps take the tiles in turn (group i & 1 has tile i); warp
    // qd of either owns rows 32 qd .. 32 qd + 31.  The two threads of a row agree on
    // its reference through ref[group][row]: tile i's thread reads what tile i - 1's
    // has set, moves it if its scores outgrew it, and sets it for tile i + 1's.
    grid_dependency_wait();  // outputs are written below
    const int wg = (warp - 4) >> 2, qd = warp & 3;
    const int t128 = threadIdx.x & 127;
    const int r = 32 * qd + lane;  // this thread's query row (TMEM lane)
    const uint32_t lane_base = static_cast<uint32_t>(32 * qd) << 16;
    const int32_t Hq = g.n_kv_heads * g.group;
    float *ref_own = ref + wg * Cfg::M + r, *ref_other = ref + (wg ^ 1) * Cfg::M + r;
    uint64_t *set_own = &refset[wg * 4 + qd], *set_other = &refset[(wg ^ 1) * 4 + qd];
    const float sign = p.qscale >= 0.f ? 1.f : -1.f;
    const float2x qscale2 = pack2(p.qscale, p.qscale), minus_one = pack2(-1.f, -1.f);
    const SmallTanh small_tanh(p.qscale, p.post);
    bool ok = true;
    uint32_t i = 0;       // tiles so far
    uint32_t n_own = 0;   // references this warp set
    uint32_t n_other = 0; // references the other group's warp set, up to this tile
    // Behind a segment whose last tile was the other group's, that group reads the sum
    // this warp left in ref_own: wait for it before the slot is written again.
    bool lent = false;
    auto take_back_ref = [&]() {
      if (lent) pair_sync(5 + qd);
      lent = false;
    };
    const int32_t tq = r / g.group, h = r - tq * g.group;  // the row's token and head
    for (uint32_t n = 0; take(n); ++n) {
      // The row: its token, sequence and head, and the positions it sees.
      const int32_t qt = seg.prefix ? g.qt_pre : g.qt_seq;
      const int32_t all = seg.prefix ? g.tokens * g.batch : g.tokens;  // of this axis
      const int32_t nrow = imin32(qt, all - seg.qb * qt) * g.group;
      const bool row_ok = r < nrow;
      RowRange rg = {0, 0, 0};
      if (row_ok) {
        const int32_t a = seg.qb * qt + tq;
        if (seg.prefix) {
          const int32_t tok = a / g.batch;
          rg = prefix_row_range(g, __ldg(g.seqlens + a - tok * g.batch), tok, plan.prefix_len);
        } else {
          rg = own_row_range(g, seg.L, a);
        }
      }
      const bool act = 32 * qd < nrow;  // the warp has rows (warp-uniform)
      float m_ref = -INFINITY, l = 0.f;  // l: sum of this group's weights, for m_ref
      for (int32_t t = seg.t0; t < seg.t1; ++t, ++i) {
        const int sb = i & 3;
        if (static_cast<int>(i & 1) != wg) {
          if (act) ++n_other;
          continue;
        }
        if (ok) ok = mbar_wait(&sfull[sb], (i >> 2) & 1, abort_flag, p.status);
        ok = __all_sync(0xffffffffu, ok);
        const RowTile tile = unit_tile(seg.u, t);
        const uint32_t s_col = tmem + lane_base + Cfg::S_COL + sb * TILE;
        if (act) {
          // The tile is walked by CW columns in loops that stay rolled (see above): the
          // second read of the scores costs less than what keeping them would spill.
          if (ok) tc_fence_after();
          if (NH == 2) {
            // The peer holds the scores' other half of the dims: swap, then add (below).
            // (Sending the next tile's scores in front of this one's weights instead took
            // half as long again: it keeps the weights from P.V.)
            if (ok && n_own > 0)
              ok = mbar_wait_cluster(&xfree[wg * 4 + qd], (n_own - 1) & 1, abort_flag, p.status);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              const uint32_t dst = peer_smem(smem_u32(xs + wg * (Cfg::XB / 16) + r), rank ^ 1);
#pragma unroll 1
              for (int ch = 0; ch < TILE / CW; ++ch) {
                float s[CW];
                tmem_ld16(s_col + CW * ch, s);
#pragma unroll
                for (int c = 0; c < CW / 4; ++c)
                  st_peer_v4(dst + (CW / 4 * ch + c) * (Cfg::M * 16), s[4 * c], s[4 * c + 1],
                             s[4 * c + 2], s[4 * c + 3]);
              }
              __syncwarp();
              if (lane == 0) mbar_arrive_peer(peer_smem(smem_u32(&xfull[wg * 4 + qd]), rank ^ 1));
              ok = mbar_wait_cluster(&xfull[wg * 4 + qd], n_own & 1, abort_flag, p.status);
            }
            ok = __all_sync(0xffffffffu, ok);
          }
          auto walk = [&](auto &&f) {  // f(chunk, its CW scores)
#pragma unroll 1
            for (int ch = 0; ch < TILE / CW; ++ch) {
              float s[CW];
              if (ok) tmem_ld16(s_col + CW * ch, s);
              f(ch, s);
            }
          };
          // Column c is position tile.pos + c; bit c of `seen` says whether the row sees
          // it.  A tile that every row of the warp sees in full needs no mask.  (Lanes
          // without a row may compute anything: nothing of it is stored.)
          const bool inside = ok && tile.ntok == TILE &&
                              (!row_ok || (tile.pos >= rg.lo && tile.pos + TILE <= rg.hi));
          const bool masked = !__all_sync(0xffffffffu, inside);
          uint64_t seen = ~0ull;
          if (masked) {
            const int32_t hi = ok ? imin32(rg.hi - tile.pos, tile.ntok) : 0;
            seen = (~low_bits(rg.lo - tile.pos) | low_bits(rg.pin - tile.pos)) & low_bits(hi);
          }
          // The largest product (times the scale's sign: scale and soft-cap are monotonic).
          float best = -INFINITY;
          float widest = 0.f;  // with a soft-cap: the largest magnitude among the seen columns
          auto scan = [&](int ch, float (&s)[CW]) {
            if (NH == 2 && ok) {
              const float4 *x = xs + wg * (Cfg::XB / 16) + ch * (CW / 4) * Cfg::M + r;
#pragma unroll
              for (int c = 0; c < CW / 4; ++c) {
                const float4 o = x[c * Cfg::M];
                s[4 * c] += o.x;
                s[4 * c + 1] += o.y;
                s[4 * c + 2] += o.z;
                s[4 * c + 3] += o.w;
              }
              tmem_store16(s_col + CW * ch, s);
            }
            float m4[4] = {best, best, best, best};
            if (masked) {
              const uint32_t bits = static_cast<uint32_t>(seen >> (CW * ch));
#pragma unroll
              for (int c = 0; c < CW; ++c)
                m4[c & 3] = fmaxf(m4[c & 3], (bits >> c) & 1 ? s[c] * sign : -INFINITY);
              // A column that nobody sees may hold anything (what shared memory held before,
              // for one), so it has no say in how the others' weights are computed.
              if (CAP)
#pragma unroll
                for (int c = 0; c < CW; ++c) s[c] = (bits >> c) & 1 ? s[c] : 0.f;
            } else if (sign > 0.f) {
#pragma unroll
              for (int c = 0; c < CW; c += 2)
                m4[c / 2 & 3] = max3(m4[c / 2 & 3], s[c], s[c + 1]);
            } else {
#pragma unroll
              for (int c = 0; c < CW; c += 2)
                m4[c / 2 & 3] = -min3(-m4[c / 2 & 3], s[c], s[c + 1]);
            }
            best = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            if (CAP) {
              float a4[4] = {widest, widest, widest, widest};
#pragma unroll
              for (int c = 0; c < CW; c += 2)
                a4[c / 2 & 3] = max3(a4[c / 2 & 3], fabsf(s[c]), fabsf(s[c + 1]));
              widest = fmaxf(fmaxf(a4[0], a4[1]), fmaxf(a4[2], a4[3]));
            }
          };
          walk(scan);
          if (NH == 2 && ok) {
            tmem_store_wait();
            __syncwarp();
            if (lane == 0) mbar_arrive_peer(peer_smem(smem_u32(&xfree[wg * 4 + qd]), rank ^ 1));
          }
          const float mx =
              best == -INFINITY ? -INFINITY : score_log2<CAP>(best * sign, p.qscale, p.post);
          // The row's reference, as the tile before left it.
          float prev = -INFINITY;
          if (t > seg.t0) {
            if (ok) ok = mbar_wait(set_other, (n_other - 1) & 1, abort_flag, p.status);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) prev = *ref_other;
          }
          const bool moved = row_ok && mx > prev + kRefStep;
          // (A row without a reference has only zeros in O.)
          const bool rescale = moved && prev != -INFINITY;
          if (__any_sync(0xffffffffu, rescale)) {
            // The TMEM loads and stores are warp-wide: other rows multiply by 1.
            const float alpha = rescale ? exp2f(prev - mx) : 1.f;
            if (ok) ok = mbar_wait(&odone[(i - 1) & 3], ((i - 1) >> 2) & 1, abort_flag, p.status);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              tc_fence_after();
#pragma unroll 1
              for (int cb = 0; cb < DH / 16; ++cb) {
                float o[16];
                tmem_ld16(tmem + lane_base + Cfg::O_COL + cb * 16, o);
#pragma unroll
                for (int q = 0; q < 16; ++q) o[q] *= alpha;
                tmem_store16(tmem + lane_base + Cfg::O_COL + cb * 16, o);
              }
              tmem_store_wait();
            }
          }
          const float now = moved ? mx : prev;
          take_back_ref();
          *ref_own = now;
          __syncwarp();
          if (lane == 0) mbar_arrive(set_own);
          ++n_own;
          if (now != m_ref) {
            l = m_ref == -INFINITY ? 0.f : l * exp2f(m_ref - now);
            m_ref = now;
          }
          // Weights: bf16 pairs (column j holds rows 2j, 2j + 1) and remainders, both
          // truncated (the upper halves of the fp32 bits; the remainder is exact in
          // fp32 before its own truncation): 2^-14 relative.  A row without any score
          // yet (reference -inf) has only masked columns here.
          const float mr = now == -INFINITY ? 0.f : now;
          const bool small =
              CAP && __all_sync(0xffffffffu, !row_ok || widest * fabsf(p.qscale) <= kSmallTanh);
          const float2x minus_mr = pack2(-mr, -mr);
          float2x l2[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
          auto weigh = [&](int ch, float (&s)[CW]) {
            if (CAP && !small) {
#pragma unroll
              for (int c = 0; c < CW; ++c)
                s[c] = ex2_approx(score_log2<CAP>(s[c], p.qscale, p.post) - mr);
            } else {
#pragma unroll
              for (int c = 0; c < CW; c += 2) {
                const float2x x = pack2(s[c], s[c + 1]);
                float ea, eb;
                unpack2(CAP ? small_tanh(x, minus_mr) : fma2(x, qscale2, minus_mr), ea, eb);
                s[c] = ex2_approx(ea);
                s[c + 1] = ex2_approx(eb);
              }
            }
            if (masked) {
              const uint32_t bits = static_cast<uint32_t>(seen >> (CW * ch));
#pragma unroll
              for (int c = 0; c < CW; ++c) s[c] = (bits >> c) & 1 ? s[c] : 0.f;
            }
            float w[CW];
#pragma unroll
            for (int j = 0; j < CW / 2; ++j) {
              const uint32_t ua = __float_as_uint(s[2 * j]), ub = __float_as_uint(s[2 * j + 1]);
              const float2x pw = pack2(s[2 * j], s[2 * j + 1]);
              l2[j & 1] = add2(l2[j & 1], pw);
              const float2x hi = pack2(__uint_as_float(ua & 0xFFFF0000u),
                                       __uint_as_float(ub & 0xFFFF0000u));
              float ra, rb;
              unpack2(fma2(hi, minus_one, pw), ra, rb);
              w[j] = __uint_as_float(__byte_perm(ua, ub, 0x7632));  // 8 columns of weights,
              w[j + 8] = __uint_as_float(                           // 8 of remainders
                  __byte_perm(__float_as_uint(ra), __float_as_uint(rb), 0x7632));
            }
            if (ok) tmem_store16(s_col + CW * ch, w);
          };
          walk(weigh);
          if (ok) tmem_store_wait();
          float la, lb;
          unpack2(add2(l2[0], l2[1]), la, lb);
          l += la + lb;
        }
        if (ok && tile.ntok < TILE) {
          // Rows behind the tile's end hold other slots, or what the ring held
          // before (possibly NaN, which a weight of 0 would not silence): clear
          // them.  With K = V the tile's Q.K is done: its scores are there.  Last, so that
          // a V tile still on its way holds nothing up.
          const int st = v_entry<NH, SHARED>(i) % NST;
          ok = mbar_wait(SHARED ? &kfull[i & 7] : &vfull[i & 7], (i >> 3) & 1, abort_flag, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (ok) {
            uint8_t *vt = kv + st * Cfg::TB;
            const int per_box = (TILE - tile.ntok) * 8;
#pragma unroll 1
            for (int q = t128; q < per_box; q += 128)
#pragma unroll
              for (int box = 0; box < DH / 64; ++box)
                *reinterpret_cast<uint4 *>(vt + box * Cfg::BOXB + (tile.ntok + (q >> 3)) * 128 +
                                           (q & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();  // for the tensor core
          }
        }
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&pfull[sb]);
      }
      // --- the rows' output, by the group of the segment's last tile, which has the
      // final reference; the other leaves its sum in ref[] and goes on to the next
      // segment's first tile.
      const bool have_last = static_cast<int>((i - 1) & 1) == wg;
      if (!have_last) {
        if (act) {
          // (n_other counts the last tile's)
          if (ok) ok = mbar_wait(set_other, (n_other - 1) & 1, abort_flag, p.status);
          ok = __all_sync(0xffffffffu, ok);
          const float last = ok ? *ref_other : m_ref;
          take_back_ref();
          *ref_own = m_ref == -INFINITY ? 0.f : l * exp2f(m_ref - last);
          pair_arrive(1 + qd);
          lent = true;
        }
        continue;
      }
      if (act) {
        pair_sync(1 + qd);
        l += *ref_other;
        pair_arrive(5 + qd);
      }
      if (ok) ok = mbar_wait(&odone[(i - 1) & 3], ((i - 1) >> 2) & 1, abort_flag, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (act) {
        const float inv = (ok && l > 0.f) ? __fdividef(1.f, l) : 0.f;
        const bool final_rows = g.prefix_len == nullptr && seg.whole();
        // (the row's token and sequence: only own units write final rows)
        const int64_t orow =
            (static_cast<int64_t>(seg.qb * qt + tq) * g.batch + seg.b) * Hq + seg.x * g.group + h;
        const int64_t prow =
            static_cast<int64_t>(
                partial_slot(g.prefix_len != nullptr, worker, seg.unit, seg.opens)) *
                (seg.prefix ? p.rp : p.rs) + r;
        uint8_t *base =
            final_rows
                ? reinterpret_cast<uint8_t *>(p.out + orow * Cfg::D + rank * DH)
                : reinterpret_cast<uint8_t *>((seg.prefix ? p.pre_o : p.own_o) + prow * Cfg::D +
                                              rank * DH);
        // Four lanes swap 32-byte pieces so that each store of theirs is a whole line
        // of one row (stores of 32 bytes in 32 rows took 7000 cycles for 128 rows).
        uint8_t *row_base[4];
        uint32_t row_there = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          row_base[k] = reinterpret_cast<uint8_t *>(__shfl_sync(
              0xffffffffu, reinterpret_cast<uint64_t>(base), (lane & ~3) + k));
          row_there |= __shfl_sync(0xffffffffu, row_ok ? 1u : 0u, (lane & ~3) + k) << k;
        }
        if (ok) tc_fence_after();
        if (nrow <= 8 && !final_rows && ok) {
          // A few rows' pieces: no line is worth the swap, and reading 64 columns at a
          // time leaves fewer waits.
#pragma unroll 1
          for (int u = 0; u < DH / 64; ++u) {
            float o[64];
            tmem_ld64(tmem + lane_base + Cfg::O_COL + u * 64, o);
            if (u + 1 == DH / 64) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(oempty);
            }
            if (row_ok) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                uint32_t v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = __float_as_uint(o[8 * k + q] * inv);
                st_global_v8(base + u * 256 + k * 32, v);
              }
            }
          }
        } else {
          const int units = final_rows ? DH / 64 : DH / 32;  // 128-byte lines of a row
          const bool halves = final_rows && p.out_halves != 0;
#pragma unroll 1
          for (int u = 0; u < units; ++u) {
            uint32_t v[32];
            if (!ok) {
#pragma unroll
              for (int q = 0; q < 32; ++q) v[q] = 0;
            } else if (final_rows) {
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                float o[32];
                tmem_load32(tmem + lane_base + Cfg::O_COL + u * 64 + half * 32, o);
#pragma unroll
                for (int q = 0; q < 16; ++q)
                  v[16 * half + q] = pack_bf16x2(o[2 * q] * inv, o[2 * q + 1] * inv);
              }
            } else {
              float o[32];
              tmem_load32(tmem + lane_base + Cfg::O_COL + u * 32, o);
#pragma unroll
              for (int q = 0; q < 32; ++q) v[q] = __float_as_uint(o[q] * inv);
            }
            if (u + 1 == units) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(oempty);
            }
            swap_pieces(v, lane);
            if (halves) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if ((row_there >> k) & 1)
                  st_global_2v4(row_base[k] + u * 128 + (lane & 3) * 32, v + 8 * k);
              continue;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if ((row_there >> k) & 1)
                st_global_v8(row_base[k] + u * 128 + (lane & 3) * 32, v + 8 * k);
          }
        }
        const float lse2 = l > 0.f ? m_ref + log2f(l) : -INFINITY;
        if (row_ok && !seg.prefix && !final_rows) {
          // Both CTAs of a pair: the CTA that joins a cut unit's pieces has counted the
          // CTAs of its own rank, so it may read only what those wrote.
          p.own_lse[rank * p.lse_stride + prow] = lse2;
        } else if (row_ok && rank == 0) {
          if (seg.prefix)
            p.pre_lse[prow] = lse2;
          else if (p.lse != nullptr)
            p.lse[orow] = l > 0.f ? lse2 * kLn2 : -INFINITY;
        }
      } else if (lane == 0) {
        mbar_arrive(oempty);
      }
      if (p.cuts == nullptr && g.prefix_len == nullptr && !seg.whole()) {
        // A piece of a cut unit of few rows: the CTA that leaves the last one joins them
        // (a kernel behind this one took 5 us of a 20 us decode call).
        const int32_t first = seg.start + g.unit_cost;
        const int32_t cf = chunk_of(plan.total, p.workers, first);
        PartSlots at;
        cut_parts(plan.total, p.workers, cf, seg.start, g.unit_cost, seg.u.n, at);
        __threadfence();
        group_sync(9 + wg);
        if (t128 == 0) {
          uint32_t *cnt = p.counters + cf * NH + rank;
          const uint32_t old = atomic_add_acq_rel_gpu(cnt, 1);
          const bool last = old + 1 == static_cast<uint32_t>(at.n);
          if (last) *cnt = 0;
          last_piece[wg] = last ? 1 : 0;
        }
        group_sync(9 + wg);
        if (last_piece[wg] != 0) {
#pragma unroll 1
          for (int32_t row = qd; row < nrow; row += 4) {
            const int32_t rq = row / g.group, rh = row - rq * g.group;
            const int64_t to = (static_cast<int64_t>(seg.qb * g.qt_seq + rq) * g.batch + seg.b) * Hq +
                               seg.x * g.group + rh;
            join_pieces<Cfg::D>(p.own_o + rank * DH, p.own_lse + rank * p.lse_stride, at, p.rs, row,
                                p.out + to * Cfg::D + rank * DH,
                                p.lse != nullptr && rank == 0 ? p.lse + to : nullptr);
          }
        }
      }
    }
    take_back_ref();
  }

  tc_fence_before();
  __syncthreads();
  if (NH == 2) cluster_sync();  // neither CTA leaves while the other may write into it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::TMEM_COLS);
  }
}

}  // namespace gdattn
