// C ABI of the continuous-batching operators (declared in include/gdattn.h):
// attention with pinned first tokens, attention over a shared prefix, slot maps
// and cache writes.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <mutex>

#include "gdattn.h"

#include "../host_common.h"
#include "cache_rows.cuh"
#include "rows_attn.cuh"
#include "rows_merge.cuh"

using namespace gdattn;

namespace {

constexpr int32_t kMaxRowsTokens = 1 << 20;
constexpr int32_t kMaxGroup = 128;  // query heads per KV head: one block of query rows

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// What both attention entry points check of the pointers (the workspace aside).
gdattn_status check_rows_args(const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *seqlens, const gdattn_layer_desc *desc,
                              const void *out, const float *lse) {
  if (q == nullptr || k_cache == nullptr || seqlens == nullptr || out == nullptr ||
      desc == nullptr)
    return GDATTN_ERR_INVALID_ARG;
  const gdattn_status st = check_desc(desc);
  if (st != GDATTN_OK) return st;
  if ((desc->kv_shared == 1) != (v_cache == nullptr)) return GDATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned4(seqlens) || !aligned4(lse))
    return GDATTN_ERR_MISALIGNED;
  return GDATTN_OK;
}

// What they check of the shape, shared with the workspace queries.
gdattn_status check_rows_shape(int32_t batch, int32_t n_tokens, int32_t max_seqlen,
                               const gdattn_layer_desc *desc, int32_t n_sink) {
  const gdattn_status st = check_desc(desc);
  if (st != GDATTN_OK) return st;
  if (batch <= 0 || max_seqlen <= 0 || n_tokens < 1 || n_tokens > kMaxRowsTokens ||
      n_tokens > max_seqlen || n_sink < 0 || n_sink >= desc->cache_capacity)
    return GDATTN_ERR_INVALID_ARG;
  // The first token's window must still be in the ring, unless it never wraps.
  if (desc->window > 0 && desc->cache_capacity < max_seqlen &&
      static_cast<int64_t>(desc->cache_capacity) - n_sink <
          static_cast<int64_t>(desc->window) + n_tokens - 1)
    return GDATTN_ERR_INVALID_ARG;
  if ((desc->head_dim != 256 && desc->head_dim != 512) ||
      desc->n_q_heads / desc->n_kv_heads > kMaxGroup)
    return GDATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(batch) * n_tokens * desc->n_q_heads > INT32_MAX)
    return GDATTN_ERR_UNSUPPORTED;
  return GDATTN_OK;
}

// ------------------------------------------------------------- row kernels
using RowsFn = void (*)(RowsMaps, RowsParams);

RowsFn rows_kernel(const gdattn_layer_desc *d) {
  static const RowsFn fns[2][2][2] = {
      {{rows_attn_kernel<1, false, false>, rows_attn_kernel<1, false, true>},
       {rows_attn_kernel<1, true, false>, rows_attn_kernel<1, true, true>}},
      {{rows_attn_kernel<2, false, false>, rows_attn_kernel<2, false, true>},
       {rows_attn_kernel<2, true, false>, rows_attn_kernel<2, true, true>}}};
  return fns[d->head_dim / 256 - 1][d->kv_shared][d->softcap > 0.f ? 1 : 0];
}

cudaLaunchConfig_t rows_launch(int nh, int workers, cudaStream_t stream,
                               cudaLaunchAttribute (&attr)[2]) {
  const int smem = nh == 1 ? RowsConfig<1>::SMEM : RowsConfig<2>::SMEM;
  cudaLaunchConfig_t cfg =
      launch_config(dim3(static_cast<unsigned>(workers * nh)), RowsConfig<1>::kThreads, smem,
                    stream, attr);
  if (nh == 2) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cfg;
}

// CTAs (or CTA pairs) of the geometry's kernel that the current device holds at
// once, and its SMs; also sets the kernel's shared-memory limit.  Found once per context:
// the limit belongs to it.
struct DeviceRoom {
  int workers, sms;
};

DeviceRoom device_room(const gdattn_layer_desc *d) {
  constexpr int kDevices = 64;
  struct Entry {
    unsigned long long ctx_id;
    DeviceRoom room;
  };
  static std::mutex mu;
  static Entry known[kDevices][2][2][2] = {};
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return {};
  const int nh = d->head_dim / 256;
  Entry &e = known[dev][nh - 1][d->kv_shared][d->softcap > 0.f ? 1 : 0];
  const unsigned long long ctx_id = current_context_id();  // 0: there is none yet
  std::lock_guard<std::mutex> lock(mu);
  if (ctx_id != 0 && e.ctx_id == ctx_id) return e.room;
  const void *fn = reinterpret_cast<const void *>(rows_kernel(d));
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           nh == 1 ? RowsConfig<1>::SMEM : RowsConfig<2>::SMEM) != cudaSuccess)
    return {};
  // The merge runs between row kernels: with the same split of L1 and shared memory the
  // SMs need no reconfiguration, which each way waits for an idle SM.
  const void *merges[2] = {nh == 1 ? reinterpret_cast<const void *>(merge_cut_units_kernel<256>)
                                   : reinterpret_cast<const void *>(merge_cut_units_kernel<512>),
                           nh == 1 ? reinterpret_cast<const void *>(merge_prefix_kernel<256>)
                                   : reinterpret_cast<const void *>(merge_prefix_kernel<512>)};
  for (const void *m : merges)
    if (cudaFuncSetAttribute(m, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess)
      return {};
  DeviceRoom got = {0, sm_count()};
  if (nh == 1) {
    got.workers = got.sms;
  } else {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = rows_launch(nh, got.sms / 2, nullptr, attr);
    if (cudaOccupancyMaxActiveClusters(&got.workers, fn, &cfg) != cudaSuccess) return {};
  }
  if (got.workers > 0) e = {ctx_id != 0 ? ctx_id : current_context_id(), got};
  return got;
}

struct RowsLayout {
  RowsGeom g = {};
  int nh = 1, workers = 0, sms = 0;
  int32_t rs = 0, rp = 0;
  int64_t lse_stride = 0;
  size_t table = 0, own_o = 0, own_lse = 0, pre_o = 0, pre_lse = 0, bytes = 0;
};

// Blocks, workers and workspace of a call (prefix_rows 0: a call without a prefix).
gdattn_status plan_layout(int32_t batch, int32_t n_tokens, const gdattn_layer_desc *d,
                          int32_t n_sink, int32_t prefix_rows, RowsLayout &lay) {
  RowsGeom &g = lay.g;
  g.batch = batch;
  g.tokens = n_tokens;
  g.n_kv_heads = d->n_kv_heads;
  g.group = d->n_q_heads / d->n_kv_heads;
  g.window = d->window;
  g.sinks = n_sink;
  g.capacity = d->cache_capacity;
  g.prefix_rows = prefix_rows;
  const int32_t per_block = RowsConfig<1>::M / g.group;  // tokens of a full block
  g.qt_seq = n_tokens < per_block ? n_tokens : per_block;
  g.nqb = (n_tokens + g.qt_seq - 1) / g.qt_seq;
  const int32_t pairs = batch * n_tokens;
  g.qt_pre = pairs < per_block ? pairs : per_block;
  g.npb = (pairs + g.qt_pre - 1) / g.qt_pre;
  lay.rs = g.qt_seq * g.group;
  // What a unit costs besides its tiles, in tiles.  Full blocks: three (one: prompt of
  // 8192 tokens 307 us, three: 278; 512 question tokens 364 and 328).  A few rows: two
  // (decode at batch 8 23.7 -> 22.8 us), or one where every piece goes to the merge anyway
  // (4 sequences behind a prefix 23.4 -> 22.6).
  g.unit_cost = lay.rs > 32 ? 3 : prefix_rows > 0 ? 1 : 2;
  lay.rp = g.qt_pre * g.group;
  const int64_t own_units = static_cast<int64_t>(batch) * g.nqb * g.n_kv_heads;
  // The kernels count steps in 32 bits.
  const int64_t reach = static_cast<int64_t>(d->window) + g.qt_seq + n_sink;  // of a block
  const int64_t own_rows_most =
      d->window > 0 && reach < d->cache_capacity ? reach : d->cache_capacity;
  const int64_t most_steps =
      own_units * (own_rows_most / kRowTile + 4 + g.unit_cost) +
      (prefix_rows > 0 ? static_cast<int64_t>(g.npb) * g.n_kv_heads *
                             (prefix_rows / kRowTile + 1 + g.unit_cost)
                       : 0);
  if (most_steps > INT32_MAX) return GDATTN_ERR_UNSUPPORTED;
  const DeviceRoom room = device_room(d);
  const int most = room.workers;
  if (most <= 0) return GDATTN_ERR_CUDA;
  lay.sms = room.sms;
  lay.nh = d->head_dim / 256;
  lay.workers = d->split_ctas > 0 && d->split_ctas < most ? d->split_ctas : most;
  const int64_t own_slots = prefix_rows > 0 ? lay.workers + own_units : 2 * lay.workers;
  const int64_t pre_slots =
      prefix_rows > 0 ? lay.workers + static_cast<int64_t>(g.npb) * g.n_kv_heads : 0;
  if (own_slots > INT32_MAX || pre_slots > INT32_MAX) return GDATTN_ERR_UNSUPPORTED;
  const size_t own_rows = static_cast<size_t>(own_slots) * lay.rs;
  const size_t pre_rows = static_cast<size_t>(pre_slots) * lay.rp;
  // Behind the header: what the row kernel tells the merge.
  lay.table = kHeaderBytes;
  const size_t table_bytes =
      prefix_rows > 0 ? 256 + (static_cast<size_t>(batch) * g.nqb + 1) * sizeof(int32_t)
                      : static_cast<size_t>(lay.workers) * sizeof(CutEntry);
  lay.own_lse = align256(lay.table + table_bytes);
  lay.lse_stride = static_cast<int64_t>(own_rows);
  lay.pre_lse = align256(lay.own_lse + lay.nh * own_rows * 4);
  lay.own_o = align256(lay.pre_lse + pre_rows * 4);
  lay.pre_o = align256(lay.own_o + own_rows * d->head_dim * 4);
  // The row kernel stores 32 bytes at a time, and a workspace may start between two
  // 32-byte boundaries: room to move own_o and pre_o up to the next.
  lay.bytes = align256(lay.pre_o + pre_rows * d->head_dim * 4 + 16);
  return GDATTN_OK;
}

template <int D>
cudaError_t launch_merge(const RowsLayout &lay, const RowsParams &p, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  const int rows_per_cta = kMergeWarps / p.merge_shares;  // of a CTA
  if (lay.g.prefix_len != nullptr) {
    const int64_t rows =
        static_cast<int64_t>(lay.g.batch) * lay.g.tokens * lay.g.n_kv_heads * lay.g.group;
    cudaLaunchConfig_t cfg = launch_config(dim3(static_cast<unsigned>((rows + rows_per_cta - 1) / rows_per_cta)),
                                           kMergeThreads, 0, stream, attr);
    return cudaLaunchKernelEx(&cfg, merge_prefix_kernel<D>, p);
  }
  if (lay.workers == 1) return cudaSuccess;  // no boundary
  cudaLaunchConfig_t cfg =
      launch_config(dim3(static_cast<unsigned>(lay.workers - 1),
                         static_cast<unsigned>((lay.rs + rows_per_cta - 1) / rows_per_cta)),
                    kMergeThreads, 0, stream, attr);
  return cudaLaunchKernelEx(&cfg, merge_cut_units_kernel<D>, p);
}

gdattn_status enqueue_rows(RowsLayout &lay, const void *q, const void *k_prefix,
                           const void *v_prefix, const int32_t *prefix_len, const void *k_cache,
                           const void *v_cache, const int32_t *seqlens,
                           const gdattn_layer_desc *desc, void *out, float *lse, uint8_t *ws,
                           cudaStream_t stream) {
  RowsGeom &g = lay.g;
  g.seqlens = seqlens;
  g.prefix_len = prefix_len;
  const int32_t D = desc->head_dim, Hkv = desc->n_kv_heads, Hq = desc->n_q_heads;
  const int64_t bstride = desc->cache_batch_stride != 0
                              ? desc->cache_batch_stride
                              : static_cast<int64_t>(desc->cache_capacity) * Hkv * D;
  EncodeTiledFn enc = encode_tiled();
  if (enc == nullptr) return GDATTN_ERR_CUDA;
  RowsMaps m = {};
  bool ok = true;
  auto cache = [&](CUtensorMap *full, CUtensorMap *part, const void *base, int32_t rows,
                   int32_t batch, int64_t stride) {
    if (base == nullptr) return;
    ok = ok && encode_cache_map(enc, full, base, D, Hkv, rows, batch, stride, kRowTile) &&
         encode_cache_map(enc, part, base, D, Hkv, rows, batch, stride, 16);
  };
  cache(&m.k, &m.k16, k_cache, g.capacity, g.batch, bstride);
  cache(&m.v, &m.v16, v_cache, g.capacity, g.batch, bstride);
  const int64_t pstride = static_cast<int64_t>(g.prefix_rows) * Hkv * D;
  cache(&m.pk, &m.pk16, k_prefix, g.prefix_rows, 1, pstride);
  cache(&m.pv, &m.pv16, v_prefix, g.prefix_rows, 1, pstride);
  ok = ok && encode_q_tokens_map(enc, &m.q_own, q, D, static_cast<int64_t>(g.batch) * Hq,
                                 g.tokens, g.qt_seq, g.group);
  if (prefix_len != nullptr)
    ok = ok && encode_q_tokens_map(enc, &m.q_pre, q, D, Hq, g.tokens * g.batch, g.qt_pre, g.group);
  if (!ok) return GDATTN_ERR_CUDA;
  RowsParams p = {};
  p.g = g;
  p.out = static_cast<uint16_t *>(out);
  p.out_halves = (reinterpret_cast<uintptr_t>(out) & 31u) != 0 ? 1 : 0;
  p.lse = lse;
  const size_t up = (0 - reinterpret_cast<uintptr_t>(ws)) & 31u;  // 0 or 16
  p.own_o = reinterpret_cast<float *>(ws + lay.own_o + up);
  p.own_lse = reinterpret_cast<float *>(ws + lay.own_lse);
  p.lse_stride = lay.lse_stride;
  p.pre_o = reinterpret_cast<float *>(ws + lay.pre_o + up);
  p.pre_lse = reinterpret_cast<float *>(ws + lay.pre_lse);
  // A block of few rows is joined by the row kernel itself; with more rows the four warps
  // that would do it take longer than a kernel with a warp for each.
  const bool join_here = prefix_len == nullptr && lay.rs <= 16;
  p.cuts = join_here ? nullptr : reinterpret_cast<CutEntry *>(ws + lay.table);
  p.counters = reinterpret_cast<uint32_t *>(ws + kOffCounters);
  p.prefix_entry = reinterpret_cast<PrefixEntry *>(ws + lay.table);
  p.pair_start = reinterpret_cast<int32_t *>(ws + lay.table + 256);
  p.status = reinterpret_cast<uint32_t *>(ws);
  p.workers = lay.workers;
  p.rs = lay.rs;
  p.rp = lay.rp;
  const int32_t rows = prefix_len != nullptr && lay.rp > lay.rs ? lay.rp : lay.rs;
  p.q_stride = (rows + 7) / 8 * 1024;
  p.q_bufs = 2 * 4 * p.q_stride <= RowsConfig<1>::QB ? 2 : 1;
  p.q_bytes_own = lay.rs * 128;
  p.q_bytes_pre = lay.rp * 128;
  const float log2e = 1.4426950408889634f;
  p.qscale = desc->softcap > 0.f ? desc->scale / desc->softcap : desc->scale * log2e;
  p.post = desc->softcap > 0.f ? desc->softcap * log2e : 0.f;
  p.test_withhold = (desc->flags & GDATTN_FLAG_TEST_WITHHOLD_KV) ? 1 : 0;
  // Warps per row of the merge: enough to fill the SMs twice over, where the rows do not.
  const int64_t merge_rows = prefix_len != nullptr
                                 ? static_cast<int64_t>(g.batch) * g.tokens * Hq
                                 : static_cast<int64_t>(lay.workers) * lay.rs;
  p.merge_shares = 1;
  while (p.merge_shares < kMergeWarps &&
         merge_rows * p.merge_shares < static_cast<int64_t>(lay.sms) * 2 * kMergeWarps)
    p.merge_shares *= 2;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = rows_launch(lay.nh, lay.workers, stream, attr);
  if (cudaLaunchKernelEx(&cfg, rows_kernel(desc), m, p) != cudaSuccess) return GDATTN_ERR_CUDA;
  if (join_here) return GDATTN_OK;
  const cudaError_t e =
      lay.nh == 1 ? launch_merge<256>(lay, p, stream) : launch_merge<512>(lay, p, stream);
  return e == cudaSuccess ? GDATTN_OK : GDATTN_ERR_CUDA;
}

gdattn_status check_write_args(const void *k_rows, const void *v_rows, int64_t row_stride,
                               const int32_t *row_seq, const int32_t *row_slot, int32_t n_rows,
                               int32_t batch, const gdattn_layer_desc *desc, const void *k_cache,
                               const void *v_cache) {
  if (desc == nullptr || k_cache == nullptr) return GDATTN_ERR_INVALID_ARG;
  gdattn_status st = check_desc(desc);
  if (st != GDATTN_OK) return st;
  if ((desc->kv_shared == 1) != (v_cache == nullptr)) return GDATTN_ERR_INVALID_ARG;
  // Without rows there is nothing to point at.
  if (n_rows != 0 && (k_rows == nullptr || row_seq == nullptr || row_slot == nullptr ||
                      (desc->kv_shared == 1) != (v_rows == nullptr)))
    return GDATTN_ERR_INVALID_ARG;
  if (n_rows < 0 || batch <= 0 ||
      row_stride < static_cast<int64_t>(desc->n_kv_heads) * desc->head_dim || row_stride % 8 != 0)
    return GDATTN_ERR_INVALID_ARG;
  if (desc->head_dim != 256 && desc->head_dim != 512) return GDATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(desc->n_kv_heads) * desc->head_dim > INT32_MAX)
    return GDATTN_ERR_UNSUPPORTED;
  if (!aligned16(k_rows) || !aligned16(v_rows) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned4(row_seq) || !aligned4(row_slot))
    return GDATTN_ERR_MISALIGNED;
  return GDATTN_OK;
}

CacheWriteParams write_params(const void *k_rows, const void *v_rows, int64_t row_stride,
                              const int32_t *row_seq, const int32_t *row_slot, int32_t n_rows,
                              int32_t batch, const gdattn_layer_desc *desc, void *k_cache,
                              void *v_cache) {
  CacheWriteParams p = {};
  p.k_rows = static_cast<const uint16_t *>(k_rows);
  p.v_rows = static_cast<const uint16_t *>(v_rows);
  p.k_cache = static_cast<uint8_t *>(k_cache);
  p.v_cache = static_cast<uint8_t *>(v_cache);
  p.row_seq = row_seq;
  p.row_slot = row_slot;
  p.row_stride = row_stride;
  p.batch_stride = desc->cache_batch_stride != 0 ? desc->cache_batch_stride
                                                 : static_cast<int64_t>(desc->cache_capacity) *
                                                       desc->n_kv_heads * desc->head_dim;
  p.n_rows = n_rows;
  p.batch = batch;
  p.capacity = desc->cache_capacity;
  p.n_kv_heads = desc->n_kv_heads;
  p.head_dim = desc->head_dim;
  return p;
}

}  // namespace

extern "C" {

size_t gdattn_sink_workspace_size(int32_t batch, int32_t n_tokens, int32_t max_seqlen,
                                  const gdattn_layer_desc *desc, int32_t n_sink) {
  if (check_rows_shape(batch, n_tokens, max_seqlen, desc, n_sink) != GDATTN_OK ||
      desc->window == 0)
    return 0;
  RowsLayout lay;
  return plan_layout(batch, n_tokens, desc, n_sink, 0, lay) == GDATTN_OK ? lay.bytes : 0;
}

gdattn_status gdattn_decode_sink(const void *q, const void *k_cache, const void *v_cache,
                                 const int32_t *seqlens, int32_t batch, int32_t n_tokens,
                                 int32_t max_seqlen, const gdattn_layer_desc *desc,
                                 int32_t n_sink, void *out, float *lse, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  gdattn_status st = check_rows_args(q, k_cache, v_cache, seqlens, desc, out, lse);
  if (st != GDATTN_OK) return st;
  st = check_rows_shape(batch, n_tokens, max_seqlen, desc, n_sink);
  if (st != GDATTN_OK) return st;
  if (desc->window == 0) return GDATTN_ERR_INVALID_ARG;
  if (workspace == nullptr) return GDATTN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return GDATTN_ERR_MISALIGNED;
  RowsLayout lay;
  st = plan_layout(batch, n_tokens, desc, n_sink, 0, lay);
  if (st != GDATTN_OK) return st;
  if (workspace_bytes < lay.bytes) return GDATTN_ERR_WORKSPACE;
  return enqueue_rows(lay, q, nullptr, nullptr, nullptr, k_cache, v_cache, seqlens, desc, out, lse,
                      static_cast<uint8_t *>(workspace), static_cast<cudaStream_t>(stream));
}

size_t gdattn_prefix_workspace_size(int32_t batch, int32_t n_tokens, int32_t max_seqlen,
                                    int32_t prefix_rows, const gdattn_layer_desc *desc) {
  if (check_rows_shape(batch, n_tokens, max_seqlen, desc, 0) != GDATTN_OK || prefix_rows < 1)
    return 0;
  RowsLayout lay;
  return plan_layout(batch, n_tokens, desc, 0, prefix_rows, lay) == GDATTN_OK ? lay.bytes : 0;
}

gdattn_status gdattn_decode_prefix(const void *q, const void *k_prefix, const void *v_prefix,
                                   const int32_t *prefix_len, int32_t prefix_rows,
                                   const void *k_cache, const void *v_cache,
                                   const int32_t *seqlens, int32_t batch, int32_t n_tokens,
                                   int32_t max_seqlen, const gdattn_layer_desc *desc, void *out,
                                   float *lse, void *workspace, size_t workspace_bytes,
                                   void *stream) {
  if (k_prefix == nullptr || prefix_len == nullptr || prefix_rows < 1)
    return GDATTN_ERR_INVALID_ARG;
  gdattn_status st = check_rows_args(q, k_cache, v_cache, seqlens, desc, out, lse);
  if (st != GDATTN_OK) return st;
  if ((desc->kv_shared == 1) != (v_prefix == nullptr)) return GDATTN_ERR_INVALID_ARG;
  st = check_rows_shape(batch, n_tokens, max_seqlen, desc, 0);
  if (st != GDATTN_OK) return st;
  if (!aligned16(k_prefix) || !aligned16(v_prefix) || !aligned4(prefix_len))
    return GDATTN_ERR_MISALIGNED;
  if (workspace == nullptr) return GDATTN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return GDATTN_ERR_MISALIGNED;
  RowsLayout lay;
  st = plan_layout(batch, n_tokens, desc, 0, prefix_rows, lay);
  if (st != GDATTN_OK) return st;
  if (workspace_bytes < lay.bytes) return GDATTN_ERR_WORKSPACE;
  return enqueue_rows(lay, q, k_prefix, v_prefix, prefix_len, k_cache, v_cache, seqlens, desc, out,
                      lse, static_cast<uint8_t *>(workspace), static_cast<cudaStream_t>(stream));
}

gdattn_status gdattn_slot_map(const int32_t *seqlens, const int32_t *new_lens, int32_t batch,
                              int32_t n_rows, int32_t cache_capacity, int32_t n_sink,
                              int32_t *row_start, int32_t *row_seq, int32_t *row_pos,
                              int32_t *row_slot, void *stream) {
  if (seqlens == nullptr || new_lens == nullptr || row_start == nullptr || batch <= 0 ||
      n_rows < 0 || cache_capacity <= 0 || n_sink < 0 || n_sink >= cache_capacity)
    return GDATTN_ERR_INVALID_ARG;
  if (n_rows > 0 && (row_seq == nullptr || row_pos == nullptr || row_slot == nullptr))
    return GDATTN_ERR_INVALID_ARG;
  if (!aligned4(seqlens) || !aligned4(new_lens) || !aligned4(row_start) || !aligned4(row_seq) ||
      !aligned4(row_pos) || !aligned4(row_slot))
    return GDATTN_ERR_MISALIGNED;
  const SlotMapParams p = {seqlens, new_lens, row_start,      row_seq, row_pos,
                           row_slot, batch,   n_rows, cache_capacity, n_sink};
  const unsigned grid =
      n_rows > 0 ? static_cast<unsigned>((static_cast<int64_t>(n_rows) + kSlotMapRows - 1) /
                                         kSlotMapRows)
                 : 1u;
  slot_map_kernel<<<grid, kSlotMapThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? GDATTN_OK : GDATTN_ERR_CUDA;
}

gdattn_status gdattn_cache_write(const void *k_rows, const void *v_rows, int64_t row_stride,
                                 const int32_t *row_seq, const int32_t *row_slot, int32_t n_rows,
                                 int32_t batch, const gdattn_layer_desc *desc, void *k_cache,
                                 void *v_cache, void *stream) {
  const gdattn_status st = check_write_args(k_rows, v_rows, row_stride, row_seq, row_slot, n_rows,
                                            batch, desc, k_cache, v_cache);
  if (st != GDATTN_OK) return st;
  if (n_rows == 0) return GDATTN_OK;
  const CacheWriteParams p = write_params(k_rows, v_rows, row_stride, row_seq, row_slot, n_rows,
                                          batch, desc, k_cache, v_cache);
  const int64_t pieces = static_cast<int64_t>(n_rows) * desc->n_kv_heads * desc->head_dim / 8;
  const int64_t grid = ceil_div(pieces, kCacheWriteThreads * kCacheWritePieces);
  if (grid > INT32_MAX) return GDATTN_ERR_UNSUPPORTED;
  cache_write_kernel<<<static_cast<unsigned>(grid), kCacheWriteThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? GDATTN_OK : GDATTN_ERR_CUDA;
}

gdattn_status gdattn_cache_write_fp8(const void *k_rows, const void *v_rows, int64_t row_stride,
                                     const int32_t *row_seq, const int32_t *row_slot,
                                     int32_t n_rows, int32_t batch, const gdattn_layer_desc *desc,
                                     void *k_codes, void *v_codes, float *k_scale, float *v_scale,
                                     void *stream) {
  const gdattn_status st = check_write_args(k_rows, v_rows, row_stride, row_seq, row_slot, n_rows,
                                            batch, desc, k_codes, v_codes);
  if (st != GDATTN_OK) return st;
  if (k_scale == nullptr || (desc->kv_shared == 1) != (v_scale == nullptr))
    return GDATTN_ERR_INVALID_ARG;
  if (!aligned4(k_scale) || !aligned4(v_scale) || desc->cache_batch_stride % 16 != 0)
    return GDATTN_ERR_MISALIGNED;
  if (n_rows == 0) return GDATTN_OK;
  CacheWriteParams p = write_params(k_rows, v_rows, row_stride, row_seq, row_slot, n_rows, batch,
                                    desc, k_codes, v_codes);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  const int64_t ctas = ceil_div(static_cast<int64_t>(n_rows) * desc->n_kv_heads,
                                kCacheWriteThreads / (desc->head_dim / 32));
  if (ctas > INT32_MAX) return GDATTN_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(ctas), v_rows ? 2 : 1);
  if (desc->head_dim == 256)
    cache_write_fp8_kernel<256>
        <<<grid, kCacheWriteThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  else
    cache_write_fp8_kernel<512>
        <<<grid, kCacheWriteThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? GDATTN_OK : GDATTN_ERR_CUDA;
}

}  // extern "C"
