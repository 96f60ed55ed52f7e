// C ABI of the continuous-batching operators (declared in include/gdattn.h):
// attention with pinned first tokens, attention over a shared prefix, slot maps
// and cache writes.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "gdattn.h"

#include "../host_common.h"
#include "cache_rows.cuh"
#include "rows_plan.cuh"
#include "simple_rows.cuh"

using namespace gdattn;

namespace {

constexpr int32_t kMaxRowsTokens = 1 << 20;
constexpr int32_t kMaxGroup = 128;  // query heads per KV head: one block of query rows

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// What both attention entry points check on the host (the workspace aside).
gdattn_status check_rows_args(const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *seqlens, int32_t batch, int32_t n_tokens,
                              int32_t max_seqlen, const gdattn_layer_desc *desc, int32_t n_sink,
                              const void *out, const float *lse) {
  if (q == nullptr || k_cache == nullptr || seqlens == nullptr || out == nullptr ||
      desc == nullptr)
    return GDATTN_ERR_INVALID_ARG;
  gdattn_status st = check_desc(desc);
  if (st != GDATTN_OK) return st;
  if ((desc->kv_shared == 1) != (v_cache == nullptr)) return GDATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || (v_cache && !aligned16(v_cache)) ||
      !aligned16(out) || !aligned4(seqlens) || !aligned4(lse))
    return GDATTN_ERR_MISALIGNED;
  (void)batch, (void)n_tokens, (void)max_seqlen, (void)n_sink;
  return GDATTN_OK;
}

// Shape checks, shared with the workspace queries.
gdattn_status check_rows_shape(int32_t batch, int32_t n_tokens, int32_t max_seqlen,
                               const gdattn_layer_desc *desc, int32_t n_sink) {
  gdattn_status st = check_desc(desc);
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

gdattn_status enqueue_rows(const void *q, const void *k_prefix, const void *v_prefix,
                           const int32_t *prefix_len, int32_t prefix_rows, const void *k_cache,
                           const void *v_cache, const int32_t *seqlens, int32_t batch,
                           int32_t n_tokens, const gdattn_layer_desc *desc, int32_t n_sink,
                           void *out, float *lse, void *workspace, cudaStream_t stream) {
  const float log2e = 1.4426950408889634f;
  SimpleRowsParams p = {};
  p.g.seqlens = seqlens;
  p.g.prefix_len = prefix_len;
  p.g.batch = batch;
  p.g.tokens = n_tokens;
  p.g.n_kv_heads = desc->n_kv_heads;
  p.g.group = desc->n_q_heads / desc->n_kv_heads;
  p.g.window = desc->window;
  p.g.sinks = n_sink;
  p.g.capacity = desc->cache_capacity;
  p.g.prefix_rows = prefix_rows;
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k_cache);
  p.v = static_cast<const uint16_t *>(v_cache ? v_cache : k_cache);
  p.pk = static_cast<const uint16_t *>(k_prefix);
  p.pv = static_cast<const uint16_t *>(v_prefix ? v_prefix : k_prefix);
  p.batch_stride = desc->cache_batch_stride != 0 ? desc->cache_batch_stride
                                                 : static_cast<int64_t>(desc->cache_capacity) *
                                                       desc->n_kv_heads * desc->head_dim;
  p.out = static_cast<uint16_t *>(out);
  p.lse = lse;
  p.status = static_cast<uint32_t *>(workspace);
  p.qscale = desc->softcap > 0.f ? desc->scale / desc->softcap : desc->scale * log2e;
  p.post = desc->softcap > 0.f ? desc->softcap * log2e : 0.f;
  if (desc->n_q_heads > 65535) return GDATTN_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(batch) * n_tokens, desc->n_q_heads);
  if (desc->head_dim == 256)
    simple_rows_kernel<256><<<grid, 32 * kSimpleWarps, 0, stream>>>(p);
  else
    simple_rows_kernel<512><<<grid, 32 * kSimpleWarps, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? GDATTN_OK : GDATTN_ERR_CUDA;
}

gdattn_status check_write_args(const void *k_rows, const void *v_rows, int64_t row_stride,
                               const int32_t *row_seq, const int32_t *row_slot, int32_t n_rows,
                               int32_t batch, const gdattn_layer_desc *desc, const void *k_cache,
                               const void *v_cache) {
  if (desc == nullptr || k_cache == nullptr || k_rows == nullptr || row_seq == nullptr ||
      row_slot == nullptr)
    return GDATTN_ERR_INVALID_ARG;
  gdattn_status st = check_desc(desc);
  if (st != GDATTN_OK) return st;
  if ((desc->kv_shared == 1) != (v_cache == nullptr) ||
      (desc->kv_shared == 1) != (v_rows == nullptr))
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
  p.rows[0] = static_cast<const uint16_t *>(k_rows);
  p.rows[1] = static_cast<const uint16_t *>(v_rows);
  p.cache[0] = static_cast<uint8_t *>(k_cache);
  p.cache[1] = static_cast<uint8_t *>(v_cache);
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

unsigned write_grid(int64_t items, int64_t per_cta) {
  const int64_t n = (items + per_cta - 1) / per_cta;
  return static_cast<unsigned>(n < 1 ? 1 : (n < 148 * 16 ? n : 148 * 16));
}

}  // namespace

extern "C" {

size_t gdattn_sink_workspace_size(int32_t batch, int32_t n_tokens, int32_t max_seqlen,
                                  const gdattn_layer_desc *desc, int32_t n_sink) {
  if (check_rows_shape(batch, n_tokens, max_seqlen, desc, n_sink) != GDATTN_OK ||
      desc->window == 0)
    return 0;
  return kHeaderBytes;
}

gdattn_status gdattn_decode_sink(const void *q, const void *k_cache, const void *v_cache,
                                 const int32_t *seqlens, int32_t batch, int32_t n_tokens,
                                 int32_t max_seqlen, const gdattn_layer_desc *desc,
                                 int32_t n_sink, void *out, float *lse, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  gdattn_status st = check_rows_args(q, k_cache, v_cache, seqlens, batch, n_tokens, max_seqlen,
                                     desc, n_sink, out, lse);
  if (st != GDATTN_OK) return st;
  st = check_rows_shape(batch, n_tokens, max_seqlen, desc, n_sink);
  if (st != GDATTN_OK) return st;
  if (desc->window == 0) return GDATTN_ERR_INVALID_ARG;
  if (workspace == nullptr) return GDATTN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return GDATTN_ERR_MISALIGNED;
  if (workspace_bytes < kHeaderBytes) return GDATTN_ERR_WORKSPACE;
  return enqueue_rows(q, nullptr, nullptr, nullptr, 0, k_cache, v_cache, seqlens, batch, n_tokens,
                      desc, n_sink, out, lse, workspace, static_cast<cudaStream_t>(stream));
}

size_t gdattn_prefix_workspace_size(int32_t batch, int32_t n_tokens, int32_t max_seqlen,
                                    int32_t prefix_rows, const gdattn_layer_desc *desc) {
  if (check_rows_shape(batch, n_tokens, max_seqlen, desc, 0) != GDATTN_OK || prefix_rows < 1)
    return 0;
  return kHeaderBytes;
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
  gdattn_status st = check_rows_args(q, k_cache, v_cache, seqlens, batch, n_tokens, max_seqlen,
                                     desc, 0, out, lse);
  if (st != GDATTN_OK) return st;
  if ((desc->kv_shared == 1) != (v_prefix == nullptr)) return GDATTN_ERR_INVALID_ARG;
  st = check_rows_shape(batch, n_tokens, max_seqlen, desc, 0);
  if (st != GDATTN_OK) return st;
  if (!aligned16(k_prefix) || !aligned16(v_prefix) || !aligned4(prefix_len))
    return GDATTN_ERR_MISALIGNED;
  if (workspace == nullptr) return GDATTN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return GDATTN_ERR_MISALIGNED;
  if (workspace_bytes < kHeaderBytes) return GDATTN_ERR_WORKSPACE;
  return enqueue_rows(q, k_prefix, v_prefix, prefix_len, prefix_rows, k_cache, v_cache, seqlens,
                      batch, n_tokens, desc, 0, out, lse, workspace,
                      static_cast<cudaStream_t>(stream));
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
  const dim3 grid(write_grid(static_cast<int64_t>(n_rows) * desc->n_kv_heads * desc->head_dim / 8,
                             kCacheWriteThreads),
                  v_rows ? 2 : 1);
  cache_write_kernel<<<grid, kCacheWriteThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
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
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  const dim3 grid(write_grid(static_cast<int64_t>(n_rows) * desc->n_kv_heads,
                             kCacheWriteThreads / 32),
                  v_rows ? 2 : 1);
  if (desc->head_dim == 256)
    cache_write_fp8_kernel<256>
        <<<grid, kCacheWriteThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  else
    cache_write_fp8_kernel<512>
        <<<grid, kCacheWriteThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? GDATTN_OK : GDATTN_ERR_CUDA;
}

}  // extern "C"
