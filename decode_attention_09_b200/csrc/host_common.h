// Host-side pieces that the library's translation units share: the workspace
// header's layout, argument checks, launch attributes and tensor-map encoding.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "gdattn.h"

namespace gdattn {

constexpr size_t kStatusBytes = 256;
// Every workspace starts with the same header, whatever the plan: the status
// word, then one part counter and one epoch per unit index below kMaxUnits.
// Counters must read zero and epochs must hold the last call's tag when a call
// starts; with fixed offsets no plan's partials ever land on them, so calls
// with different plans (geometry, batch, split) can take turns on one
// workspace.  A plan with more units is refused.
constexpr int64_t kMaxUnits = 16384;
constexpr size_t kOffCounters = kStatusBytes;
constexpr size_t kOffEpochs = kOffCounters + 4 * kMaxUnits;
constexpr size_t kHeaderBytes = kOffEpochs + 4 * kMaxUnits;
static_assert(kHeaderBytes % 256 == 0, "partials start 256-byte aligned");

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

// Process-unique id of the current CUDA context (cuCtxGetId), so that a
// context created after a reset is never mistaken for its predecessor even if
// it reuses the handle.  0 when the driver cannot say.
inline unsigned long long current_context_id() {
  using CtxGetCurrentFn = CUresult (*)(CUcontext *);
  using CtxGetIdFn = CUresult (*)(CUcontext, unsigned long long *);
  static CtxGetCurrentFn get_current = []() -> CtxGetCurrentFn {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<CtxGetCurrentFn>(p);
  }();
  static CtxGetIdFn get_id = []() -> CtxGetIdFn {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuCtxGetId", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<CtxGetIdFn>(p);
  }();
  CUcontext ctx = nullptr;
  unsigned long long id = 0;
  if (get_current == nullptr || get_id == nullptr || get_current(&ctx) != CUDA_SUCCESS ||
      ctx == nullptr || get_id(ctx, &id) != CUDA_SUCCESS)
    return 0;
  return id;
}

// ----------------------------------------------------------------- checks
inline gdattn_status check_desc(const gdattn_layer_desc *d) {
  if (d == nullptr) return GDATTN_ERR_INVALID_ARG;
  if (d->n_q_heads <= 0 || d->n_kv_heads <= 0 || d->head_dim <= 0 || d->cache_capacity <= 0)
    return GDATTN_ERR_INVALID_ARG;
  if (d->n_q_heads % d->n_kv_heads != 0) return GDATTN_ERR_INVALID_ARG;
  if (d->window < 0 || d->split_ctas < 0 ||
      (d->flags & ~(GDATTN_FLAG_EVEN_UNITS | GDATTN_FLAG_TEST_WITHHOLD_KV)) != 0)
    return GDATTN_ERR_INVALID_ARG;
  if (!(d->softcap >= 0.f) || !std::isfinite(d->softcap) || !std::isfinite(d->scale))
    return GDATTN_ERR_INVALID_ARG;
  if (d->kv_shared != 0 && d->kv_shared != 1) return GDATTN_ERR_INVALID_ARG;
  const int64_t dense = static_cast<int64_t>(d->cache_capacity) * d->n_kv_heads * d->head_dim;
  if (d->cache_batch_stride != 0 && (d->cache_batch_stride < dense || d->cache_batch_stride % 8 != 0))
    return GDATTN_ERR_INVALID_ARG;
  return GDATTN_OK;
}

// --------------------------------------------------------------- launching
inline cudaLaunchConfig_t launch_config(dim3 grid, int threads, int smem, cudaStream_t stream,
                                 cudaLaunchAttribute *attr, bool pdl = true) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  // Programmatic dependent launch: the kernel may start while its predecessor
  // drains; every kernel here waits (griddepcontrol.wait) before touching memory.
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cfg;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled() {
  static EncodeTiledFn fn = []() -> EncodeTiledFn {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// K or V cache [B][C][Hkv][D] as a 4-D tensor map {D, Hkv, C, B} read in
// 128-byte x 1-head x 64-token boxes with 128-byte swizzle: 64 bf16 elements,
// or 128 e4m3 codes (fp8), per box row.
inline bool encode_cache_map(EncodeTiledFn enc, CUtensorMap *map, const void *base, int32_t D,
                      int32_t Hkv, int32_t C, int32_t batch, int64_t bstride, uint32_t tile,
                      bool fp8 = false) {
  const cuuint64_t esz = fp8 ? 1 : 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hkv),
                              static_cast<cuuint64_t>(C), static_cast<cuuint64_t>(batch)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * esz,
                                 static_cast<cuuint64_t>(Hkv) * D * esz,
                                 static_cast<cuuint64_t>(bstride) * esz};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(128 / esz), 1, tile, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q [T][rows][D] bf16 (rows = B * Hq) as a 3-D tensor map read in
// {64 d, box_heads rows, box_tokens tokens} boxes with 128-byte swizzle: the
// query rows of a unit (box_heads heads x box_tokens tokens) land as consecutive
// 128-byte rows, token-major; tokens past T read as zeros.
inline bool encode_q_tokens_map(EncodeTiledFn enc, CUtensorMap *map, const void *q, int32_t D,
                         int64_t rows, int32_t T, int32_t box_tokens, int32_t box_heads = 2) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2,
                                 static_cast<cuuint64_t>(rows) * D * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads),
                             static_cast<cuuint32_t>(box_tokens)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gdattn
