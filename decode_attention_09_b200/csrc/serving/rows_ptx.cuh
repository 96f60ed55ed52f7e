// PTX wrappers of the row kernels: loads of query blocks, TMEM stores, wide global
// stores, and distributed shared memory of a CTA pair.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "../ptx.cuh"

namespace gdattn {

// A row's reference moves when a score exceeds it by a factor of 2^kRefStep.
constexpr float kRefStep = 24.f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// A box of query rows: 64 dims of consecutive heads of consecutive tokens.
__device__ __forceinline__ void tma_load_tokens(void *dst_smem, const CUtensorMap *map, int32_t d,
                                                int32_t head, int32_t token, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst_smem)),
      "l"(map), "r"(d), "r"(head), "r"(token), "r"(smem_u32(bar))
      : "memory");
}

// 32 consecutive columns of this thread's TMEM lane; load and wait in one statement.
__device__ __forceinline__ void tmem_load32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Store 16 consecutive columns; tmem_store_wait before anyone reads them.
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const float (&v)[16]) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_store_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 32 bytes to global memory: one sector per lane.
// On a 32-byte boundary ...
__device__ __forceinline__ void st_global_v8(void *dst, const uint32_t *v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// ... and on a 16-byte one.
__device__ __forceinline__ void st_global_2v4(void *dst, const uint32_t *v) {
  uint4 *to = static_cast<uint4 *>(dst);
  to[0] = make_uint4(v[0], v[1], v[2], v[3]);
  to[1] = make_uint4(v[4], v[5], v[6], v[7]);
}

// Four neighbouring lanes with four pieces of 8 words each: afterwards lane j holds,
// as piece k, piece j of lane k.
__device__ __forceinline__ void swap_pieces(uint32_t (&v)[32], int lane) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (a & bit) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t &lo = v[8 * a + i], &hi = v[8 * (a | bit) + i];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, bit);
        if (up)
          lo = got;
        else
          hi = got;
      }
    }
  }
}

// The two warps that share rows (64 threads), on named barrier `id`.
__device__ __forceinline__ void pair_sync(int id) {
  asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}

// Arrive there for the other warp's pair_sync, without waiting.
__device__ __forceinline__ void pair_arrive(int id) {
  asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory");
}

// The four warps of a softmax group, on named barrier `id`.
__device__ __forceinline__ void group_sync(int id) {
  asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}

// The n lowest bits set (none for n <= 0, all for n >= 64).
__device__ __forceinline__ uint64_t low_bits(int32_t n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// A score in log2 units from its dot product: scaled, or scaled, capped and scaled
// again.  tanh x = 1 - 2 / (e^2x + 1): absolute error a few 2^-24, and only the
// absolute error of a score matters to its weight.
template <bool CAP>
__device__ __forceinline__ float score_log2(float s, float qscale, float post) {
  if (!CAP) return s * qscale;
  const float e = ex2_approx(s * (qscale * 2.8853900817779268f));  // 2 log2(e)
  return fmaf(__fdividef(-2.f, e + 1.f), post, post);
}

// For |s qscale| <= kSmallTanh tanh's Taylor series is used, whose first term left out,
// 1382 / 155925 x^11, is below 2^-28 there.  No exponential and no division: the
// capped weights of a tile take half the time.
constexpr float kSmallTanh = 0.25f;

// Two fp32 numbers that one instruction works on (half the issue slots of the softmax).
using float2x = uint64_t;
__device__ __forceinline__ float2x pack2(float a, float b) {
  float2x r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(float2x v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ float2x fma2(float2x a, float2x b, float2x c) {
  float2x r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float2x mul2(float2x a, float2x b) {
  float2x r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float2x add2(float2x a, float2x b) {
  float2x r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// The largest, or smallest, of three.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// cap log2(e) tanh(x) - mr by the series, x = s qscale; k are the series' factors of
// x^3 to x^9 times post = cap log2(e).
struct SmallTanh {
  float2x qscale, post, k3, k5, k7, k9;
  __device__ __forceinline__ SmallTanh(float q, float cap_log2e)
      : qscale(pack2(q, q)),
        post(pack2(cap_log2e, cap_log2e)),
        k3(pack2(-1.f / 3.f * cap_log2e, -1.f / 3.f * cap_log2e)),
        k5(pack2(2.f / 15.f * cap_log2e, 2.f / 15.f * cap_log2e)),
        k7(pack2(-17.f / 315.f * cap_log2e, -17.f / 315.f * cap_log2e)),
        k9(pack2(62.f / 2835.f * cap_log2e, 62.f / 2835.f * cap_log2e)) {}
  __device__ __forceinline__ float2x operator()(float2x s, float2x minus_mr) const {
    const float2x x = mul2(s, qscale), y = mul2(x, x);
    const float2x g = mul2(y, fma2(y, fma2(y, fma2(y, k9, k7), k5), k3));
    return fma2(x, g, fma2(x, post, minus_mr));
  }
};

// --------------------------------------------- distributed shared memory
// All threads of the cluster's CTAs; orders their earlier shared-memory accesses.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// The address, in CTA `rank` of the cluster, of the shared location `saddr` here.
__device__ __forceinline__ uint32_t peer_smem(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}

__device__ __forceinline__ void st_peer_v4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b),
               "f"(c), "f"(d)
               : "memory");
}

// Arrive on a barrier of another CTA; what this thread observed before (the
// warp's stores, after __syncwarp) is visible to who waits there at cluster scope.
__device__ __forceinline__ void mbar_arrive_peer(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
               : "memory");
}

// mbar_wait for a barrier that the peer CTA arrives on.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity,
                                                  volatile int *abort, uint32_t *status) {
  const long long t0 = clock64();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendHintNs)
        : "memory");
    if (ok) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      *abort = 1;
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
}

}  // namespace gdattn
