// kvp_matmul.cuh -- what the block-scaled matrix products share: waits, rings, clusters,
// and the store of a result.
#pragma once

#include "kvp_device.cuh"
#include "kvp_project.h"

namespace kvp {
namespace mm {

// dev::mbar_wait_bounded without a call: a called function's registers do not go with
// setmaxnreg.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity,
                                     uint64_t limit_ns = dev::kWaitTimeoutNs) {
  // (reading the timer takes longer than most waits last)
#pragma unroll 1
  for (int i = 0; i < 64; ++i) {
    if (dev::mbar_try_wait(bar, parity)) return true;
  }
  const uint64_t t0 = dev::global_timer_ns();
#pragma unroll 1
  for (uint32_t i = 0; i < (1u << 26); ++i) {
    if (dev::mbar_try_wait_sleep(bar, parity, dev::kWaitHintNs)) return true;
    if ((i & 15u) == 15u && dev::global_timer_ns() - t0 > limit_ns) break;
  }
  return false;
}

// A ring's place and how often it has wrapped (mod 2): what is waited for is the phase
// `flip` of a full place, and `flip ^ 1` of a free one (a new barrier's passes).
template <int kPlaces>
struct Ring {
  int at = 0;
  uint32_t flip = 0;
  __device__ __forceinline__ void next() {
    if (++at == kPlaces) {
      at = 0;
      flip ^= 1;
    }
  }
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Where CTA `rank` of the cluster has what lies at shared address `addr` here.
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
  uint32_t there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(addr), "r"(rank));
  return there;
}
__device__ __forceinline__ void store_remote(uint32_t there, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there), "r"(v) : "memory");
}

__device__ __forceinline__ float4 load_remote4(uint32_t there) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(there)
               : "memory");
  return v;
}

__device__ __forceinline__ void store_out(const MatmulParams& p, long long at, float v) {
  if (p.out_type == KVP_F32) static_cast<float*>(p.out)[at] = v;
  else if (p.out_type == KVP_BF16) static_cast<uint16_t*>(p.out)[at] = dev::from_float<true>(v);
  else static_cast<uint16_t*>(p.out)[at] = dev::from_float<false>(v);
}

// Four neighbouring results of a row that starts on 4 elements.
__device__ __forceinline__ void store_out4(const MatmulParams& p, long long at, float4 v) {
  if (p.out_type == KVP_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = v;
  } else {
    const bool bf = p.out_type == KVP_BF16;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
        make_uint2(bf ? dev::pack2<true>(v.x, v.y) : dev::pack2<false>(v.x, v.y),
                   bf ? dev::pack2<true>(v.z, v.w) : dev::pack2<false>(v.z, v.w));
  }
}

}  // namespace mm
}  // namespace kvp
