// TMA and cluster pieces of the tree attention kernel: tiled loads, a 64-byte-swizzled operand
// descriptor, 4-byte remote stores, and a commit that arrives in both CTAs of a pair.
#pragma once
#include <cstdint>
#include <cuda.h>

#include "ptx.cuh"

namespace irm {

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// Box of a 2-d tensor map at element (x, y) into shared memory; its bytes complete on `bar`.
// x * element size must be a multiple of 16; rows outside the tensor read as zeros.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(m), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// Shared-memory matrix descriptor, 64-byte swizzle (layout type 4): rows 64 B apart, 8-row
// groups `sbo` bytes apart.
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) |
         (4ull << 61);
}

// 4-byte store into a peer CTA's shared memory, counted in bytes on the peer's mbarrier.
__device__ __forceinline__ void st_async_b32(uint32_t cluster_addr, uint32_t v, uint32_t cluster_bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(cluster_addr), "r"(v),
               "r"(cluster_bar)
               : "memory");
}

// `bytes` (a multiple of 16) of this CTA's shared memory to a peer's, counted on the peer's mbarrier.
__device__ __forceinline__ void bulk_to_peer(uint32_t cluster_addr, uint32_t src, uint32_t bytes, uint32_t cluster_bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   cluster_addr),
               "r"(src), "r"(bytes), "r"(cluster_bar)
               : "memory");
}

// The bounded waits of ptx.cuh in fewer instructions: the tree attention kernel's warps wait in some forty places, and
// with those its code does not fit the SM's instruction cache (8-bit cache, 64 x 32768 rows: 1210 us, with these
// 1110).  try_wait suspends the thread for a while, so the clock is read on every turn.
template <bool kCluster>
__device__ __forceinline__ bool mbar_wait_compact(uint32_t bar, uint32_t parity, const volatile int* abort_flag) {
  uint64_t since = 0;
#pragma unroll 1
  while (!(kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity))) {
    const uint64_t now = globaltimer_ns();
    if (since == 0) since = now;
    if ((abort_flag != nullptr && *abort_flag) || now - since > kWaitLimitNs) return false;
  }
  return true;
}
// By a whole warp, which agrees on the verdict.
template <bool kCluster>
__device__ __forceinline__ bool warp_wait_compact(uint32_t bar, uint32_t parity, const volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait_compact<kCluster>(bar, parity, abort_flag));
}

// 16-byte load from this CTA's shared memory.
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t saddr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(saddr) : "memory");
  return v;
}

// Arrive (once) on the mbarrier at this offset in every CTA of `mask` when all UMMAs issued so
// far are complete.
__device__ __forceinline__ void umma_commit_multicast(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}

}  // namespace irm
