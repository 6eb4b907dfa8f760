// hlq_tma.cuh -- mbarrier waits (bounded) and TMA tile loads, shared by the
// tensor-core GEMMs and the TMA-staged transform kernels.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "hlq.h"

namespace hlq {

constexpr unsigned long long kWaitNs = 2000000000ull;  // 2 s per wait

__device__ __forceinline__ uint32_t saddr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(count)
               : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(b)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(b)) : "memory");
}

__device__ __forceinline__ bool mbar_test(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(saddr(b)), "r"(parity)
      : "memory");
  return ok != 0;
}

// try_wait with cluster-scope acquire, for barriers that threads of other
// CTAs of the cluster arrive on (with release at cluster scope).
__device__ __forceinline__ bool mbar_test_cluster(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(saddr(b)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Wait for the phase of parity `parity` to complete; gives up after
// `limit_ns` (or as soon as another role gave up), raising HLQ_DEV_TIMEOUT
// once.
__device__ __forceinline__ bool mbar_wait_for(uint64_t* b, uint32_t parity,
                                              volatile int* abort_flag,
                                              unsigned int* status,
                                              unsigned long long limit_ns,
                                              bool cluster_scope = false) {
  auto test = [&]() {
    return cluster_scope ? mbar_test_cluster(b, parity) : mbar_test(b, parity);
  };
  if (test()) return true;
  const unsigned long long t0 = now_ns();
  while (true) {
    if (test()) return true;
    if (*abort_flag) return false;
    if (now_ns() - t0 > limit_ns) {
      if (atomicExch((int*)abort_flag, 1) == 0) atomicOr(status, HLQ_DEV_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity,
                                          volatile int* abort_flag,
                                          unsigned int* status,
                                          bool cluster_scope = false) {
  return mbar_wait_for(b, parity, abort_flag, status, kWaitNs, cluster_scope);
}

// Four floats of another CTA's shared memory (a shared::cluster address).
__device__ __forceinline__ float4 load_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// After a wait on a ring of stages gave up: wait, each within the same limit,
// for the copies that are still on their way into shared memory.  `issued`
// rows have been copied so far, row r into stage r % stages.
__device__ __forceinline__ void ring_drain(uint64_t* full, int stages, int64_t issued) {
  for (int s = 0; s < stages && s < issued; ++s) {
    const uint32_t parity = (uint32_t)((issued - 1 - s) / stages) & 1;
    const unsigned long long t0 = now_ns();
    while (!mbar_test(&full[s], parity) && now_ns() - t0 < kWaitNs) {
    }
  }
}

// Address of the same shared-memory object in CTA `rank` of the cluster
// (a shared::cluster address).
__device__ __forceinline__ uint32_t cluster_map(uint32_t local_saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local_saddr), "r"(rank));
  return r;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Every thread of every CTA of the cluster (release / acquire at cluster
// scope, so shared-memory writes before it are seen by peers after it).
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same barrier in two steps, without ordering memory: between them a
// thread goes on; after the wait every CTA of the cluster has started, which
// an access to its shared memory needs.
__device__ __forceinline__ void cluster_started_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_started_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// Arrive on an mbarrier of another CTA of the cluster (shared::cluster
// address), releasing this thread's earlier writes at cluster scope.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                   cluster_addr)
               : "memory");
}

// Tile load into this CTA's shared memory whose completion is signalled on
// an mbarrier that may live in the peer CTA of a CTA pair (shared::cluster
// address of the barrier): the operand loads of the pair GEMM.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(saddr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar_cluster)
      : "memory");
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map,
                                            uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(saddr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(saddr(bar))
      : "memory");
}

// Untiled copy of `bytes` (a multiple of 16; both addresses 16-byte aligned)
// into this CTA's shared memory, signalled on one of its mbarriers.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(saddr(bar))
      : "memory");
}

// Tiled store of a shared-memory box to global memory (the box layout of the
// tensor map, swizzle included); parts outside the tensor are not written.
// Completion is tracked per thread in bulk groups: commit after issuing,
// `tma_store_wait_read` before reusing the source, `tma_store_wait_all`
// before the thread exits.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y,
                                             const void* src) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(saddr(src))
      : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Tiled reduce-add of a shared-memory box into global memory (element type
// of the tensor map, here s32), the same bulk-group completion as the store.
__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap* map, int x, int y,
                                                  const void* src) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group"
      " [%0, {%1, %2}], [%3];" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(saddr(src))
      : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// Orders this thread's generic shared-memory writes before later async-proxy
// (TMA) reads of them.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

}  // namespace hlq
