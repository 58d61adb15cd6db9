// Inline-PTX helpers for kernels whose tensor-core products run on a CTA pair (two SMs, one 256-row
// product, each CTA holding its half of A, of B and of the accumulator rows). The pair is a cluster of
// two; its even CTA issues the products. Written from the PTX ISA description of the instructions.
#pragma once

#include <stdint.h>

#include "tc_utils.cuh"

namespace rapt {
namespace tcp {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of the pair; orders the shared-memory accesses before it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared-memory location `addr` in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// tc::mbar_wait, but a phase that is already complete costs one probe and no clock.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, long long max_cycles) {
  return tc::mbar_try_wait(bar, parity) || tc::mbar_wait(bar, parity, max_cycles);
}
// A place in a ring of N stages and how often the ring has been round, for a single thread's loop.
template <int N>
struct Ring {
  int s = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void step() {
    if (++s == N) {
      s = 0;
      ++round;
    }
  }
};

// One arrival on an mbarrier of any CTA of the cluster (an address from map_rank). What it announces here
// is that TMEM has been read, which tcgen05.fence::before_thread_sync orders before it; a release at
// cluster scope, which would wait for the thread's shared-memory stores as well, took 40 % of the
// epilogue's time.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One warp of each CTA of the pair executes them.
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// A box of a 2-D tensor map into this CTA's shared memory; its bytes count on `bar`, which may lie in
// the pair's other CTA. x (the innermost coordinate) is a multiple of 8 elements.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// The same of a 3-D map.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const void* tmap, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}

// D[tmem] (+)= A B; the descriptors' offsets hold in both CTAs.
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One arrival, once every product issued so far by this thread is done, on `bar` here and at the same
// place in the pair's other CTA.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

}  // namespace tcp
}  // namespace rapt
