// losses_common.cuh -- shared by the kernels of the drafter's losses: barriers for copies that the
// copy engine makes, and waits that end.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "sv_internal.h"

namespace sv {

__device__ __forceinline__ uint32_t shared_addr(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void barrier_init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_addr(bar)), "r"(count) : "memory");
}
// initialised barriers become visible to the copy engine and to other CTAs of the cluster
__device__ __forceinline__ void barrier_init_fence() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void barrier_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_addr(bar)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool barrier_try(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(shared_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ unsigned long long global_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}
// Whether the barrier's phase came to its end within `limit` ns.
static __device__ __noinline__ bool barrier_wait_slow(uint64_t* bar, uint32_t parity, unsigned long long limit) {
    const unsigned long long t0 = global_ns();
    do {
        for (int i = 0; i < 64; ++i)
            if (barrier_try(bar, parity))
                return true;
    } while (global_ns() - t0 < limit);
    return false;
}
__device__ __forceinline__ bool barrier_wait(uint64_t* bar, uint32_t parity, unsigned long long limit) {
    return barrier_try(bar, parity) || barrier_wait_slow(bar, parity, limit);
}
// The same place in another CTA of the cluster, an arrival there after what this thread wrote or saw written, and a
// bounded wait for such arrivals.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(shared_addr(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void barrier_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ bool barrier_try_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(shared_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
static __device__ __noinline__ bool barrier_wait_cluster(uint64_t* bar, uint32_t parity, unsigned long long limit) {
    const unsigned long long t0 = global_ns();
    do {
        for (int i = 0; i < 64; ++i)
            if (barrier_try_cluster(bar, parity))
                return true;
    } while (global_ns() - t0 < limit);
    return false;
}
// all threads of the cluster, in two halves
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// global to this CTA's shared memory, both ends on 16 bytes, a multiple of 16 bytes
__device__ __forceinline__ void copy_bulk(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     shared_addr(dst)),
                 "l"(src), "r"(bytes), "r"(shared_addr(bar))
                 : "memory");
}

// Of launches that may overlap: lets the next one begin, and waits until the one before has ended and its writes
// are seen.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// global to L2, the same alignment
__device__ __forceinline__ void prefetch_bulk(const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

}  // namespace sv
