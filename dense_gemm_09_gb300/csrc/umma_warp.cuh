// umma_warp.cuh -- what the warp-specialised tensor-core kernels for 8-bit
// operands share beyond ptx.cuh: commits and arrivals of a CTA or a pair, small
// TMEM loads, and bounded waits of whole warps.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "bounded_wait.cuh"
#include "ptx.cuh"

namespace dgemm {
namespace {

// Arrive on the barrier at this offset in every CTA of the pair (or in this
// CTA) when the MMAs issued so far by this thread complete.
template <int kCtas>
__device__ __forceinline__ void commit_all(uint32_t bar)
{
    if constexpr (kCtas == 2)
        ptx::umma_commit_pair_multicast(bar, 0x3);
    else
        ptx::umma_commit(bar);
}

__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// Arrive on an mbarrier of another CTA of the cluster with release at CTA
// scope: what it publishes is this CTA's tensor memory and, fenced to the async
// proxy, its shared memory, which this SM's own half of the pair's MMA reads;
// no thread of the other CTA does.  (A release at cluster scope waits ~650
// clocks for every earlier store of the thread to be acknowledged.)
__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// True in one thread of the (converged) warp.  The compiler keeps the operands
// of tcgen05 instructions under this predicate in uniform registers.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Meet the other CTA of the cluster without ordering memory.  (A releasing
// arrival waits for all earlier stores, up to ~1 us.)
__device__ __forceinline__ void cluster_meet()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ void fence_cluster()
{
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

__device__ __forceinline__ void named_barrier(uint32_t id, uint32_t threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Bounded waits of a whole converged warp.  Every step is decided by a vote, so
// that no branch diverges: a divergent wait (one lane probing, or a per-thread
// loop) costs hundreds of clocks in reconvergence on each half.  False for the
// whole warp on time-out or abort.
template <bool kCluster>
__device__ __forceinline__ bool probe(uint32_t bar, uint32_t parity)
{
    return __all_sync(0xFFFFFFFFu, kCluster ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity));
}

template <bool kCluster>
__device__ __noinline__ bool warp_wait_slow(uint32_t bar, uint32_t parity, WaitCtl *wc)
{
#pragma unroll 1
    for (int i = 0; i < 4; ++i)
        if (probe<kCluster>(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns(), limit = wc->limit_ns;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (probe<kCluster>(bar, parity)) return true;
        if (__any_sync(0xFFFFFFFFu, aborted(wc))) return false;
        if (__any_sync(0xFFFFFFFFu, ptx::globaltimer_ns() - t0 > limit)) {
            raise_abort(wc);
            return false;
        }
    }
}

template <int kCtas>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, WaitCtl *wc)
{
    return probe<kCtas == 2>(bar, parity) || warp_wait_slow<kCtas == 2>(bar, parity, wc);
}

}  // namespace
}  // namespace dgemm
