// bounded_wait.cuh -- mbarrier waits with a limit, for the warp-specialised
// tensor-core kernels.  A wait that runs out records DGEMM_ERR_TIMEOUT in the
// unit's status word and raises the CTA's abort flag, which its other waits
// poll; every role then leaves by itself.  Device code is not linked across
// translation units, so each unit that includes this header has its own
// status word (read_wait_status).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "dgemm.h"
#include "ptx.cuh"

namespace dgemm {
namespace {

__device__ int g_wait_status;

constexpr uint64_t kWaitLimitNs = 4000000000ull;   // 4 s, default wait bound
constexpr uint64_t kDrainLimitNs = 1000000000ull;  // 1 s

// Per-CTA wait control: the abort flag every role polls and the wait limit.
struct WaitCtl {
    int abort;
    int pad;
    uint64_t limit_ns;
};

__device__ __forceinline__ bool aborted(const WaitCtl *wc)
{
    return *reinterpret_cast<const volatile int *>(&wc->abort) != 0;
}

__device__ __forceinline__ void raise_abort(WaitCtl *wc)
{
    if (atomicExch(&g_wait_status, DGEMM_ERR_TIMEOUT) == 0) __threadfence();
    *reinterpret_cast<volatile int *>(&wc->abort) = 1;
}

// Bounded wait for the phase of the given parity; false on time-out or when
// another role raised the abort flag.
__device__ __noinline__ bool wait_bounded(uint32_t bar, uint32_t parity, WaitCtl *wc)
{
    if (ptx::mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
    for (int i = 0; i < 4; ++i)  // most waits end here, before the first look at the clock
        if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns(), limit = wc->limit_ns;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (ptx::mbar_try_wait(bar, parity)) return true;
        if (aborted(wc)) return false;
        if (ptx::globaltimer_ns() - t0 > limit) {
            raise_abort(wc);
            return false;
        }
    }
}

// Same, with cluster-scope acquire (barriers that the other CTA of a pair
// arrives on, directly or through a multicast commit).
__device__ __noinline__ bool wait_bounded_cluster(uint32_t bar, uint32_t parity, WaitCtl *wc)
{
    if (ptx::mbar_try_wait_cluster(bar, parity)) return true;
#pragma unroll 1
    for (int i = 0; i < 4; ++i)  // most waits end here, before the first look at the clock
        if (ptx::mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns(), limit = wc->limit_ns;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (ptx::mbar_try_wait_cluster(bar, parity)) return true;
        if (aborted(wc)) return false;
        if (ptx::globaltimer_ns() - t0 > limit) {
            raise_abort(wc);
            return false;
        }
    }
}

// Bounded wait used on the way out, after an abort: ignores the abort flag.
__device__ __noinline__ bool drain_wait(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, parity))
        if (ptx::globaltimer_ns() - t0 > kDrainLimitNs) return false;
    return true;
}

// The unit's status word: 0 or DGEMM_ERR_TIMEOUT; reset when clear != 0.
int read_wait_status(int clear)
{
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_wait_status, sizeof(int)) != cudaSuccess) return DGEMM_ERR_LAUNCH;
    if (clear) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_wait_status, &zero, sizeof(int)) != cudaSuccess) return DGEMM_ERR_LAUNCH;
    }
    return v;
}

}  // namespace
}  // namespace dgemm
