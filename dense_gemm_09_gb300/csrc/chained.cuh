// chained.cuh -- launches that overlap their start with the end of the kernel
// before them on the stream (programmatic dependent launch), for the 8-bit
// calls, which often run for a few microseconds each, one after another.
//
// A kernel launched by launch_chained calls chain_wait() in every thread before
// it touches global memory: it returns when the kernels before it have
// finished and their writes are visible, so the order of the stream holds as
// ever; only the launch itself, and what a kernel sets up before the call
// (barriers, tensor memory), lie beside the previous kernel.  chain_next()
// lets the next such launch begin as soon as all blocks of this one run.
//
// So an operand of such a kernel may be written while the kernel already runs,
// and the non-coherent loads (ld.global.nc, __ldg, const __restrict__
// parameters), which may count on read-only data and move across the wait, do
// not fit.  Vectors and scales are loaded through the functions here, whose
// assembly is volatile like chain_wait()'s and stays behind it.  Single elements
// are plain loads through pointers without restrict: chain_wait() says that it
// writes memory, so the compiler keeps them behind it too.
#pragma once

#include <cstdint>
#include <utility>

#include <cuda_runtime.h>

namespace dgemm {

__device__ __forceinline__ void chain_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void chain_next()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float load_f32(const float *p)
{
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t load_u32(const uint32_t *p)
{
    uint32_t v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// kOnce: the bytes are not read again (not kept in L1).
template <bool kOnce = false>
__device__ __forceinline__ uint4 load_v4(const void *p)
{
    uint4 v;
    if constexpr (kOnce)
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(p));
    else
        asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(p));
    return v;
}

// The bytes are read once and may leave the caches first.
__device__ __forceinline__ uint4 load_v4_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

inline cudaLaunchAttribute chained_attribute()
{
    cudaLaunchAttribute a = {};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    return a;
}

// `cluster` CTAs to a cluster (1: none).
template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                           unsigned cluster, Args &&...args)
{
    cudaLaunchAttribute attr[2];
    attr[0] = chained_attribute();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace dgemm
