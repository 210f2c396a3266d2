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
#pragma once

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
