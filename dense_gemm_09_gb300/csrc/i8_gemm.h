// i8_gemm.h -- what the kernels behind gemm_i8_tn share: the call's
// parameters and the output types' conversions.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace dgemm {

struct I8Params {
    int64_t M, N, K;
    const int8_t *A, *B;
    int64_t lda, ldb;
    const float *scale_a, *scale_b;
    const float *bias;  // may be null
    float beta;
    void *C;
    int64_t ldc;
};

__device__ __forceinline__ float i8_to_f32(float v) { return v; }
__device__ __forceinline__ float i8_to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float i8_to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T i8_from_f32(float v);
template <>
__device__ __forceinline__ float i8_from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half i8_from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 i8_from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

}  // namespace dgemm
