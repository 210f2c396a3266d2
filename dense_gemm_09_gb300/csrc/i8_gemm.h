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

// Kernel of one call: variant, tile width and split (as dgemm_tune_i8_next
// numbers them).
enum { kI8Auto = 0, kI8Mma = 1, kI8PairTokens = 2, kI8PairChannels = 3, kI8Split = 4, kI8Decode = 5, kI8Dot = 6 };
struct I8Config {
    int variant;
    int bn;     // tile columns: channels (kI8PairTokens) or tokens
    int split;  // kI8Split: CTAs that share a tile along K
};

// The tensor-core kernels (i8_umma.cu), for operands TMA can describe: false,
// and nothing launched, where the configuration cannot run.
bool i8_umma_config_ok(const I8Config &cfg);
bool launch_i8_umma(const I8Params &c, int c_type, const I8Config &cfg, cudaStream_t stream);
// Whether the configuration's CTAs can be resident together where they have to
// (split-K, wide tiles); true without a GPU and for the other kernels.
bool i8_umma_fits(const I8Params &c, const I8Config &cfg);

// The kernels for few tokens (i8_decode.cu), for operands with 16-byte aligned
// rows: as above.
bool i8_decode_config_ok(const I8Config &cfg);
bool launch_i8_decode(const I8Params &p, int c_type, const I8Config &cfg, int sm_count, cudaStream_t stream);

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
