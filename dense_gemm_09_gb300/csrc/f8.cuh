// f8.cuh -- 8-bit floating point: what the kernels share, conversions and the
// quantisation of a block.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dgemm.h"

namespace dgemm {

constexpr int kF8Block = 128;  // columns that share a scale

// An operand of a product, as the kernels take it.
struct F8Operand {
    const uint8_t *p;
    int64_t ld;
    const float *scale;
    int64_t s_row, s_blk;
    int type, block;

    // the row of scales of a row
    __host__ __device__ int64_t band(int64_t row) const { return block == 1 ? row : row / kF8Block; }
};

inline F8Operand f8_operand(const dgemm_f8 &m)
{
    return {static_cast<const uint8_t *>(m.data), m.ld, m.scale, m.scale_row, m.scale_blk, m.type, m.block};
}

struct F8Params {
    int64_t M, N, K;
    F8Operand a, b;
    int experts;             // 1 and offsets == nullptr: one matrix
    const int32_t *offsets;
    int64_t b_stride, sb_stride;
    const float *bias;       // may be null
    float beta;
    void *C;
    int64_t ldc;
    int c_type;
};

constexpr int kMaxExperts = 1024;

// Kernel of one call: variant, tile width and split (as dgemm_tune_f8_next numbers them).
enum { kF8Auto = 0, kF8Any = 1, kF8Pair = 2, kF8Channels = 3, kF8Decode = 4 };
struct F8Config {
    int variant;
    int bn;     // tile columns: channels (kF8Pair) or tokens (kF8Channels)
    int split;  // kF8Channels: CTAs that share a tile along K; kF8Decode: warps of a thread block
};

// The tensor-core kernels (f8_umma.cu): false, and nothing launched, where the
// configuration cannot run.
bool f8_umma_config_ok(const F8Config &cfg);
bool launch_f8_umma(const F8Params &c, const F8Config &cfg, cudaStream_t stream);

// The kernel for a few tokens (f8_decode.cu), for operands with 16-byte aligned rows: as above.
constexpr int kF8DecodeTokens = 8;
bool f8_decode_config_ok(const F8Config &cfg);
bool launch_f8_decode(const F8Params &p, const F8Config &cfg, cudaStream_t stream);

// Tuning hook behind dgemm_tune_f8_next: the request of this host thread, and its
// taking (by every gemm_f8_tn and gemm_f8_tn_experts call, whatever becomes of it).
int f8_tune_next(int variant, int bn, int split);
F8Config f8_take_tune();

#ifdef __CUDACC__
namespace {

// Two 8-bit values (in the low 16 bits) as FP16, exactly.
template <bool kE5>
__device__ __forceinline__ uint32_t f8x2_to_f16x2(uint32_t v)
{
    uint32_t h;
    if constexpr (kE5)
        asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e5m2x2 %0, a;\n\t}" : "=r"(h) : "r"(v));
    else
        asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(v));
    return h;
}

// Two FP32 values to 8 bits, nearest, ties to even, the largest value for what is past it.
template <bool kE5>
__device__ __forceinline__ uint32_t f32x2_to_f8x2(float lo, float hi)
{
    uint16_t r;
    if constexpr (kE5)
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// A block's scale and factor, from its largest |y| (as bits: for magnitudes
// unsigned order is the order of the values, infinities and then NaNs last).
template <bool kE5>
struct F8Block {
    float scale, inv;  // inv: 0 of zeros, and of a block that is not finite
    bool tiny;         // y is multiplied by 2^100 before inv

    __device__ __forceinline__ explicit F8Block(uint32_t most_bits)
    {
        constexpr float kTop = kE5 ? 57344.f : 448.f;
        const float a = __uint_as_float(most_bits);
        const bool finite = most_bits < 0x7F800000u;
        scale = finite ? a / kTop : __uint_as_float(0x7FC00000u);
        tiny = a < 0x1p-100f && a > 0.f;
        inv = finite && a > 0.f ? kTop / (tiny ? a * 0x1p100f : a) : 0.f;
    }
};

// Eight values of one block, or (inv[i]) of eight.  Without a factor they give zeros (their
// product with 0 may be NaN).
template <bool kE5>
__device__ __forceinline__ uint2 f8_eight(const float (&y)[8], float inv)
{
    uint32_t h[4];
    uint64_t inv2;
    asm("mov.b64 %0, {%1, %1};" : "=l"(inv2) : "f"(inv));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint64_t v;
        float lo, hi;
        asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(y[2 * i]), "f"(y[2 * i + 1]));
        asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(inv2));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
        h[i] = f32x2_to_f8x2<kE5>(lo, hi);
    }
    if (inv == 0.f) return make_uint2(0u, 0u);
    return make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
}

}  // namespace
#endif

}  // namespace dgemm
