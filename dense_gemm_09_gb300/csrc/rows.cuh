// rows.cuh -- what the kernels over rows of values share: loads and stores of
// vectors of 8 elements, conversions, magnitudes, packed FP32 arithmetic.
// (Include after checked.cuh: the unit's checks apply.)
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chained.cuh"

namespace dgemm {
namespace {

constexpr int kVec = 8;  // elements of one vector: 16 bytes of a 16-bit type, 8 bytes of q

// ---- loads and stores of one vector (or its first n elements)

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Elements of the vector at column c.
__device__ __forceinline__ int vec_len(int64_t cols, int64_t c)
{
    const int64_t left = cols - c;
    return left >= kVec ? kVec : left > 0 ? static_cast<int>(left) : 0;
}

// A vector as it lies in memory.
template <typename T>
struct Raw {
    static constexpr int kWords = kVec * sizeof(T) / 16;
    uint4 w[kWords];
};

// kAligned: the vector starts on a 16-byte boundary; n < kVec, or an unaligned
// operand, takes element loads.  Elements past n are 0.
// kKeep: the vector is read again by other rows (else it streams through).
template <typename T, bool kAligned, bool kKeep = false>
__device__ __forceinline__ Raw<T> load_raw(const T *p, int n)
{
    Raw<T> r;
    if (kAligned && n == kVec) {
#pragma unroll
        for (int i = 0; i < Raw<T>::kWords; ++i)
            r.w[i] = kKeep ? load_v4(reinterpret_cast<const uint4 *>(p) + i)
                           : load_v4_stream(reinterpret_cast<const uint4 *>(p) + i);
        return r;
    }
    alignas(16) T e[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) e[i] = i < n ? p[i] : from_f32<T>(0.f);
#pragma unroll
    for (int i = 0; i < Raw<T>::kWords; ++i) r.w[i] = reinterpret_cast<const uint4 *>(e)[i];
    return r;
}

template <typename T>
__device__ __forceinline__ void unpack(const Raw<T> &r, float (&v)[kVec])
{
    if constexpr (sizeof(T) == 4) {
        const float *e = reinterpret_cast<const float *>(r.w);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = e[i];
    } else {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(r.w);
#pragma unroll
        for (int i = 0; i < kVec / 2; ++i) {
            float2 f;
            if constexpr (std::is_same<T, __half>::value)
                f = __half22float2(*reinterpret_cast<const __half2 *>(w + i));
            else
                f = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

template <typename T, bool kAligned>
__device__ __forceinline__ void store_vec(T *p, int n, const float (&v)[kVec])
{
    if (kAligned && n == kVec && DGEMM_CHECK((reinterpret_cast<uintptr_t>(p) & 15u) == 0)) {
        Raw<T> r;
        uint32_t *w = reinterpret_cast<uint32_t *>(r.w);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) {
                if constexpr (std::is_same<T, __half>::value) {
                    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t *>(&h);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t *>(&h);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < Raw<T>::kWords; ++i) reinterpret_cast<uint4 *>(p)[i] = r.w[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (i < n) p[i] = from_f32<T>(v[i]);
}

// max(|a|, |b|, |c|), NaN if one of them is.
__device__ __forceinline__ float max3_abs(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float max_abs(float amax, const float (&v)[kVec])
{
#pragma unroll
    for (int i = 0; i < kVec; i += 2) amax = max3_abs(amax, v[i], v[i + 1]);
    return amax;
}

// Two FP32 operations at a time.
__device__ __forceinline__ uint64_t pack2(float lo, float hi)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// g / (1 + exp(-g)).  1 + exp(-g) is formed as 4 (1/4 + 2^(-g log2 e - 2)), whose
// second factor's reciprocal is a normal number up to the largest finite sum (2^128,
// at g = -88.7, where the quotient is 2^-121: a large u makes an ordinary value of
// it), so that the plain approximations do, flushing what is below (ex2 within
// 2^-22, rcp within 2^-23).  Past it the quotient is 0, as in FP32 arithmetic.
__device__ __forceinline__ float silu(float g)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(g, -1.4426950408889634f, -2.f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(0.25f + e));
    return g * (0.25f * r);
}

// Whether rows at this pitch (in elements) all start on a boundary of `to` bytes.
inline bool aligned(const void *p, int64_t ld, int64_t elem, int64_t to)
{
    return reinterpret_cast<uintptr_t>(p) % to == 0 && (ld * elem) % to == 0;
}

}  // namespace
}  // namespace dgemm
