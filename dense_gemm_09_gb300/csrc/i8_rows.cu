// i8_rows.cu -- the row operators around the 8-bit product (gemm_i8_tn):
// each reads rows of FP32 / FP16 / BF16 values and writes int8 rows with one
// FP32 scale a row, or the reverse.
//
//   quantize    y = x
//   rmsnorm     h = x + r;  y = h * gamma / sqrt(mean(h^2) + eps);  H = h
//   swiglu      y = g / (1 + exp(-g)) * u
//   then        a = max |y|,  scale = a / 127,  q = rint(y * 127 / a)
//   dequantize  x = q * scale
//
// All of it is FP32 arithmetic on the stored values; a rounding to fewer bits
// happens once, where q or H is stored (the norm uses the unrounded h).
//
// The bound is HBM: every input byte is read once and every output byte
// written once.  A row needs two results over all of its elements before the
// first q can be written (the norm's sum of squares, then the maximum), so the
// row's values stay in registers between: a warp or a block holds a row, kVecs
// vectors of 8 elements a thread.  Rows longer than the registers
// of one block (32768 elements) are read again from memory for each pass.
// At 3 to 7 bytes an element the instructions count too (an SM has ~8 of them
// for each of its threads' elements at HBM speed), hence the packed
// conversions, the three-input maximum and the rounding by one addition below.
#include <atomic>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chained.cuh"
#include "dgemm.h"
#include "internal.h"

#define DGEMM_UNIT 6
#include "checked.cuh"

namespace dgemm {
namespace {

constexpr int kVec = 8;  // elements of one vector: 16 bytes of a 16-bit type, 8 bytes of q
constexpr int64_t kResident = 152 * 2048;  // threads that run at once

// kOpNorm with a residual, kOpNormAlone without
enum { kOpQuantize = 0, kOpNorm = 1, kOpSwiglu = 2, kOpNormAlone = 3 };

constexpr bool is_norm(int op)
{
    return op == kOpNorm || op == kOpNormAlone;
}

constexpr bool has_second(int op)
{
    return op == kOpNorm || op == kOpSwiglu;
}

struct RowParams {
    int64_t rows, cols;
    const void *x;  // the row to quantise / norm; the gate of swiglu
    int64_t ldx;
    const void *y;  // residual (kOpNorm) or the up rows (swiglu)
    int64_t ldy;
    const void *gamma;
    int gamma_f32;  // gamma is FP32 whatever the rows' type
    float eps;
    void *h;  // norm: x + residual, rounded (may be null)
    int64_t ldh;
    int8_t *q;
    int64_t ldq;
    float *scale;
};

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

// ---- the quantisation's scale and steps

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

// How a row's quotients 127 y / a are formed.  A product with the rounded 127 / a
// leans to one side, and half of all ties (a whole number and a half) go to the
// wrong step.  y (hi + lo), with hi + lo = 127 / a to ~2^-46 and the sum rounded
// once, makes a tie of every quotient that is one.
//   kOneProduct   for y with several FP32 roundings in them, ties there being
//                 chance;
//   kTies         ties are right.  Quotients of 16-bit y that are no ties are at
//                 least 2^-20 (relative) away from all ties and cannot come out
//                 as one;
//   kTiesAndNear  those of FP32 y may be as near as 2^-33: what comes out as a
//                 tie is looked at again.
// 8192 x 8192, one product and the form in use: quantize bf16 30.2 and 30.5 us, FP32
// 48.2 and 49.1; norm of bf16 40.1 and 39.0 (its quotients do without 1 / sqrt).
enum { kOneProduct, kTies, kTiesAndNear };

template <int kOp, typename T>
constexpr int quotient_form()
{
    if (kOp == kOpSwiglu) return kOneProduct;
    return kOp == kOpQuantize && sizeof(T) == 4 ? kTiesAndNear : kTies;
}

// The steps rint(127 y / a), ties to even, of a row whose largest |y| is a.
// Rounding to a whole number is the addition of 1.5 * 2^23, whose unit in the last
// place is 1: the step is the sum's low byte.  |y| <= a, and a quotient that
// rounds up past 127 still rounds to 127.
template <int kForm>
struct Quantiser {
    float scale, hi, lo, factor;
    bool finite;

    static constexpr float kWhole = 12582912.f;

    // For y = values * times: the largest |value| as its bits, and times.  (For
    // non-negative floats unsigned order is the order of the values, infinities
    // and then NaNs above every finite one, so the threads' maxima meet in an
    // integer maximum.)  The steps do not depend on `times`.
    __device__ __forceinline__ explicit Quantiser(uint32_t most_bits, float times = 1.f)
    {
        float most = __uint_as_float(most_bits);
        const float a = most * times;
        finite = a < __uint_as_float(0x7F800000u);
        scale = finite ? a / 127.f : __uint_as_float(0x7FC00000u);
        // far from 1, hi or lo would leave FP32's range: such rows are first
        // multiplied by a power of two.  (That is exact upwards; downwards it
        // may round values below 2^-26 of the largest, whose steps are 0.)
        factor = most < 0x1p-100f ? 0x1p100f : most > 0x1p100f ? 0x1p-100f : 1.f;
        most *= factor;
        hi = a > 0.f ? 127.f / most : 0.f;
        lo = fmaf(-hi, most, 127.f) * (hi * (1.f / 127.f));  // what hi is short of, over `most`
    }

    // kWhole + the step of one y, where the rounded quotient t may be a tie without
    // y's own being one; rest: what the rounding took.
    __device__ __forceinline__ float past_tie(float y) const
    {
        const float t = fmaf(y, hi, y * lo), sum = t + kWhole, side = t - (sum - kWhole);
        const float rest = fmaf(y, lo, fmaf(y, hi, -t));
        if (fabsf(side) == 0.5f && fabsf(rest) > 0x1p-38f * fabsf(t)) {
            if (side > 0.f && rest > 0.f) return sum + 1.f;
            if (side < 0.f && rest < 0.f) return sum - 1.f;
        }
        return sum;
    }

    // the steps of eight values, a byte each
    __device__ __forceinline__ uint2 steps(const float (&y)[kVec]) const
    {
        if (!finite) return make_uint2(0u, 0u);
        float z[kVec], sum[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) z[i] = y[i];
        if (factor != 1.f) {
            asm volatile("");  // a branch, not eight predicated products for every row
#pragma unroll
            for (int i = 0; i < kVec; ++i) z[i] *= factor;
        }
        if constexpr (kForm == kOneProduct) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) sum[i] = fmaf(z[i], hi, kWhole);
        } else {
            const uint64_t hi2 = pack2(hi, hi), lo2 = pack2(lo, lo), whole2 = pack2(kWhole, kWhole);
            float off = 0.f;  // the largest distance from a whole number
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) {
                const uint64_t y2 = pack2(z[2 * i], z[2 * i + 1]), t2 = fma2(y2, hi2, mul2(y2, lo2));
                const uint64_t sum2 = add2(t2, whole2);
                unpack2(sum2, sum[2 * i], sum[2 * i + 1]);
                if constexpr (kForm == kTiesAndNear) {
                    const uint64_t step2 = add2(sum2, pack2(-kWhole, -kWhole));
                    float d[2];
                    unpack2(fma2(step2, pack2(-1.f, -1.f), t2), d[0], d[1]);
                    off = max3_abs(off, d[0], d[1]);
                }
            }
            if constexpr (kForm == kTiesAndNear) {
                if (off == 0.5f) {
                    asm volatile("");
#pragma unroll
                    for (int i = 0; i < kVec; ++i) sum[i] = past_tie(z[i]);
                }
            }
        }
        uint32_t b[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) b[i] = __float_as_uint(sum[i]);
        const uint32_t p0 = __byte_perm(b[0], b[1], 0x0040), p1 = __byte_perm(b[2], b[3], 0x0040);
        const uint32_t p2 = __byte_perm(b[4], b[5], 0x0040), p3 = __byte_perm(b[6], b[7], 0x0040);
        return make_uint2(__byte_perm(p0, p1, 0x5410), __byte_perm(p2, p3, 0x5410));
    }
};

template <int kOp, typename T>
using RowQuantiser = Quantiser<quotient_form<kOp, T>()>;

template <bool kAligned, int kForm>
__device__ __forceinline__ void store_q(int8_t *p, int n, const float (&y)[kVec], const Quantiser<kForm> &qz)
{
    const uint2 b = qz.steps(y);
    if (kAligned && n == kVec && DGEMM_CHECK((reinterpret_cast<uintptr_t>(p) & 7u) == 0)) {
        *reinterpret_cast<uint2 *>(p) = b;
        return;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (i < n) p[i] = static_cast<int8_t>((i < 4 ? b.x : b.y) >> (8 * (i & 3)));
}

// ---- reductions over the threads of a row

// over a warp (kWarp) or the whole block
template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float *shared)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (kWarp) return v;
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < (blockDim.x >> 5) ? shared[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

template <bool kWarp>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *shared)
{
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if constexpr (kWarp) return v;
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < (blockDim.x >> 5) ? shared[threadIdx.x & 31] : 0u;
    return __reduce_max_sync(0xFFFFFFFFu, v);
}

// Both at once: one meeting of the row's threads instead of two.
template <bool kWarp>
__device__ __forceinline__ void row_sum_max(float &sum, uint32_t &most, float *s_sum, uint32_t *s_max)
{
    most = __reduce_max_sync(0xFFFFFFFFu, most);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if constexpr (kWarp) return;
    if ((threadIdx.x & 31) == 0) {
        s_sum[threadIdx.x >> 5] = sum;
        s_max[threadIdx.x >> 5] = most;
    }
    __syncthreads();
    const bool in = (threadIdx.x & 31) < (blockDim.x >> 5);
    sum = in ? s_sum[threadIdx.x & 31] : 0.f;
    most = __reduce_max_sync(0xFFFFFFFFu, in ? s_max[threadIdx.x & 31] : 0u);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
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

// The values before the norm / quantisation: x, the residual's sum, or the
// gated product.
template <int kOp, typename T>
__device__ __forceinline__ void combine(const RowParams &p, const Raw<T> &x, const Raw<T> &y, float (&v)[kVec])
{
    unpack(x, v);
    if constexpr (!has_second(kOp)) return;
    float u[kVec];
    unpack(y, u);
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = kOp == kOpNorm ? v[i] + u[i] : silu(v[i]) * u[i];
}

template <int kOp, typename T, bool kAligned>
__device__ __forceinline__ Raw<T> load_second(const RowParams &p, int64_t row, int64_t c, int n)
{
    if constexpr (has_second(kOp)) return load_raw<T, kAligned>(static_cast<const T *>(p.y) + row * p.ldy + c, n);
    return Raw<T>{};
}

template <typename T, bool kAligned>
__device__ __forceinline__ void load_gamma(const RowParams &p, int64_t c, int n, float (&g)[kVec])
{
    if (p.gamma_f32)
        unpack(load_raw<float, kAligned, true>(static_cast<const float *>(p.gamma) + c, n), g);
    else
        unpack(load_raw<T, kAligned, true>(static_cast<const T *>(p.gamma) + c, n), g);
}

__device__ __forceinline__ int vec_len(int64_t cols, int64_t c)
{
    const int64_t left = cols - c;
    return left >= kVec ? kVec : left > 0 ? static_cast<int>(left) : 0;
}

// 1 / sqrt(mean + eps) from the sum of a row's squares.  A sum past FP32's range
// marks the row like a NaN in it.
__device__ __forceinline__ float norm_factor(float ss, int64_t cols, float eps)
{
    return ss < __uint_as_float(0x7F800000u) ? rsqrtf(ss / static_cast<float>(cols) + eps) : __uint_as_float(0x7FC00000u);
}

// A row held by its threads, from its values before the norm / quantisation to
// H, the scale and q.  weights(j, g) gives the norm's weights of vector j.
template <int kOp, typename T, bool kAligned, bool kWarp, int kVecs, typename W>
__device__ __forceinline__ void finish_row(const RowParams &p, int64_t row, int t, int threads, const int (&n)[kVecs],
                                           float (&v)[kVecs][kVec], const W &weights, float *s_sum, uint32_t *s_max)
{
    const int cols = static_cast<int>(p.cols);
    float amax = 0.f, rstd = 1.f;
    uint32_t most;
    if constexpr (is_norm(kOp)) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int c = (j * threads + t) * kVec;
            if (p.h) store_vec<T, kAligned>(static_cast<T *>(p.h) + row * p.ldh + c, n[j], v[j]);
#pragma unroll
            for (int i = 0; i < kVec; ++i) ss = fmaf(v[j][i], v[j][i], ss);
        }
        // neither the weights nor the maximum wait for the sum, and the steps
        // need no 1 / sqrt at all: it cancels in y / a
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            float g[kVec];
            weights(j, g);
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[j][i] *= g[i];
            amax = max_abs(amax, v[j]);
        }
        most = __float_as_uint(amax) & 0x7FFFFFFFu;
        row_sum_max<kWarp>(ss, most, s_sum, s_max);
        rstd = norm_factor(ss, cols, p.eps);
    } else {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) amax = max_abs(amax, v[j]);
        most = row_max<kWarp>(__float_as_uint(amax) & 0x7FFFFFFFu, s_max);
    }
    const RowQuantiser<kOp, T> qz(most, rstd);
    if (t == 0) p.scale[row] = qz.scale;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int c = (j * threads + t) * kVec;
        if (DGEMM_CHECK(n[j] == 0 || (row >= 0 && row < p.rows && c + n[j] <= cols)))
            store_q<kAligned>(p.q + row * p.ldq + c, n[j], v[j], qz);
    }
}

// One row a block of at most kMost threads, or (kMost == 32) a warp, four rows
// a block: the row's values stay in registers, kVecs vectors a thread.
template <int kOp, typename T, bool kAligned, int kMost, int kVecs>
__global__ void __launch_bounds__(kMost < 128 ? 128 : kMost, kMost < 128 ? 6 : 1024 / kMost) rows_kernel(const RowParams p)
{
    constexpr bool kWarp = kMost == 32;
    const int threads = kWarp ? 32 : static_cast<int>(blockDim.x);
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    chain_wait();
    chain_next();
    const int64_t row = kWarp ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= p.rows) return;  // (whole warps; a block of one row never leaves here)
    const int t = static_cast<int>(kWarp ? threadIdx.x & 31 : threadIdx.x);
    const int cols = static_cast<int>(p.cols);
    int n[kVecs];  // this thread's elements of each vector, from column (j * threads + t) * kVec
    Raw<T> x[kVecs], y[kVecs], w[kVecs];
    // the norm's weights in the rows' type come beside the row where registers
    // are left for them
    const bool early = is_norm(kOp) && kVecs <= 2 && (sizeof(T) == 4 || !p.gamma_f32);
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int c = (j * threads + t) * kVec;
        n[j] = max(0, min(kVec, cols - c));
        x[j] = load_raw<T, kAligned>(static_cast<const T *>(p.x) + row * p.ldx + c, n[j]);
        y[j] = load_second<kOp, T, kAligned>(p, row, c, n[j]);
    }
    if (early) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
            w[j] = load_raw<T, kAligned, true>(static_cast<const T *>(p.gamma) + (j * threads + t) * kVec, n[j]);
    }
    float v[kVecs][kVec];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) combine<kOp>(p, x[j], y[j], v[j]);
    finish_row<kOp, T, kAligned, kWarp, kVecs>(
        p, row, t, threads, n, v,
        [&](int j, float(&g)[kVec]) {
            if (early)
                unpack(w[j], g);
            else
                load_gamma<T, kAligned>(p, (j * threads + t) * kVec, n[j], g);
        },
        s_sum, s_max);
}

// 16 bytes from global to shared memory, of which `bytes` are read and the rest
// are zeros, without a register in between.
__device__ __forceinline__ void copy_async16(uint4 *dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(bytes)
                 : "memory");
}

// As rows_kernel for many rows of a 16-bit type: a block (warp) takes one row
// after another, and while it works on one, the next is on its way to shared
// memory.  Each thread fetches the vectors that it will use itself, so that no
// thread waits for another's; a slot is free again as soon as its thread has
// read it.  The norm's weights (in the rows' type) stay in shared memory too.
// 8192 rows of bf16, rows_kernel and this one: quantize of 8192 33.0 and 30.7
// us, of 12288 58.9 and 46.1; swiglu of 8192 52.7 and 50.5, of 12288 85.4 and
// 74.4; norm of 8192 43.6 and 39.4, of 12288 78.3 and 59.6.  The norm with
// residual, which stores H too, loses (of 8192 71.3 and 85.8) except where an SM
// holds one row at a time, from 16385 columns on: 4096 rows of 16400 97.2 and 80.7,
// of 20000 105.3 and 89.4, of 24576 119.7 and 116.7, 700 of 28672 29.6 and 24.9;
// the end of that range is even (2048 of 32768 81.8 and 83.3).
constexpr bool is_piped(int op, int most_threads)
{
    return op != kOpNorm || most_threads == 1024;
}

template <int kOp, typename T, int kMost, int kVecs>
__global__ void __launch_bounds__(kMost < 128 ? 128 : kMost, kMost < 128 ? 6 : 1024 / kMost)
    piped_rows_kernel(const RowParams p)
{
    static_assert(sizeof(T) == 2, "a vector is one 16-byte word");
    constexpr bool kWarp = kMost == 32;
    constexpr int kInputs = has_second(kOp) ? 2 : 1;
    extern __shared__ uint4 slots[];  // [input, then weights][vector][thread of the block]
    const int threads = kWarp ? 32 : static_cast<int>(blockDim.x);
    __shared__ float s_sum[2][32];  // by turns, so that one barrier a row is enough
    __shared__ uint32_t s_max[2][32];
    chain_wait();
    chain_next();
    const int64_t first = kWarp ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = kWarp ? static_cast<int64_t>(gridDim.x) * 4 : gridDim.x;
    const int t = static_cast<int>(kWarp ? threadIdx.x & 31 : threadIdx.x);
    const int cols = static_cast<int>(p.cols);
    int n[kVecs];
    auto slot = [&](int input, int j) { return slots + (input * kVecs + j) * static_cast<int>(blockDim.x) + threadIdx.x; };
    const bool keep = is_norm(kOp) && !p.gamma_f32;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int c = (j * threads + t) * kVec;
        n[j] = max(0, min(kVec, cols - c));
        if (keep) copy_async16(slot(kInputs, j), static_cast<const T *>(p.gamma) + (n[j] ? c : 0), n[j] * 2);
    }
    auto fetch = [&](int64_t row) {
        if (row >= p.rows) return;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int c = n[j] ? (j * threads + t) * kVec : 0, bytes = n[j] * 2;
            copy_async16(slot(0, j), static_cast<const T *>(p.x) + row * p.ldx + c, bytes);
            if constexpr (kInputs == 2) copy_async16(slot(1, j), static_cast<const T *>(p.y) + row * p.ldy + c, bytes);
        }
    };
    fetch(first);
    int turn = 0;
    for (int64_t row = first; row < p.rows; row += step) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        float v[kVecs][kVec];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            Raw<T> x, y{};
            x.w[0] = *slot(0, j);
            if constexpr (kInputs == 2) y.w[0] = *slot(1, j);
            combine<kOp>(p, x, y, v[j]);
        }
        fetch(row + step);
        finish_row<kOp, T, true, kWarp, kVecs>(
            p, row, t, threads, n, v,
            [&](int j, float(&g)[kVec]) {
                if (keep) {
                    Raw<T> w;
                    w.w[0] = *slot(kInputs, j);
                    unpack(w, g);
                } else {
                    load_gamma<T, true>(p, (j * threads + t) * kVec, n[j], g);
                }
            },
            s_sum[turn], s_max[turn]);
        turn ^= 1;
    }
}

// The norm with an eps below this comes here whatever the row's length.  The squares
// of a row of small values leave FP32's range; from 2^-100 on, what is lost of them
// is nothing beside eps.  Without, a row of values below 2^-40, some of whose squares
// would be lost, is multiplied by 2^90, exactly, and eps by its square.  (The
// squares of 2^-149 and 2^-40 become 2^-118 and 2^100.)  A row of zeros stays one,
// even with an eps of 0.
// It costs passes over the row (norm with residual, bf16, eps of 1e-6 and of 0: 8192
// rows of 1024 9.4 and 17.3 us, of 8192 71 and 210); in the kernels above the branch
// alone would cost every norm its registers (32 values a thread in 64 of them: up
// to 152 bytes spilled).
constexpr float kSmallEps = 0x1p-100f, kSmallRow = 0x1p-40f, kSmallFactor = 0x1p90f;

// Rows longer than one block's registers: the same three steps, each reading
// the row again (the second and third mostly from L2).  H is stored in the
// last pass, so it may be the buffer of X or of the residual here too.
// Two blocks an SM, so that one reads while the other waits, even where that
// spills a few registers (2048 rows of 40000, one block and two: norm bf16 146
// and 113 us, with residual 231 and 190, swiglu 145 and 115, quantize FP32 131 and
// 112); not for element loads without weights, which lose by it (swiglu FP32 at
// an odd pitch 352 and 391).
template <int kOp, typename T, bool kAligned>
__global__ void __launch_bounds__(1024, kAligned || is_norm(kOp) ? 2 : 0) long_rows_kernel(const RowParams p)
{
    const int step = static_cast<int>(blockDim.x) * kVec;
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    chain_wait();
    chain_next();
    const int64_t row = blockIdx.x;
    auto value = [&](int64_t c, int n, float (&v)[kVec]) {
        combine<kOp>(p, load_raw<T, kAligned>(static_cast<const T *>(p.x) + row * p.ldx + c, n),
                     load_second<kOp, T, kAligned>(p, row, c, n), v);
    };
    float rstd = 1.f, amax = 0.f, factor = 1.f;
    if constexpr (is_norm(kOp)) {
        float ss = 0.f, eps = p.eps;
        bool zeros = false;
        if (eps < kSmallEps) {
            float largest = 0.f;
            for (int64_t c = static_cast<int64_t>(threadIdx.x) * kVec; c < p.cols; c += step) {
                float v[kVec];
                value(c, vec_len(p.cols, c), v);
                largest = max_abs(largest, v);
            }
            largest = __uint_as_float(row_max<false>(__float_as_uint(largest) & 0x7FFFFFFFu, s_max));
            zeros = largest == 0.f;
            if (largest < kSmallRow) {
                factor = kSmallFactor;
                eps = eps * kSmallFactor * kSmallFactor;  // (the factors' own product is past FP32)
            }
        }
        for (int64_t c = static_cast<int64_t>(threadIdx.x) * kVec; c < p.cols; c += step) {
            float v[kVec];
            value(c, vec_len(p.cols, c), v);
#pragma unroll
            for (int i = 0; i < kVec; ++i) ss = fmaf(v[i] * factor, v[i] * factor, ss);
        }
        ss = row_sum<false>(ss, s_sum);
        rstd = zeros ? 0.f : norm_factor(ss, p.cols, eps);
    }
    auto weigh = [&](int64_t c, int n, float (&v)[kVec]) {
        if constexpr (is_norm(kOp)) {
            float g[kVec];
            load_gamma<T, kAligned>(p, c, n, g);
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[i] *= factor * g[i];
        }
    };
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * kVec; c < p.cols; c += step) {
        float v[kVec];
        const int n = vec_len(p.cols, c);
        value(c, n, v);
        weigh(c, n, v);
        amax = max_abs(amax, v);
    }
    const RowQuantiser<kOp, T> qz(row_max<false>(__float_as_uint(amax) & 0x7FFFFFFFu, s_max), rstd);
    if (threadIdx.x == 0) p.scale[row] = qz.scale;
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * kVec; c < p.cols; c += step) {
        float v[kVec];
        const int n = vec_len(p.cols, c);
        value(c, n, v);
        // the last read of this thread's elements: H may now overwrite an input
        if constexpr (is_norm(kOp))
            if (p.h) store_vec<T, kAligned>(static_cast<T *>(p.h) + row * p.ldh + c, n, v);
        weigh(c, n, v);
        if (DGEMM_CHECK(c + n <= p.cols)) store_q<kAligned>(p.q + row * p.ldq + c, n, v, qz);
    }
}

// The int8 value whose byte (with the sign bit flipped, so that it is v + 128)
// is the k-th of u: under the exponent of 2^23 the byte is the number 2^23 +
// v + 128, exactly.
__device__ __forceinline__ float byte_to_f32(uint32_t u, int k)
{
    return __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + k)) - 8388736.f;
}

// A thread's piece: two vectors of one row, 16 bytes of q.
constexpr int kPiece = 2 * kVec;

// `pieces` to a row; rows * pieces is below 2^31.  q and x on 16-byte rows.
template <typename T>
__global__ void __launch_bounds__(256)
    dequantize_kernel(uint32_t rows, int64_t cols, const int8_t *q, int64_t ldq,
                      const float *scale, T *x, int64_t ldx, uint32_t pieces)
{
    chain_wait();
    chain_next();
    const uint32_t total = rows * pieces;
    for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < total; i += gridDim.x * 256u) {
        const uint32_t row = i / pieces;
        const int64_t c = static_cast<int64_t>(i - row * pieces) * kPiece;
        const int64_t left = cols - c;
        const int8_t *src = q + row * ldq + c;
        T *dst = x + row * ldx + c;
        const float s = load_f32(scale + row);
        alignas(16) int8_t e[kPiece];
        if (left >= kPiece) {
            *reinterpret_cast<uint4 *>(e) = load_v4_stream(src);
        } else {
#pragma unroll
            for (int k = 0; k < kPiece; ++k) e[k] = k < left ? src[k] : static_cast<int8_t>(0);
        }
        const uint32_t *w = reinterpret_cast<const uint32_t *>(e);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[kVec];
#pragma unroll
            for (int k = 0; k < kVec; ++k) v[k] = byte_to_f32(w[h * 2 + k / 4] ^ 0x80808080u, k & 3) * s;
            const int64_t l = left - h * kVec;
            const int n = l >= kVec ? kVec : l > 0 ? static_cast<int>(l) : 0;
            if (DGEMM_CHECK((row < rows && c + h * kVec + n <= cols) || n == 0))
                store_vec<T, true>(dst + h * kVec, n, v);
        }
    }
}

// Rows of any alignment: element by element, consecutive threads on
// consecutive columns; blocks of 1024 columns, rows over the grid's other
// dimension.
constexpr int kAnyCols = 1024;

template <typename T>
__global__ void __launch_bounds__(256)
    dequantize_any_kernel(int64_t rows, int64_t cols, const int8_t *q, int64_t ldq,
                          const float *scale, T *x, int64_t ldx)
{
    chain_wait();
    chain_next();
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kAnyCols + threadIdx.x;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const float s = load_f32(scale + row);
        // all of them loaded before the first store, which the compiler has to take
        // for a store into q
        int8_t v[kAnyCols / 256];
#pragma unroll
        for (int k = 0; k < kAnyCols / 256; ++k) {
            const int64_t c = c0 + k * 256;
            v[k] = c < cols ? q[row * ldq + c] : static_cast<int8_t>(0);
        }
#pragma unroll
        for (int k = 0; k < kAnyCols / 256; ++k) {
            const int64_t c = c0 + k * 256;
            if (c < cols && DGEMM_CHECK(row >= 0)) x[row * ldx + c] = from_f32<T>(static_cast<float>(v[k]) * s);
        }
    }
}

// ---- host side

template <int kOp, int kVecs>
constexpr size_t piped_smem(unsigned threads)
{
    return static_cast<size_t>((has_second(kOp) ? 2 : 1) + (is_norm(kOp) ? 1 : 0)) * kVecs * threads * 16;
}

// Blocks of this many threads of piped_rows_kernel that the current device runs at
// once, cached; 0 if it cannot run.
template <int kOp, typename T, int kMost, int kVecs>
int piped_blocks(unsigned threads)
{
    constexpr int kMaxDevices = 64;
    static std::atomic<int> cached[kMaxDevices][33];  // blocks + 1, by warps
    int dev = 0;
    if (threads > 1024 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    std::atomic<int> &c = cached[dev][threads / 32];
    int blocks = c.load(std::memory_order_relaxed) - 1;
    if (blocks >= 0) return blocks;
    auto kernel = piped_rows_kernel<kOp, T, kMost, kVecs>;
    int sms = 0, per_sm = 0;
    const bool ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(piped_smem<kOp, kVecs>(kMost < 128 ? 128 : kMost))) == cudaSuccess &&
                    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
                    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, static_cast<int>(threads),
                                                                  piped_smem<kOp, kVecs>(threads)) == cudaSuccess;
    blocks = ok ? sms * per_sm : 0;
    cudaGetLastError();  // a failed query leaves no sticky error behind
    c.store(blocks + 1, std::memory_order_relaxed);
    return blocks;
}

template <int kOp, typename T, bool kAligned, int kMost, int kVecs>
void launch_rows(const RowParams &p, cudaStream_t stream)
{
    const int64_t vecs = (p.cols - 1) / kVec + 1;
    // threads: a warp for each 32 * kVecs vectors
    const unsigned threads = kMost == 32 ? 128u : static_cast<unsigned>((vecs + 32 * kVecs - 1) / (32 * kVecs) * 32);
    const unsigned grid = static_cast<unsigned>(kMost == 32 ? (p.rows + 3) / 4 : p.rows);
    if constexpr (is_piped(kOp, kMost) && kAligned && sizeof(T) == 2 && kVecs == 4) {
        const int resident = piped_blocks<kOp, T, kMost, kVecs>(threads);
        if (resident > 0 && grid > static_cast<unsigned>(resident)) {
            launch_chained(piped_rows_kernel<kOp, T, kMost, kVecs>, static_cast<unsigned>(resident), threads,
                           piped_smem<kOp, kVecs>(threads), stream, 1, p);
            return;
        }
    }
    launch_chained(rows_kernel<kOp, T, kAligned, kMost, kVecs>, grid, threads, 0, stream, 1, p);
}

// Four vectors a thread where there are rows enough to fill the SMs; work that
// is resident at once with one vector a thread (two, for rows of more than
// 8192) is spread that wide instead.  Through the norm with residual, bf16,
// wide against four vectors: one row of 4096 2.4 and 4.7 us, 333 rows of 4096
// 3.3 and 3.8, 333 rows of 8192 (not resident) 5.7 and 4.9.  More rows of four
// vectors than run at once go to piped_rows_kernel.
template <int kOp, typename T, bool kAligned>
const char *launch_rows_by_length(const RowParams &p, cudaStream_t stream)
{
    const int64_t vecs = (p.cols - 1) / kVec + 1;
    const int64_t wide = p.rows * (vecs <= 1024 ? vecs : (vecs + 1) / 2);  // threads
    const bool few = wide <= kResident;
    if (vecs > 4096 || (is_norm(kOp) && p.eps < kSmallEps)) {
        // (shorter rows, there for their eps: four vectors a thread)
        const unsigned threads = vecs > 4096 ? 1024u : static_cast<unsigned>((vecs + 127) / 128 * 32);
        launch_chained(long_rows_kernel<kOp, T, kAligned>, static_cast<unsigned>(p.rows), threads, 0, stream, 1, p);
        return "i8_long_rows";
    }
    if (few && vecs > 32 && vecs <= 1024)
        launch_rows<kOp, T, kAligned, 1024, 1>(p, stream);
    else if (few && vecs > 1024 && vecs <= 2048)
        launch_rows<kOp, T, kAligned, 1024, 2>(p, stream);
    else if (vecs <= 32)
        launch_rows<kOp, T, kAligned, 32, 1>(p, stream);
    else if (vecs <= 64)
        launch_rows<kOp, T, kAligned, 32, 2>(p, stream);
    else if (vecs <= 128)
        launch_rows<kOp, T, kAligned, 32, 4>(p, stream);
    else if (vecs <= 1024)
        launch_rows<kOp, T, kAligned, 256, 4>(p, stream);
    else if (vecs <= 2048)
        launch_rows<kOp, T, kAligned, 512, 4>(p, stream);
    else
        launch_rows<kOp, T, kAligned, 1024, 4>(p, stream);
    return is_norm(kOp) ? "i8_rmsnorm_rows" : kOp == kOpSwiglu ? "i8_swiglu_rows" : "i8_quantize_rows";
}

bool aligned(const void *p, int64_t ld, int64_t elem, int64_t to)
{
    return reinterpret_cast<uintptr_t>(p) % to == 0 && (ld * elem) % to == 0;
}

// Vector accesses need every operand's rows to start on their vector's
// boundary: 16 bytes, or 8 for q.
template <int kOp, typename T>
const char *launch_rows_typed(const RowParams &p, cudaStream_t stream)
{
    constexpr int64_t e = sizeof(T);
    const bool ok = aligned(p.x, p.ldx, e, 16) && (!p.y || aligned(p.y, p.ldy, e, 16)) &&
                    (!p.h || aligned(p.h, p.ldh, e, 16)) && (!p.gamma || aligned(p.gamma, 0, e, 16)) &&
                    aligned(p.q, p.ldq, 1, 8);
    return ok ? launch_rows_by_length<kOp, T, true>(p, stream) : launch_rows_by_length<kOp, T, false>(p, stream);
}

template <int kOp>
const char *launch_rows_op(int type, const RowParams &p, cudaStream_t stream)
{
    switch (type) {
    case DGEMM_TYPE_F32: return launch_rows_typed<kOp, float>(p, stream);
    case DGEMM_TYPE_F16: return launch_rows_typed<kOp, __half>(p, stream);
    case DGEMM_TYPE_BF16: return launch_rows_typed<kOp, __nv_bfloat16>(p, stream);
    default: return nullptr;
    }
}

template <typename T>
const char *launch_dequantize_typed(int64_t rows, int64_t cols, const int8_t *q, int64_t ldq, const float *scale,
                                    void *x, int64_t ldx, cudaStream_t stream, const DeviceInfo &dev)
{
    T *out = static_cast<T *>(x);
    if (!aligned(q, ldq, 1, 16) || !aligned(x, ldx, sizeof(T), 16)) {
        const int64_t across = (cols - 1) / kAnyCols + 1;
        if (across > INT32_MAX) return nullptr;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(across), static_cast<unsigned>(rows < 65535 ? rows : 65535));
        cfg.blockDim = dim3(256);
        cfg.stream = stream;
        cudaLaunchAttribute attr = chained_attribute();
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        cudaLaunchKernelEx(&cfg, dequantize_any_kernel<T>, rows, cols, q, ldq, scale, out, ldx);
        return "i8_dequantize_any";
    }
    const int64_t pieces = (cols - 1) / kPiece + 1;
    if (pieces > INT32_MAX) return nullptr;
    const int64_t cap = static_cast<int64_t>(dev.sm_count) * 32;
    const int64_t most = INT32_MAX / pieces;  // rows of one launch: 32-bit piece numbers
    for (int64_t r = 0; r < rows; r += most) {
        const int64_t n = rows - r < most ? rows - r : most;
        const int64_t want = (n * pieces + 255) / 256;
        const unsigned grid = static_cast<unsigned>(want < cap ? want : cap);
        launch_chained(dequantize_kernel<T>, grid, 256, 0, stream, 1, static_cast<uint32_t>(n), cols, q + r * ldq, ldq,
                       scale + r, out + r * ldx, ldx, static_cast<uint32_t>(pieces));
    }
    return "i8_dequantize";
}

}  // namespace

const char *launch_quantize_i8(int64_t rows, int64_t cols, const void *x, int64_t ldx, int type, int8_t *q,
                               int64_t ldq, float *scale, cudaStream_t stream)
{
    RowParams p{};
    p.rows = rows;
    p.cols = cols;
    p.x = x;
    p.ldx = ldx;
    p.q = q;
    p.ldq = ldq;
    p.scale = scale;
    return launch_rows_op<kOpQuantize>(type, p, stream);
}

const char *launch_rmsnorm_i8(int64_t rows, int64_t cols, const void *x, int64_t ldx, const void *residual,
                              int64_t ldr, const void *gamma, bool gamma_f32, float eps, int type, void *h,
                              int64_t ldh, int8_t *q, int64_t ldq, float *scale, cudaStream_t stream)
{
    RowParams p{};
    p.rows = rows;
    p.cols = cols;
    p.x = x;
    p.ldx = ldx;
    p.y = residual;
    p.ldy = ldr;
    p.gamma = gamma;
    p.gamma_f32 = gamma_f32 ? 1 : 0;
    p.eps = eps;
    p.h = h;
    p.ldh = ldh;
    p.q = q;
    p.ldq = ldq;
    p.scale = scale;
    return residual ? launch_rows_op<kOpNorm>(type, p, stream) : launch_rows_op<kOpNormAlone>(type, p, stream);
}

const char *launch_swiglu_i8(int64_t rows, int64_t cols, const void *g, int64_t ldg, const void *u, int64_t ldu,
                             int type, int8_t *q, int64_t ldq, float *scale, cudaStream_t stream)
{
    RowParams p{};
    p.rows = rows;
    p.cols = cols;
    p.x = g;
    p.ldx = ldg;
    p.y = u;
    p.ldy = ldu;
    p.q = q;
    p.ldq = ldq;
    p.scale = scale;
    return launch_rows_op<kOpSwiglu>(type, p, stream);
}

const char *launch_dequantize_i8(int64_t rows, int64_t cols, const int8_t *q, int64_t ldq, const float *scale,
                                 void *x, int64_t ldx, int type, cudaStream_t stream, const DeviceInfo &dev)
{
    switch (type) {
    case DGEMM_TYPE_F32: return launch_dequantize_typed<float>(rows, cols, q, ldq, scale, x, ldx, stream, dev);
    case DGEMM_TYPE_F16: return launch_dequantize_typed<__half>(rows, cols, q, ldq, scale, x, ldx, stream, dev);
    case DGEMM_TYPE_BF16:
        return launch_dequantize_typed<__nv_bfloat16>(rows, cols, q, ldq, scale, x, ldx, stream, dev);
    default: return nullptr;
    }
}

}  // namespace dgemm

DGEMM_DEFINE_CHECK_READER(check_status_i8_rows)
