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
// written once, with a few operations a byte.  A row needs two results over
// all of its elements before the first q can be written (the norm's sum of
// squares, then the maximum), so the row's values stay in registers between:
// a group of kThreads threads holds a row, kVecs vectors of 8 elements a
// thread.  Rows longer than the registers of one block (32768 elements) are
// read again from memory for each pass.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dgemm.h"
#include "internal.h"

#define DGEMM_UNIT 6
#include "checked.cuh"

namespace dgemm {
namespace {

constexpr int kVec = 8;  // elements of one vector: 16 bytes of a 16-bit type, 8 bytes of q

enum { kOpQuantize = 0, kOpNorm = 1, kOpSwiglu = 2 };

struct RowParams {
    int64_t rows, cols;
    const void *x;  // the row to quantise / norm; the gate of swiglu
    int64_t ldx;
    const void *y;  // residual (norm; may be null) or the up rows (swiglu)
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

// kAligned: the vector starts on a 16-byte boundary (sizeof(T) == 2) or two
// (FP32); n < kVec, or an unaligned operand, takes element loads.  Elements
// past n are 0.
template <typename T, bool kAligned>
__device__ __forceinline__ void load_vec(const T *p, int n, float (&v)[kVec])
{
    if (kAligned && n == kVec) {
        constexpr int kWords = kVec * sizeof(T) / 16;
        uint4 w[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
        const T *e = reinterpret_cast<const T *>(w);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = to_f32(e[i]);
        return;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
}

template <typename T, bool kAligned>
__device__ __forceinline__ void store_vec(T *p, int n, const float (&v)[kVec])
{
    if (kAligned && n == kVec && DGEMM_CHECK((reinterpret_cast<uintptr_t>(p) & 15u) == 0)) {
        alignas(16) T e[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) e[i] = from_f32<T>(v[i]);
#pragma unroll
        for (int i = 0; i < static_cast<int>(kVec * sizeof(T) / 16); ++i)
            reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(e)[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (i < n) p[i] = from_f32<T>(v[i]);
}

// ---- the quantisation's scale and steps

// A row's largest |y| as the bits of a non-negative float: unsigned order is
// the order of the values, with infinities and then NaNs above every finite
// value, so one integer maximum also finds a row that is not finite.
__device__ __forceinline__ uint32_t abs_bits(float v)
{
    return __float_as_uint(v) & 0x7FFFFFFFu;
}

struct Quantiser {
    float scale, pre, inv;
    bool finite;

    __device__ __forceinline__ explicit Quantiser(uint32_t amax_bits)
    {
        const float a = __uint_as_float(amax_bits);
        finite = amax_bits < 0x7F800000u;
        scale = finite ? a / 127.f : __uint_as_float(0x7FC00000u);
        // 127 / a leaves FP32's range below a = 2^-121; such rows are first
        // multiplied by a power of two, which is exact
        pre = a < 0x1p-100f ? 0x1p100f : 1.f;
        inv = finite && a > 0.f ? 127.f / (a * pre) : 0.f;
    }

    // rint(y * 127 / a), ties to even; within [-127, 127] because |y| <= a,
    // and a product that rounds up past 127 still rounds to 127
    __device__ __forceinline__ int32_t step(float y) const
    {
        return finite ? __float2int_rn(y * pre * inv) : 0;
    }
};

template <bool kAligned>
__device__ __forceinline__ void store_q(int8_t *p, int n, const float (&y)[kVec], const Quantiser &qz)
{
    uint32_t b[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) b[i] = static_cast<uint32_t>(qz.step(y[i])) & 0xFFu;
    if (kAligned && n == kVec && DGEMM_CHECK((reinterpret_cast<uintptr_t>(p) & 7u) == 0)) {
        const uint32_t lo = b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
        const uint32_t hi = b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24;
        *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
        return;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (i < n) p[i] = static_cast<int8_t>(b[i]);
}

// ---- reductions over the threads of a row

template <int kThreads>
__device__ __forceinline__ float row_sum(float v, float *shared)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (kThreads == 32) return v;
    constexpr int kWarps = kThreads / 32;
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    v = static_cast<int>(threadIdx.x & 31) < kWarps ? shared[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

template <int kThreads>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *shared)
{
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if constexpr (kThreads == 32) return v;
    constexpr int kWarps = kThreads / 32;
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    v = static_cast<int>(threadIdx.x & 31) < kWarps ? shared[threadIdx.x & 31] : 0u;
    return __reduce_max_sync(0xFFFFFFFFu, v);
}

// g / (1 + exp(-g)).  The fast division is within 2 ulp up to 2^126 and gives
// 0 above, where the quotient is below 1e-35 anyway.
__device__ __forceinline__ float silu(float g)
{
    return __fdividef(g, 1.f + __expf(-g));
}

// The values before the norm / quantisation of the vector at column c: x, the
// residual's sum, or the gated product.
template <int kOp, typename T, bool kAligned>
__device__ __forceinline__ void load_row_vec(const RowParams &p, int64_t row, int64_t c, int n, float (&v)[kVec])
{
    load_vec<T, kAligned>(static_cast<const T *>(p.x) + row * p.ldx + c, n, v);
    if constexpr (kOp == kOpNorm) {
        if (p.y) {
            float r[kVec];
            load_vec<T, kAligned>(static_cast<const T *>(p.y) + row * p.ldy + c, n, r);
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[i] += r[i];
        }
    }
    if constexpr (kOp == kOpSwiglu) {
        float u[kVec];
        load_vec<T, kAligned>(static_cast<const T *>(p.y) + row * p.ldy + c, n, u);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = silu(v[i]) * u[i];
    }
}

template <typename T, bool kAligned>
__device__ __forceinline__ void load_gamma(const RowParams &p, int64_t c, int n, float (&g)[kVec])
{
    if (p.gamma_f32)
        load_vec<float, kAligned>(static_cast<const float *>(p.gamma) + c, n, g);
    else
        load_vec<T, kAligned>(static_cast<const T *>(p.gamma) + c, n, g);
}

__device__ __forceinline__ int vec_len(int64_t cols, int64_t c)
{
    const int64_t left = cols - c;
    return left >= kVec ? kVec : left > 0 ? static_cast<int>(left) : 0;
}

// One row a block (kThreads > 32) or a warp (kThreads == 32, four rows a
// block): the row's values stay in registers, kVecs vectors a thread.
template <int kOp, typename T, bool kAligned, int kThreads, int kVecs>
__global__ void __launch_bounds__(kThreads < 128 ? 128 : kThreads) rows_kernel(const RowParams p)
{
    constexpr int kRowsPerBlock = kThreads < 128 ? 128 / kThreads : 1;
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + threadIdx.x / kThreads;
    if (row >= p.rows) return;  // (whole warps; a block of one row never leaves here)
    const int t = static_cast<int>(threadIdx.x % kThreads);
    float v[kVecs][kVec];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int64_t c = static_cast<int64_t>(j * kThreads + t) * kVec;
        load_row_vec<kOp, T, kAligned>(p, row, c, vec_len(p.cols, c), v[j]);
    }
    uint32_t amax = 0;
    if constexpr (kOp == kOpNorm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int64_t c = static_cast<int64_t>(j * kThreads + t) * kVec;
            if (p.h) store_vec<T, kAligned>(static_cast<T *>(p.h) + row * p.ldh + c, vec_len(p.cols, c), v[j]);
#pragma unroll
            for (int i = 0; i < kVec; ++i) ss = fmaf(v[j][i], v[j][i], ss);
        }
        ss = row_sum<kThreads>(ss, s_sum);
        // a sum of squares past FP32's range marks the row like a NaN in it
        if (!(ss < __uint_as_float(0x7F800000u))) amax = 0x7FC00000u;
        const float rstd = rsqrtf(ss / static_cast<float>(p.cols) + p.eps);
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int64_t c = static_cast<int64_t>(j * kThreads + t) * kVec;
            float g[kVec];
            load_gamma<T, kAligned>(p, c, vec_len(p.cols, c), g);
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[j][i] *= rstd * g[i];
        }
    }
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) amax = max(amax, abs_bits(v[j][i]));
    const Quantiser qz(row_max<kThreads>(amax, s_max));
    if (t == 0) p.scale[row] = qz.scale;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int64_t c = static_cast<int64_t>(j * kThreads + t) * kVec;
        const int n = vec_len(p.cols, c);
        if (DGEMM_CHECK(n == 0 || (row >= 0 && row < p.rows && c + n <= p.cols)))
            store_q<kAligned>(p.q + row * p.ldq + c, n, v[j], qz);
    }
}

// Rows longer than one block's registers: the same three steps, each reading
// the row again (the second and third mostly from L2).  H is stored in the
// last pass, so it may be the buffer of X or of the residual here too.
template <int kOp, typename T, bool kAligned>
__global__ void __launch_bounds__(1024) long_rows_kernel(const RowParams p)
{
    constexpr int kThreads = 1024;
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    const int64_t row = blockIdx.x;
    float ss = 0.f, rstd = 1.f;
    uint32_t amax = 0;
    if constexpr (kOp == kOpNorm) {
        for (int64_t c = static_cast<int64_t>(threadIdx.x) * kVec; c < p.cols; c += kThreads * kVec) {
            float v[kVec];
            load_row_vec<kOp, T, kAligned>(p, row, c, vec_len(p.cols, c), v);
#pragma unroll
            for (int i = 0; i < kVec; ++i) ss = fmaf(v[i], v[i], ss);
        }
        ss = row_sum<kThreads>(ss, s_sum);
        if (!(ss < __uint_as_float(0x7F800000u))) amax = 0x7FC00000u;
        rstd = rsqrtf(ss / static_cast<float>(p.cols) + p.eps);
    }
    auto value = [&](int64_t c, int n, float (&v)[kVec]) {
        load_row_vec<kOp, T, kAligned>(p, row, c, n, v);
    };
    auto norm = [&](int64_t c, int n, float (&v)[kVec]) {
        if constexpr (kOp == kOpNorm) {
            float g[kVec];
            load_gamma<T, kAligned>(p, c, n, g);
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[i] *= rstd * g[i];
        }
    };
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * kVec; c < p.cols; c += kThreads * kVec) {
        float v[kVec];
        const int n = vec_len(p.cols, c);
        value(c, n, v);
        norm(c, n, v);
#pragma unroll
        for (int i = 0; i < kVec; ++i) amax = max(amax, abs_bits(v[i]));
    }
    const Quantiser qz(row_max<kThreads>(amax, s_max));
    if (threadIdx.x == 0) p.scale[row] = qz.scale;
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * kVec; c < p.cols; c += kThreads * kVec) {
        float v[kVec];
        const int n = vec_len(p.cols, c);
        value(c, n, v);
        // the last read of this thread's elements: H may now overwrite an input
        if constexpr (kOp == kOpNorm)
            if (p.h) store_vec<T, kAligned>(static_cast<T *>(p.h) + row * p.ldh + c, n, v);
        norm(c, n, v);
        if (DGEMM_CHECK(c + n <= p.cols)) store_q<kAligned>(p.q + row * p.ldq + c, n, v, qz);
    }
}

template <typename T, bool kAligned>
__global__ void __launch_bounds__(256)
    dequantize_kernel(int64_t rows, int64_t cols, const int8_t *__restrict__ q, int64_t ldq,
                      const float *__restrict__ scale, T *__restrict__ x, int64_t ldx, int64_t vecs)
{
    const int64_t total = rows * vecs;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t row = i / vecs, c = (i - row * vecs) * kVec;
        const int n = vec_len(cols, c);
        const int8_t *src = q + row * ldq + c;
        const float s = scale[row];
        float v[kVec];
        if (kAligned && n == kVec) {
            const uint2 w = __ldcs(reinterpret_cast<const uint2 *>(src));
            const int8_t *e = reinterpret_cast<const int8_t *>(&w);
#pragma unroll
            for (int k = 0; k < kVec; ++k) v[k] = static_cast<float>(e[k]) * s;
        } else {
#pragma unroll
            for (int k = 0; k < kVec; ++k) v[k] = k < n ? static_cast<float>(src[k]) * s : 0.f;
        }
        if (DGEMM_CHECK(row < rows && c + n <= cols)) store_vec<T, kAligned>(x + row * ldx + c, n, v);
    }
}

// ---- host side

template <int kOp, typename T, bool kAligned, int kThreads, int kVecs>
void launch_rows(const RowParams &p, cudaStream_t stream)
{
    constexpr int kRowsPerBlock = kThreads < 128 ? 128 / kThreads : 1;
    const int64_t grid = (p.rows + kRowsPerBlock - 1) / kRowsPerBlock;
    rows_kernel<kOp, T, kAligned, kThreads, kVecs>
        <<<static_cast<unsigned>(grid), kThreads < 128 ? 128 : kThreads, 0, stream>>>(p);
}

template <int kOp, typename T, bool kAligned>
const char *launch_rows_by_length(const RowParams &p, cudaStream_t stream)
{
    const int64_t vecs = (p.cols + kVec - 1) / kVec;
    if (vecs <= 32)
        launch_rows<kOp, T, kAligned, 32, 1>(p, stream);
    else if (vecs <= 128)
        launch_rows<kOp, T, kAligned, 32, 4>(p, stream);
    else if (vecs <= 512)
        launch_rows<kOp, T, kAligned, 128, 4>(p, stream);
    else if (vecs <= 1024)
        launch_rows<kOp, T, kAligned, 256, 4>(p, stream);
    else if (vecs <= 2048)
        launch_rows<kOp, T, kAligned, 512, 4>(p, stream);
    else if (vecs <= 4096)
        launch_rows<kOp, T, kAligned, 1024, 4>(p, stream);
    else {
        long_rows_kernel<kOp, T, kAligned><<<static_cast<unsigned>(p.rows), 1024, 0, stream>>>(p);
        return "i8_long_rows";
    }
    return kOp == kOpNorm ? "i8_rmsnorm_rows" : kOp == kOpSwiglu ? "i8_swiglu_rows" : "i8_quantize_rows";
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
    const int64_t vecs = (cols + kVec - 1) / kVec;
    const int64_t cap = static_cast<int64_t>(dev.sm_count) * 16;
    const int64_t want = (rows * vecs + 255) / 256;
    const unsigned grid = static_cast<unsigned>(want < cap ? want : cap);
    T *out = static_cast<T *>(x);
    if (aligned(q, ldq, 1, 8) && aligned(x, ldx, sizeof(T), 16))
        dequantize_kernel<T, true><<<grid, 256, 0, stream>>>(rows, cols, q, ldq, scale, out, ldx, vecs);
    else
        dequantize_kernel<T, false><<<grid, 256, 0, stream>>>(rows, cols, q, ldq, scale, out, ldx, vecs);
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
    return launch_rows_op<kOpNorm>(type, p, stream);
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
