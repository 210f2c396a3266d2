// i8_decode.cu -- gemm_i8_tn for few tokens (decoding).
//
// The work is one pass over the weights B: N x K bytes, bound by HBM (~7.2 TB/s
// for a plain read on GB300); A and C are small.  So the weights go from
// memory straight to registers, without shared memory, and the kernels are
// built to have many of their bytes in flight.  Sums are exact int32; they
// cannot overflow for K < 2^17.
//
// i8_dot_kernel, 1 to 4 tokens: four-way dot products on the integer pipes.
//   A warp reads 512 contiguous bytes of each of four channels at a time, so
//   every line that leaves L2 is used whole: 8192 x 4096 weights in 7.0 us
//   against 8.9 us for i8_decode_kernel, 16384 x 16384 in 38.7 against 48 us.
//   One dot product of four bytes per token and weight word: ~1/4 of the
//   memory time for each token.
// i8_decode_kernel, up to 32 tokens: mma.sync m16n8k32 on int8, its 16 rows the
//   channels, its 8 columns the tokens.  A fragment wants four 4-byte pieces
//   of a row, 16 bytes apart; since any order of K will do as long as both
//   operands follow it, each thread instead loads 16 contiguous bytes and
//   uses them as the pieces of two products.  The integer tensor rate (a
//   product takes ~20 clocks of an SM) keeps pace with memory for one group
//   of 8 tokens; more groups pay where a tensor-core launch's fixed cost is
//   larger.
#include <cstdint>

#include <cuda_runtime.h>

#include "chained.cuh"
#include "dgemm.h"
#include "i8_gemm.h"
#include "internal.h"

#define DGEMM_UNIT 9
#include "checked.cuh"

namespace dgemm {
namespace {

constexpr int kChannels = 16;  // of a block
constexpr int kTurn = 128;     // K bytes of a warp's turn

// 16 bytes at p + k of a row of K values (zeros past its end, and for rows
// that are not there).
template <bool kStream>
__device__ __forceinline__ uint4 load16(const int8_t *p, int64_t k, int64_t K, bool row_ok)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    if (!row_ok || k >= K) return v;
    if (k + 16 <= K) {
        if constexpr (kStream)
            asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "l"(p + k));
        else
            v = __ldg(reinterpret_cast<const uint4 *>(p + k));
        return v;
    }
    uint32_t w[4] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (k + i < K) w[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(p[k + i])) << (8 * (i & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void mma_s8(int32_t (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ void store_sum(const I8Params &p, int64_t m, int64_t n, int32_t sum)
{
    T *dst = static_cast<T *>(p.C) + m * p.ldc + n;
    float v = static_cast<float>(sum) * __ldg(p.scale_a + m) * __ldg(p.scale_b + n);
    if (p.bias) v += __ldg(p.bias + n);
    if (p.beta != 0.f) v = fmaf(p.beta, i8_to_f32(*dst), v);
    *dst = i8_from_f32<T>(v);
}

constexpr int kDotRows = 4;    // channels of a warp
constexpr int kDotWarps = 8;   // of a block
constexpr int kDotTurn = 512;  // K bytes of a warp's turn

// `split` warps (a power of two up to 8) share K in turns; a thread's loads of
// kUnroll turns are issued before the first product.
template <typename T, int kTokens, int kUnroll>
__global__ void __launch_bounds__(kDotWarps * 32) i8_dot_kernel(const I8Params p, int split)
{
    __shared__ int32_t sums[kDotWarps][kDotRows * kTokens];
    chain_wait();
    chain_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = kDotWarps / split;  // of kDotRows channels, in this block
    const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * groups + warp / split) * kDotRows;
    const int8_t *b = p.B + (n0 < p.N ? n0 : 0) * p.ldb;
    int32_t acc[kDotRows][kTokens] = {};
    const int64_t stride = static_cast<int64_t>(split) * kDotTurn;
    for (int64_t k0 = (warp % split) * kDotTurn + lane * 16; k0 < p.K; k0 += stride * kUnroll) {
        uint4 w[kUnroll][kDotRows], x[kUnroll][kTokens];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t k = k0 + u * stride;  // (past the end: zeros)
#pragma unroll
            for (int r = 0; r < kDotRows; ++r) w[u][r] = load16<true>(b + r * p.ldb, k, p.K, n0 + r < p.N);
#pragma unroll
            for (int m = 0; m < kTokens; ++m) x[u][m] = load16<false>(p.A + m * p.lda, k, p.K, m < p.M);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int r = 0; r < kDotRows; ++r)
#pragma unroll
                for (int m = 0; m < kTokens; ++m) {
                    int32_t s = acc[r][m];
                    s = __dp4a(static_cast<int>(w[u][r].x), static_cast<int>(x[u][m].x), s);
                    s = __dp4a(static_cast<int>(w[u][r].y), static_cast<int>(x[u][m].y), s);
                    s = __dp4a(static_cast<int>(w[u][r].z), static_cast<int>(x[u][m].z), s);
                    acc[r][m] = __dp4a(static_cast<int>(w[u][r].w), static_cast<int>(x[u][m].w), s);
                }
    }
#pragma unroll
    for (int r = 0; r < kDotRows; ++r)
#pragma unroll
        for (int m = 0; m < kTokens; ++m) {
            const int32_t s = __reduce_add_sync(0xFFFFFFFFu, acc[r][m]);
            if (lane == 0) sums[warp][r * kTokens + m] = s;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < groups * kDotRows * kTokens; i += kDotWarps * 32) {
        const int g = i / (kDotRows * kTokens), e = i % (kDotRows * kTokens), m = e % kTokens;
        const int64_t n = (static_cast<int64_t>(blockIdx.x) * groups + g) * kDotRows + e / kTokens;
        if (m >= p.M || n >= p.N || !DGEMM_CHECK((g + 1) * split <= kDotWarps)) continue;
        int32_t sum = 0;
        for (int q = 0; q < split; ++q) sum += sums[g * split + q][e];
        store_sum<T>(p, m, n, sum);
    }
}

// kTiles groups of 8 tokens, kWarps warps to a block.
template <typename T, int kTiles, int kWarps>
__global__ void __launch_bounds__(kWarps * 32) i8_decode_kernel(const I8Params p)
{
    __shared__ int32_t sums[kWarps][kTiles * 8][kChannels];
    chain_wait();
    chain_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kChannels;
    // this thread's two channels and its tokens
    const bool b_ok[2] = {n0 + g < p.N, n0 + g + 8 < p.N};
    const int8_t *b[2] = {p.B + (b_ok[0] ? n0 + g : 0) * p.ldb, p.B + (b_ok[1] ? n0 + g + 8 : 0) * p.ldb};
    int32_t acc[kTiles][4] = {};
    const int64_t turns = (p.K + kTurn - 1) / kTurn;
    for (int64_t s = warp; s < turns; s += kWarps) {
        const int64_t k = s * kTurn + t * 16;
        uint4 w[2][2], x[kTiles][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) w[h][r] = load16<true>(b[r], k + h * 64, p.K, b_ok[r]);
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
            const int m = j * 8 + g;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                x[j][h] = load16<false>(p.A + (m < p.M ? m : 0) * p.lda, k + h * 64, p.K, m < p.M);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                mma_s8(acc[j], w[h][0].x, w[h][1].x, w[h][0].y, w[h][1].y, x[j][h].x, x[j][h].y);
                mma_s8(acc[j], w[h][0].z, w[h][1].z, w[h][0].w, w[h][1].w, x[j][h].z, x[j][h].w);
            }
    }
#pragma unroll
    for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[warp][j * 8 + t * 2 + (e & 1)][g + (e >> 1) * 8] = acc[j][e];
    __syncthreads();
    // consecutive threads take consecutive channels of a token
    for (int i = threadIdx.x; i < kTiles * 8 * kChannels; i += kWarps * 32) {
        const int m = i / kChannels, c = i % kChannels;
        if (m >= p.M || n0 + c >= p.N || !DGEMM_CHECK(m < kTiles * 8)) continue;
        int32_t sum = 0;
#pragma unroll
        for (int s = 0; s < kWarps; ++s) sum += sums[s][m][c];
        store_sum<T>(p, m, n0 + c, sum);
    }
}

template <typename T, int kTokens, int kUnroll>
void launch_dot(const I8Params &p, int split, cudaStream_t stream)
{
    const int64_t rows = kDotRows * (kDotWarps / split);
    launch_chained(i8_dot_kernel<T, kTokens, kUnroll>, static_cast<unsigned>((p.N + rows - 1) / rows), kDotWarps * 32, 0,
                   stream, 1, p, split);
}

template <typename T>
void launch_dot_tokens(const I8Params &p, int split, cudaStream_t stream)
{
    // two turns in flight where there are two and registers allow
    const bool two = p.K > static_cast<int64_t>(split) * kDotTurn;
    if (p.M == 1)
        two ? launch_dot<T, 1, 2>(p, split, stream) : launch_dot<T, 1, 1>(p, split, stream);
    else if (p.M == 2)
        two ? launch_dot<T, 2, 2>(p, split, stream) : launch_dot<T, 2, 1>(p, split, stream);
    else
        launch_dot<T, 4, 1>(p, split, stream);
}

template <typename T, int kTiles>
void launch_decode_tiles(const I8Params &p, int warps, cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>((p.N + kChannels - 1) / kChannels);
    if (warps == 8)
        launch_chained(i8_decode_kernel<T, kTiles, 8>, grid, 256, 0, stream, 1, p);
    else
        launch_chained(i8_decode_kernel<T, kTiles, 16>, grid, 512, 0, stream, 1, p);
}

template <typename T>
void launch_decode(const I8Params &p, int warps, cudaStream_t stream)
{
    if (p.M <= 8)
        launch_decode_tiles<T, 1>(p, warps, stream);
    else if (p.M <= 16)
        launch_decode_tiles<T, 2>(p, warps, stream);
    else
        launch_decode_tiles<T, 4>(p, warps, stream);
}

}  // namespace

bool i8_decode_config_ok(const I8Config &cfg)
{
    return (cfg.variant == kI8Decode && (cfg.split == 8 || cfg.split == 16)) ||
           (cfg.variant == kI8Dot && (cfg.split == 1 || cfg.split == 2 || cfg.split == 4 || cfg.split == 8));
}

bool launch_i8_decode(const I8Params &p, int c_type, const I8Config &cfg, cudaStream_t stream)
{
    const bool dot = cfg.variant == kI8Dot;
    if (!i8_decode_config_ok(cfg) || p.M > (dot ? 4 : 32) || p.K >= (1 << 17) || p.N > INT32_MAX) return false;
    switch (c_type) {
    case DGEMM_TYPE_F32:
        dot ? launch_dot_tokens<float>(p, cfg.split, stream) : launch_decode<float>(p, cfg.split, stream);
        return true;
    case DGEMM_TYPE_F16:
        dot ? launch_dot_tokens<__half>(p, cfg.split, stream) : launch_decode<__half>(p, cfg.split, stream);
        return true;
    case DGEMM_TYPE_BF16:
        dot ? launch_dot_tokens<__nv_bfloat16>(p, cfg.split, stream) : launch_decode<__nv_bfloat16>(p, cfg.split, stream);
        return true;
    default: return false;
    }
}

}  // namespace dgemm

DGEMM_DEFINE_CHECK_READER(check_status_i8_decode)
