// i8_decode.cu -- gemm_i8_tn for few tokens (decoding).
//
// The work is one pass over the weights B: N x K bytes, bound by HBM (~7.2 TB/s
// for a plain read on GB300); A and C are small.  So the weights go from
// memory straight to registers, without shared memory, and the kernels are
// built to have many of their bytes in flight.  Sums are exact int32; they
// cannot overflow for K < 2^17.
//
// i8_dot_kernel, 1 and 2 tokens: four-way dot products on the integer pipes.  A
//   warp reads 512 contiguous bytes of each of four channels at a time, so
//   every line that leaves L2 is used whole, and the work is dealt evenly
//   over all warps.  One token, weights cycled past the L2: 8192 x 4096 in 7.3 us
//   (4.6 TB/s: start and end of the launch show), 28672 x 4096 in 19.8 (5.9 TB/s),
//   16384 x 16384 in 42.7 (6.3 TB/s).  The same 8192 x 4096 weights every time
//   stay in L2: 5.6 us, and 7.0 for a tail of blocks dealt by whole rows.
// i8_decode_kernel, up to 32 tokens: mma.sync m16n8k32 on int8, its 16 rows the
//   channels, its 8 columns the tokens.  A fragment wants four 4-byte pieces
//   of a row, 16 bytes apart; since any order of K will do as long as both
//   operands follow it, each thread instead loads 16 contiguous bytes and
//   uses them as the pieces of two products.  The integer tensor rate (a
//   product takes ~20 clocks of an SM) keeps pace with memory for one group
//   of 8 tokens (8192 x 4096: 9.6 us with cold weights, 6.7 from L2); more groups
//   pay where a tensor-core launch's fixed cost is larger (32 tokens, 2048 x
//   2048: 4.2 against 6.8 us).
//   The warps of a block read neighbouring pieces of its rows; dealt in even
//   ranges like the dot products', a warp walking along K by itself, they
//   took longer (8 tokens, 8192 x 4096 9.9, 1024 x 8192 9.1 against 4.0 us).
#include <algorithm>
#include <cstdint>
#include <type_traits>

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

// The first `left` bytes of v, then zeros.
__device__ __forceinline__ uint4 cut16(const uint4 &v, int left)
{
    auto cut = [left](uint32_t w, int first) {
        const int n = left - first;  // bytes of the word to keep
        return n >= 4 ? w : n > 0 ? w & ((1u << (8 * n)) - 1u) : 0u;
    };
    return make_uint4(cut(v.x, 0), cut(v.y, 4), cut(v.z, 8), cut(v.w, 12));
}

// 16 bytes at p + k of a row of K values: all of them there (kWhole), or zeros
// past the row's end.  The last word is read whole and cut: rows start on
// 16-byte boundaries, and an aligned word that holds one byte of the matrix is
// readable.
template <bool kOnce, bool kWhole>
__device__ __forceinline__ uint4 load16(const int8_t *p, int64_t k, int64_t K)
{
    if constexpr (kWhole) return load_v4<kOnce>(p + k);
    if (k >= K) return make_uint4(0, 0, 0, 0);
    return cut16(load_v4<kOnce>(p + k), static_cast<int>(K - k));
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
    float v = static_cast<float>(sum) * load_f32(p.scale_a + m) * load_f32(p.scale_b + n);
    if (p.bias) v += load_f32(p.bias + n);
    if (p.beta != 0.f) v = fmaf(p.beta, i8_to_f32(*dst), v);
    *dst = i8_from_f32<T>(v);
}

constexpr int kDotRows = 4;     // channels of a group
constexpr int kDotWarps = 8;    // of a block
constexpr int kDotTurn = 512;   // K bytes of a unit: 16 a lane
constexpr int kDotGroups = 64;  // groups a block may have

// The work is cut into units of a group of four channels x 512 K values, and
// spread evenly: every block takes an equal range of groups, every warp an
// equal range of its block's units, whatever N and K are.  A group's sum that
// two warps share meets in shared memory; it is an integer, so the order does
// not matter.  kUnroll units are loaded before the first product.  What lies past
// a row's end within the 16 bytes that hold its last value is read (rows start on
// 16-byte boundaries) and cut off.
template <typename T, int kTokens, int kUnroll, int kBlocks>
__global__ void __launch_bounds__(kDotWarps * 32, kBlocks)
    i8_dot_kernel(const I8Params p, int groups_each, int groups_more, int turns)
{
    __shared__ int32_t sums[kDotGroups][kDotRows * kTokens];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // groups_each of them a block, and one more in the first groups_more
    const int block = static_cast<int>(blockIdx.x);
    const int g0 = block * groups_each + min(block, groups_more), ng = groups_each + (block < groups_more ? 1 : 0);
    for (int i = threadIdx.x; i < ng * kDotRows * kTokens; i += kDotWarps * 32)
        if (DGEMM_CHECK(ng <= kDotGroups)) (&sums[0][0])[i] = 0;
    const int units = ng * turns;
    int u = units * warp / kDotWarps;
    const int end = units * (warp + 1) / kDotWarps;
    int g = u / turns, turn = u - g * turns;  // of the next unit to multiply
    int gl = g, tl = turn;                    // of the next to load
    // past the row's end its last 16 bytes again, with the token's cut to zeros
    const int K = static_cast<int>(p.K), k_last = (K - 1) / 16 * 16;
    uint4 w[kUnroll][kDotRows], x[kUnroll][kTokens];
    auto load = [&](int i) {
        const int64_t n = static_cast<int64_t>(g0 + gl) * kDotRows;
        const int k = min(tl * kDotTurn + lane * 16, k_last);
#pragma unroll
        for (int r = 0; r < kDotRows; ++r)  // past the last channel: that one again, and the sum is dropped
            w[i][r] = load_v4<true>(p.B + min(n + r, p.N - 1) * p.ldb + k);
#pragma unroll
        for (int m = 0; m < kTokens; ++m) x[i][m] = load_v4(p.A + m * p.lda + k);
        if (++tl == turns) {
            tl = 0;
            ++gl;
        }
    };
    int32_t acc[kDotRows][kTokens] = {};
    auto multiply = [&](int i) {
        if ((turn + 1) * kDotTurn > K) {
#pragma unroll
            for (int m = 0; m < kTokens; ++m) x[i][m] = cut16(x[i][m], K - turn * kDotTurn - lane * 16);
        }
#pragma unroll
        for (int r = 0; r < kDotRows; ++r)
#pragma unroll
            for (int m = 0; m < kTokens; ++m) {
                int32_t s = acc[r][m];
                s = __dp4a(static_cast<int>(w[i][r].x), static_cast<int>(x[i][m].x), s);
                s = __dp4a(static_cast<int>(w[i][r].y), static_cast<int>(x[i][m].y), s);
                s = __dp4a(static_cast<int>(w[i][r].z), static_cast<int>(x[i][m].z), s);
                acc[r][m] = __dp4a(static_cast<int>(w[i][r].w), static_cast<int>(x[i][m].w), s);
            }
    };
    // the warp's sum for group g of the block, and a new one
    auto flush = [&]() {
#pragma unroll
        for (int r = 0; r < kDotRows; ++r)
#pragma unroll
            for (int m = 0; m < kTokens; ++m) {
                const int32_t s = __reduce_add_sync(0xFFFFFFFFu, acc[r][m]);
                if (lane == 0 && DGEMM_CHECK(g < ng)) atomicAdd(&sums[g][r * kTokens + m], s);
                acc[r][m] = 0;
            }
    };
    chain_wait();
    chain_next();
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
        if (u + i < end) load(i);
    __syncthreads();  // the sums' zeros
    while (u < end) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (u + i < end) {
                multiply(i);
                if (turn + 1 == turns || u + i + 1 == end) flush();
                if (++turn == turns) {
                    turn = 0;
                    ++g;
                }
            }
        }
        u += kUnroll;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (u + i < end) load(i);
    }
    __syncthreads();
    // consecutive threads take consecutive channels of a token
    const int channels = ng * kDotRows;
    for (int i = threadIdx.x; i < channels * kTokens; i += kDotWarps * 32) {
        const int m = i / channels, c = i - m * channels;
        const int64_t n = static_cast<int64_t>(g0) * kDotRows + c;
        if (m < p.M && n < p.N && DGEMM_CHECK(c / kDotRows < kDotGroups))
            store_sum<T>(p, m, n, sums[c / kDotRows][c % kDotRows * kTokens + m]);
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
    // this thread's two channels and its tokens; past the last, that one again,
    // and the sum is dropped
    const int8_t *b[2], *a[kTiles];
#pragma unroll
    for (int r = 0; r < 2; ++r) b[r] = p.B + (n0 + g + r * 8 < p.N ? n0 + g + r * 8 : p.N - 1) * p.ldb + t * 16;
#pragma unroll
    for (int j = 0; j < kTiles; ++j) a[j] = p.A + (j * 8 + g < p.M ? j * 8 + g : p.M - 1) * p.lda + t * 16;
    int32_t acc[kTiles][4] = {};
    auto turn = [&](int64_t k, auto whole) {
        constexpr bool kWhole = decltype(whole)::value;
        const int64_t K = p.K - t * 16;
        uint4 w[2][2], x[kTiles][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) w[h][r] = load16<true, kWhole>(b[r], k + h * 64, K);
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) x[j][h] = load16<false, kWhole>(a[j], k + h * 64, K);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                mma_s8(acc[j], w[h][0].x, w[h][1].x, w[h][0].y, w[h][1].y, x[j][h].x, x[j][h].y);
                mma_s8(acc[j], w[h][0].z, w[h][1].z, w[h][0].w, w[h][1].w, x[j][h].z, x[j][h].w);
            }
    };
    int64_t k = warp * kTurn;
    for (; k + kTurn <= p.K; k += kWarps * kTurn) turn(k, std::true_type{});
    if (k < p.K) turn(k, std::false_type{});
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

template <typename T, int kTokens, int kUnroll, int kBlocks>
void launch_dot(const I8Params &p, int sm_count, cudaStream_t stream)
{
    // one wave of blocks, unless a block would have more groups than it has sums for
    const int64_t groups = (p.N + kDotRows - 1) / kDotRows, resident = static_cast<int64_t>(sm_count) * kBlocks;
    const int64_t blocks = std::max(std::min(resident, groups), (groups + kDotGroups - 1) / kDotGroups);
    launch_chained(i8_dot_kernel<T, kTokens, kUnroll, kBlocks>, static_cast<unsigned>(blocks), kDotWarps * 32, 0,
                   stream, 1, p, static_cast<int>(groups / blocks), static_cast<int>(groups % blocks),
                   static_cast<int>((p.K + kDotTurn - 1) / kDotTurn));
}

// Two units of a warp in flight where blocks have few groups, else one and a
// block more an SM (1 token, the same weights every time: 4096 x 4096 3.2 and 3.6
// us, 8192 x 4096 5.9 and 5.6, 28672 x 4096 20.3 and 19.8).
template <typename T>
void launch_dot_tokens(const I8Params &p, int sm_count, cudaStream_t stream)
{
    if (p.M == 2)
        launch_dot<T, 2, 1, 4>(p, sm_count, stream);
    else if (p.N <= 6144)
        launch_dot<T, 1, 2, 4>(p, sm_count, stream);
    else
        launch_dot<T, 1, 1, 5>(p, sm_count, stream);
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
           (cfg.variant == kI8Dot && cfg.split == 1);
}

bool launch_i8_decode(const I8Params &p, int c_type, const I8Config &cfg, int sm_count, cudaStream_t stream)
{
    const bool dot = cfg.variant == kI8Dot;
    if (!i8_decode_config_ok(cfg) || p.M > (dot ? 2 : 32) || p.K >= (1 << 17) || p.N > INT32_MAX) return false;
    switch (c_type) {
    case DGEMM_TYPE_F32:
        dot ? launch_dot_tokens<float>(p, sm_count, stream) : launch_decode<float>(p, cfg.split, stream);
        return true;
    case DGEMM_TYPE_F16:
        dot ? launch_dot_tokens<__half>(p, sm_count, stream) : launch_decode<__half>(p, cfg.split, stream);
        return true;
    case DGEMM_TYPE_BF16:
        dot ? launch_dot_tokens<__nv_bfloat16>(p, sm_count, stream) : launch_decode<__nv_bfloat16>(p, cfg.split, stream);
        return true;
    default: return false;
    }
}

}  // namespace dgemm

DGEMM_DEFINE_CHECK_READER(check_status_i8_decode)
