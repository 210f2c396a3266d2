// f8_decode.cu -- gemm_f8_tn for a few tokens.
//
// The bound is the weights' bytes, each read once: 16 channels a thread block, whose
// warps take every W-th block of 128 K values.  mma.sync (m16n8k16, FP32 accumulators)
// multiplies a block's 16 x 128 weights, widened to FP16 (exactly), with 8 tokens; the
// order of K within a block is free, as long as both operands use the same, so a lane's
// 16-byte word of a row is at once what it feeds to four MMAs, without shared memory or
// shuffles in between.  The warps' sums meet in shared memory, in the order of the warps.
//
// The tensor-core kernel takes ~5 us to start, to drain and to join split sums; this one
// starts with its loads.  One token, that one and this: 4096 x 4096 8.8 and 6.4 us, 8192 x
// 4096 10.9 and 8.9; even at 28672 x 4096 (22.4 and 22.5); 16384 x 16384 45.8 and 47.8.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chained.cuh"
#include "dgemm.h"
#include "f8.cuh"
#include "internal.h"

#define DGEMM_UNIT 14
#include "checked.cuh"
#include "rows.cuh"

namespace dgemm {
namespace {

constexpr int kChannels = 16;  // of a thread block
constexpr int kMaxWarps = 8;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight 8-bit values as four FP16 pairs.
template <bool kE5>
__device__ __forceinline__ void widen8(uint32_t lo, uint32_t hi, uint32_t (&h)[4])
{
    h[0] = f8x2_to_f16x2<kE5>(lo & 0xFFFFu);
    h[1] = f8x2_to_f16x2<kE5>(lo >> 16);
    h[2] = f8x2_to_f16x2<kE5>(hi & 0xFFFFu);
    h[3] = f8x2_to_f16x2<kE5>(hi >> 16);
}

// The first `left` bytes (1 to 15) of a row's last word, then zeros: nothing past the row's end is
// read, which may be where its memory ends.  (A call, out of the way of the loop that streams
// whole words: in line it cost 8192 x 4096 0.3 of 9.0 us.)
__device__ __noinline__ uint4 last_word(const uint8_t *p, int left)
{
    uint32_t w[4], last = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (i < (left & 3)) last |= static_cast<uint32_t>(p[(left & ~3) + i]) << (8 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = left >= 4 * (i + 1) ? load_u32(reinterpret_cast<const uint32_t *>(p) + i) : i == left >> 2 ? last : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The 16-byte word of a row at k, all of it there with kWhole; else zeros past `left` bytes.
template <bool kOnce, bool kWhole>
__device__ __forceinline__ uint4 load_word(const uint8_t *p, int left)
{
    if constexpr (kWhole) return load_v4<kOnce>(p);
    if (left <= 0) return make_uint4(0u, 0u, 0u, 0u);
    if (left < 16) return last_word(p, left);
    return load_v4<kOnce>(p);
}

// A lane's part of one block: words of weight rows g and g + 8 and of token g, at 16 q and
// 64 + 16 q of the block (g = lane / 4, q = lane mod 4), and the scales of its sums.
struct Block {
    uint4 w[2][2], x[2];
    float sw[2], sx[2];
};

// Where those lie.  Rows that are not there are read as the last one, for sums that are
// not stored.
struct Places {
    const uint8_t *w[2], *x;
    const float *sw[2], *sx[2];
    int64_t w_blk, x_blk;  // of the scales
    int left;              // K values from this lane's first word of block 0 on

    __device__ __forceinline__ Places(const F8Params &p, int64_t n, int g, int q)
    {
        w_blk = p.b.s_blk;
        x_blk = p.a.s_blk;
        left = static_cast<int>(p.K) - q * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = min(n + g + 8 * h, p.N - 1);
            w[h] = p.b.p + row * p.b.ld + q * 16;
            sw[h] = p.b.scale + p.b.band(row) * p.b.s_row;
        }
        x = p.a.p + min(static_cast<int64_t>(g), p.M - 1) * p.a.ld + q * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) sx[h] = p.a.scale + p.a.band(min(static_cast<int64_t>(2 * q + h), p.M - 1)) * p.a.s_row;
    }

    template <bool kWhole>
    __device__ __forceinline__ void words(Block &b, int k) const
    {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) b.w[h][i] = load_word<true, kWhole>(w[h] + k + i * 64, left - k - i * 64);
#pragma unroll
        for (int i = 0; i < 2; ++i) b.x[i] = load_word<false, kWhole>(x + k + i * 64, left - k - i * 64);
    }

    __device__ __forceinline__ void fetch(Block &b, int kb, bool whole) const
    {
        if (whole)
            words<true>(b, kb * kF8Block);
        else
            words<false>(b, kb * kF8Block);
#pragma unroll
        for (int h = 0; h < 2; ++h) b.sw[h] = load_f32(sw[h] + kb * w_blk);
#pragma unroll
        for (int h = 0; h < 2; ++h) b.sx[h] = load_f32(sx[h] + kb * x_blk);
    }
};

// (64 registers a thread: four thread blocks an SM, whose 32 warps have the bytes on their
// way that the bandwidth takes; with the next block's words in registers too, half as many
// warps do no better)
template <typename T, bool kA5, bool kB5>
__global__ void __launch_bounds__(32 * kMaxWarps, 4) f8_decode_kernel(const F8Params p, int num_kb)
{
    __shared__ float s_sum[kMaxWarps][kChannels][kF8DecodeTokens + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = static_cast<int>(blockDim.x) >> 5;
    const int g = lane >> 2, q = lane & 3;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * kChannels;
    chain_wait();
    chain_next();
    // the value of C that this thread stores, and its old one, on its way beside the sums
    static_assert(kChannels * kF8DecodeTokens <= 4 * 32, "a thread for each, of four warps");
    const int c = static_cast<int>(threadIdx.x) % kChannels, m = static_cast<int>(threadIdx.x) / kChannels;
    const bool mine = m < p.M && n + c < p.N;
    T *const dst = static_cast<T *>(p.C) + m * p.ldc + n + c;
    const float old = mine && p.beta != 0.f ? to_f32(*dst) : 0.f;
    const Places places(p, n, g, q);
    const int whole = static_cast<int>(p.K / kF8Block);  // blocks
    float sum[4] = {};
    for (int kb = warp; kb < num_kb; kb += warps) {
        Block now;
        places.fetch(now, kb, kb < whole);
        float part[4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // eight K values of a lane at a time: two MMAs
            uint32_t w[2][4], x[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 &v = now.w[h][i >> 1];
                widen8<kB5>(i & 1 ? v.z : v.x, i & 1 ? v.w : v.y, w[h]);
            }
            const uint4 &v = now.x[i >> 1];
            widen8<kA5>(i & 1 ? v.z : v.x, i & 1 ? v.w : v.y, x);
            mma16816(part, w[0][0], w[1][0], w[0][1], w[1][1], x[0], x[1]);
            mma16816(part, w[0][2], w[1][2], w[0][3], w[1][3], x[2], x[3]);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) sum[v] = fmaf(part[v] * now.sx[v & 1], now.sw[v >> 1], sum[v]);
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) s_sum[warp][g + 8 * (v >> 1)][2 * q + (v & 1)] = sum[v];
    __syncthreads();
    if (mine && DGEMM_CHECK(m < kF8DecodeTokens)) {
        float x = 0.f;
        for (int w = 0; w < warps; ++w) x += s_sum[w][c][m];
        if (p.bias) x += load_f32(p.bias + n + c);
        if (p.beta != 0.f) x = fmaf(p.beta, old, x);
        *dst = from_f32<T>(x);
    }
}

template <typename T, bool kA5, bool kB5>
bool launch_warps(const F8Params &p, int warps, cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>((p.N + kChannels - 1) / kChannels);
    const int num_kb = static_cast<int>((p.K + kF8Block - 1) / kF8Block);
    return launch_chained(f8_decode_kernel<T, kA5, kB5>, grid, 32u * static_cast<unsigned>(warps), 0, stream, 1, p, num_kb) == cudaSuccess;
}

template <typename T>
bool launch_typed(const F8Params &p, int warps, cudaStream_t stream)
{
    const bool a5 = p.a.type == DGEMM_F8_E5M2, b5 = p.b.type == DGEMM_F8_E5M2;
    if (a5) return b5 ? launch_warps<T, true, true>(p, warps, stream) : launch_warps<T, true, false>(p, warps, stream);
    return b5 ? launch_warps<T, false, true>(p, warps, stream) : launch_warps<T, false, false>(p, warps, stream);
}

}  // namespace

bool f8_decode_config_ok(const F8Config &cfg)
{
    return cfg.variant == kF8Decode && (cfg.split == 4 || cfg.split == 8);
}

bool launch_f8_decode(const F8Params &p, const F8Config &cfg, cudaStream_t stream)
{
    if (!f8_decode_config_ok(cfg) || p.offsets || p.M > kF8DecodeTokens || (p.N - 1) / kChannels >= INT32_MAX) return false;
    switch (p.c_type) {
    case DGEMM_TYPE_F32: return launch_typed<float>(p, cfg.split, stream);
    case DGEMM_TYPE_F16: return launch_typed<__half>(p, cfg.split, stream);
    default: return launch_typed<__nv_bfloat16>(p, cfg.split, stream);
    }
}

}  // namespace dgemm

DGEMM_DEFINE_CHECK_READER(check_status_f8_decode)
