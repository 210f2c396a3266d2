// i8_gemm.cu -- gemm_i8_tn: the product of two int8 matrices with an FP32
// scale for each row of either,
//
//   C[m, n] = scale_a[m] * scale_b[n] * sum_k A[m, k] B[n, k] + bias[n] + beta * C[m, n].
//
// The choice of the kernel (choose_config below), and the one for every case.
// Operands that TMA can describe (rows on 16-byte boundaries) go to the
// tensor-core kernel (i8_umma.cu) or, for few tokens, to the dot-product and
// mma.sync kernels (i8_decode.cu).
//
// i8_mma_kernel is the kernel for every case: operands of any alignment and
// pitch, any sizes.  64 x 64 output tiles, four warps of 32 x 32; K in chunks
// of 64 bytes staged in shared memory through registers (the next chunk's
// loads are in flight while a chunk is multiplied); mma.sync m16n8k32 on
// int8 with exact int32 sums.  Bound by the integer tensor rate: 149 Top/s
// at 16-byte alignment, 125 at 4, 109 at any (1023 x 8193 x 4095 at a pitch of
// 4095: 631 us, against 53 us at a pitch of 4096 by the tensor-core kernel).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <string>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chained.cuh"
#include "dgemm.h"
#include "i8_gemm.h"
#include "internal.h"

#define DGEMM_UNIT 7
#include "checked.cuh"

namespace dgemm {
namespace {

constexpr int kTile = 64;       // rows of A and of B in a block's tile
constexpr int kChunk = 64;      // K bytes of one stage
constexpr int kPitch = 80;      // bytes between staged rows: 8 rows x 4 words fall in 32 distinct banks
constexpr int kThreads = 128;
// K a whole number of chunks below which an int32 sum cannot overflow:
// 2^16 * 128 * 128 = 2^30
constexpr int64_t kFlush = 1 << 16;

// C[row, col] from the sum of products.
template <typename T>
__device__ __forceinline__ void store_one(const I8Params &p, int64_t row, int64_t col, float sum)
{
    if (row >= p.M || col >= p.N || !DGEMM_CHECK(row >= 0 && col >= 0)) return;
    T *dst = static_cast<T *>(p.C) + row * p.ldc + col;
    float v = sum * p.scale_a[row] * p.scale_b[col];
    if (p.bias) v += p.bias[col];
    if (p.beta != 0.f) v = fmaf(p.beta, i8_to_f32(*dst), v);
    *dst = i8_from_f32<T>(v);
}

// The 32 bytes of one thread's half row of a chunk, as kW-byte loads (1: as the
// aligned words around them, shifted into place: every word holds a byte of
// the matrix); bytes past the row's end (left) or of rows outside the matrix
// are zeros.
template <int kW>
__device__ __forceinline__ void load_half_row(const int8_t *p, bool row_ok, int64_t left, uint32_t (&w)[8])
{
    if (row_ok && left >= 32 && kW == 16) {
        const uint4 a = load_v4(p), b = load_v4(p + 16);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        return;
    }
    if (row_ok && left >= 32 && kW == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = load_u32(reinterpret_cast<const uint32_t *>(p) + i);
        return;
    }
    if (row_ok && left >= 32 && kW == 1) {
        const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 3u) * 8u;
        const uint32_t *a = reinterpret_cast<const uint32_t *>(p - shift / 8);
        uint32_t lo = load_u32(a);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // the last word only if the 32 bytes reach into it
            const uint32_t hi = i < 7 || shift ? load_u32(a + i + 1) : 0u;
            w[i] = __funnelshift_r(lo, hi, shift);
            lo = hi;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t v = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
            if (row_ok && i * 4 + b < left) v |= static_cast<uint32_t>(static_cast<uint8_t>(p[i * 4 + b])) << (8 * b);
        w[i] = v;
    }
}

__device__ __forceinline__ void mma_s8(int32_t (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

template <typename T, int kW>
__global__ void __launch_bounds__(kThreads) i8_mma_kernel(const I8Params p, int64_t tiles_n)
{
    __shared__ __align__(16) uint8_t sa[kTile * kPitch], sb[kTile * kPitch];
    chain_wait();
    chain_next();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int64_t m0 = blockIdx.x / tiles_n * kTile, n0 = blockIdx.x % tiles_n * kTile;
    const int wm = (warp & 1) * 32, wn = (warp >> 1) * 32;
    // this thread stages half a row (32 bytes) of either tile
    const int srow = tid >> 1, sbyte = (tid & 1) * 32;
    const bool a_ok = m0 + srow < p.M, b_ok = n0 + srow < p.N;
    const int8_t *ap = p.A + (a_ok ? (m0 + srow) * p.lda : 0) + sbyte;
    const int8_t *bp = p.B + (b_ok ? (n0 + srow) * p.ldb : 0) + sbyte;
    int32_t acc[2][4][4] = {};
    float sum[2][4][4] = {};
    uint32_t wa[8], wb[8];
    auto fetch = [&](int64_t k) {
        load_half_row<kW>(ap + k, a_ok, p.K - k - sbyte, wa);
        load_half_row<kW>(bp + k, b_ok, p.K - k - sbyte, wb);
    };
    if (p.K > 0) fetch(0);
    for (int64_t k = 0; k < p.K; k += kChunk) {
        __syncthreads();  // the previous chunk has been read
        if (DGEMM_CHECK(srow * kPitch + sbyte + 32 <= kTile * kPitch)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                *reinterpret_cast<uint4 *>(sa + srow * kPitch + sbyte + i * 16) =
                    make_uint4(wa[4 * i], wa[4 * i + 1], wa[4 * i + 2], wa[4 * i + 3]);
                *reinterpret_cast<uint4 *>(sb + srow * kPitch + sbyte + i * 16) =
                    make_uint4(wb[4 * i], wb[4 * i + 1], wb[4 * i + 2], wb[4 * i + 3]);
            }
        }
        __syncthreads();
        if (k + kChunk < p.K) fetch(k + kChunk);
#pragma unroll
        for (int kk = 0; kk < kChunk; kk += 32) {
            uint32_t a[2][4], b[4][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    a[i][h] = *reinterpret_cast<const uint32_t *>(sa + (wm + i * 16 + g + (h & 1) * 8) * kPitch + kk +
                                                                  t * 4 + (h >> 1) * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    b[j][h] =
                        *reinterpret_cast<const uint32_t *>(sb + (wn + j * 8 + g) * kPitch + kk + t * 4 + h * 16);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) mma_s8(acc[i][j], a[i], b[j]);
        }
        if ((k + kChunk) % kFlush == 0 || k + kChunk >= p.K) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sum[i][j][e] += static_cast<float>(acc[i][j][e]);
                        acc[i][j][e] = 0;
                    }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                store_one<T>(p, m0 + wm + i * 16 + g + (e >> 1) * 8, n0 + wn + j * 8 + t * 2 + (e & 1), sum[i][j][e]);
}

template <typename T>
const char *launch_mma(const I8Params &p, cudaStream_t stream)
{
    const int64_t tiles_m = (p.M + kTile - 1) / kTile, tiles_n = (p.N + kTile - 1) / kTile;
    if (tiles_m > INT32_MAX / tiles_n) return nullptr;
    const unsigned grid = static_cast<unsigned>(tiles_m * tiles_n);
    auto on = [&](int to) {
        return reinterpret_cast<uintptr_t>(p.A) % to == 0 && reinterpret_cast<uintptr_t>(p.B) % to == 0 &&
               p.lda % to == 0 && p.ldb % to == 0;
    };
    if (on(16)) {
        launch_chained(i8_mma_kernel<T, 16>, grid, kThreads, 0, stream, 1, p, tiles_n);
        return "i8_mma_64x64x64_ld16";
    }
    if (on(4)) {
        launch_chained(i8_mma_kernel<T, 4>, grid, kThreads, 0, stream, 1, p, tiles_n);
        return "i8_mma_64x64x64_ld4";
    }
    launch_chained(i8_mma_kernel<T, 1>, grid, kThreads, 0, stream, 1, p, tiles_n);
    return "i8_mma_64x64x64_ld1";
}

// One-shot override of the next call on this host thread (dgemm_tune_i8_next).
thread_local I8Config t_tune = {kI8Auto, 0, 1};

// Whether TMA can describe both operands.
bool tma_ok(const I8Params &p)
{
    constexpr int64_t kMax = INT32_MAX - 512;
    return p.K > 0 && aligned16(p.A) && aligned16(p.B) && p.lda % 16 == 0 && p.ldb % 16 == 0 && p.M <= kMax &&
           p.N <= kMax && p.K <= kMax;
}

// ---- automatic choice, for operands that TMA can describe
//
// Estimated times in us, fitted to GB300 sweeps of every kernel over 8 shapes
// of B x 19 numbers of tokens (1 .. 4096); the smallest estimate runs.  Of the best
// time of the present kernels in such a sweep it takes 1.01 in the geometric mean
// and at most 1.27 (192 tokens, 4096 x 14336: 40.6 and 31.9 us); next 1.14 (192
// tokens, 4096 x 4096) and 1.12 (64 tokens, 2048 x 2048).
//
// 1 and 2 tokens take the dot-product kernel, 3 to 8 the mma.sync kernel without
// an estimate: at most 1.13 (2 tokens, 2048 x 2048: 2.6 and 2.3 us) and 1.05 of
// the best.
struct Candidate {
    double us;
    I8Config cfg;
};

constexpr double kHbm = 6.4e6;  // bytes a us

// Time of one K block of 128, by tile width; between the points, linear.
double stage_us(bool pair, int bn)
{
    struct Point {
        int bn;
        double us;
    };
    static constexpr Point kPair[] = {{32, 0.33}, {64, 0.337}, {96, 0.352}, {128, 0.37}, {192, 0.445}, {256, 0.575}};
    static constexpr Point kSingle[] = {{16, 0.345}, {64, 0.385}, {128, 0.54}};
    const Point *p = pair ? kPair : kSingle;
    while (bn > p[1].bn) ++p;
    return p[0].us + (p[1].us - p[0].us) * (bn - p[0].bn) / (p[1].bn - p[0].bn);
}

// mma.sync: ~20 clocks of an SM for each product of 16 channels x 8 tokens x
// 32, or ~0.2 + 0.6 us a turn of 128 K values and group of 8 tokens where
// there are few warps; and the warps' sums, for every channel and group.
// Blocks of 16 warps where each has a turn, of 8 where there are many blocks
// anyway (8 tokens, 16 and 8 warps: 4096 x 14336 13.4 and 17.5 us, 8192 x 4096
// 8.3 and 9.5; 28672 x 4096 25.4 and 23.3, 16384 x 2048 9.2 and 7.8).
Candidate decode_candidate(const I8Params &p)
{
    const int warps = p.N <= 12288 && p.K >= 2048 ? 16 : 8;
    const double groups = p.M <= 8 ? 1.0 : p.M <= 16 ? 2.0 : 4.0;
    const double turns = static_cast<double>((p.K + 127) / 128 + warps - 1) / warps;
    const double nk = static_cast<double>(p.N) * static_cast<double>(p.K);
    return {2.2 + 0.8e-4 * groups * static_cast<double>(p.N) +
                std::max({1.6e-7 * groups * nk, turns * (0.2 + 0.6 * groups), nk / kHbm}),
            {kI8Decode, 0, warps}};
}

I8Config choose_config(const I8Params &p, int sm_count, bool (*fits)(const I8Params &, const I8Config &))
{
    if (p.K < (1 << 17)) {
        if (p.M <= 2) return {kI8Dot, 0, 1};
        if (p.M <= 8) return decode_candidate(p).cfg;
    }
    const int64_t kb = (p.K + 127) / 128;
    const double hbm = static_cast<double>(p.M + p.N) * static_cast<double>(p.K) / kHbm;
    Candidate best{1e30, {kI8PairTokens, 192, 1}};
    auto take = [&](const Candidate &c) {
        if (c.us < best.us && fits(p, c.cfg)) best = c;
    };
    if (p.M <= 32 && p.K < (1 << 17)) take(decode_candidate(p));
    // one CTA per 128 channels x bn tokens: at most two widths, without a split
    // in waves, or every split that keeps all CTAs resident.  Its tail, 128
    // columns of one accumulator stored token by token, grows with bn; a split
    // costs an exchange.
    const int64_t m16 = (p.M + 15) / 16 * 16;
    for (int bn : {static_cast<int>(std::min<int64_t>(m16, 128)), 64}) {
        if (bn > m16) continue;
        const int64_t tiles = (p.N + 127) / 128 * ((p.M + bn - 1) / bn);
        const int64_t waves = (tiles + sm_count - 1) / sm_count;
        for (int S = 1; S <= 8 && (S == 1 || tiles * S <= sm_count) && S <= kb; ++S)
            take({4.8 + 0.022 * bn + (S > 1 ? 1.6 : static_cast<double>(waves - 1)) +
                      std::max(static_cast<double>(waves * ((kb + S - 1) / S)) * stage_us(false, bn), hbm),
                  {kI8Split, bn, S}});
    }
    // CTA pairs of 256 x bn, in waves: rows are the channels (for few tokens)
    // or the tokens, whose tiles drain faster into C
    const int64_t pairs = sm_count / 2;
    auto pair = [&](int variant, int bn, int64_t rows, int64_t cols, double drain) {
        const int64_t tiles = (rows + 255) / 256 * ((cols + bn - 1) / bn), waves = (tiles + pairs - 1) / pairs;
        if (bn > 192 && waves > 1) return;
        take({5.2 + 0.014 * bn + drain * static_cast<double>(waves - 1) +
                  std::max(static_cast<double>(waves * kb) * stage_us(true, bn), hbm),
              {variant, bn, 1}});
    };
    for (int bn : {64, 128, 192, 256}) pair(kI8PairTokens, bn, p.M, p.N, 0.8);
    const int64_t m32 = (p.M + 31) / 32 * 32;
    for (int bn : {64, 96, 128, 192, 256})
        if (bn <= m32) pair(kI8PairChannels, bn, p.N, p.M, 3.0);
    return best.cfg;
}

// Kernel names by configuration, built once.  A tile with fewer K blocks than the
// split asked for has one CTA a block.
const char *config_name(const I8Config &c, int64_t K)
{
    static std::string names[17][9][9];  // by width, split (0: pairs) and CTAs that ran (0, 1: pairs' rows)
    static std::once_flag once;
    std::call_once(once, [] {
        for (int w = 1; w <= 16; ++w) {
            const std::string bn = std::to_string(16 * w);
            names[w][0][0] = "i8_umma_pair_256x" + bn + "_tokens";
            names[w][0][1] = "i8_umma_pair_256x" + bn + "_channels";
            for (int S = 1; S <= 8; ++S)
                for (int ran = 1; ran <= S; ++ran)
                    names[w][S][ran] = "i8_umma_128x" + bn + "_channels_split" + std::to_string(S) +
                                       (ran < S ? "_ran_" + std::to_string(ran) : "");
        }
    });
    if (c.variant == kI8Decode) return c.split == 8 ? "i8_decode_16_channels_8_warps" : "i8_decode_16_channels_16_warps";
    if (c.variant == kI8Dot) return "i8_dot_4_channels";
    if (c.variant == kI8Split) return names[c.bn / 16][c.split][std::min<int64_t>(c.split, (K + 127) / 128)].c_str();
    return names[c.bn / 16][0][c.variant == kI8PairChannels ? 1 : 0].c_str();
}

// (A launch that cannot be prepared falls back to the kernel for every case.)
bool launch_config(const I8Params &p, int c_type, const I8Config &cfg, int sm_count, cudaStream_t stream)
{
    return cfg.variant >= kI8Decode ? launch_i8_decode(p, c_type, cfg, sm_count, stream) : launch_i8_umma(p, c_type, cfg, stream);
}

}  // namespace

const char *launch_gemm_i8(const I8Params &q, int c_type, const I8Config &tune, cudaStream_t stream,
                           const DeviceInfo &dev)
{
    I8Params p = q;
    // the pitch of a single row is never used
    if (p.M == 1) p.lda = (p.K + 15) / 16 * 16;
    if (p.N == 1) p.ldb = (p.K + 15) / 16 * 16;
    if (tma_ok(p) && tune.variant != kI8Mma) {
        if (tune.variant != kI8Auto && launch_config(p, c_type, tune, dev.sm_count, stream)) return config_name(tune, p.K);
        const I8Config cfg = choose_config(p, dev.sm_count, i8_umma_fits);
        if (launch_config(p, c_type, cfg, dev.sm_count, stream)) return config_name(cfg, p.K);
    }
    switch (c_type) {
    case DGEMM_TYPE_F32: return launch_mma<float>(p, stream);
    case DGEMM_TYPE_F16: return launch_mma<__half>(p, stream);
    case DGEMM_TYPE_BF16: return launch_mma<__nv_bfloat16>(p, stream);
    default: return nullptr;
    }
}

int i8_tune_next(int variant, int bn, int split)
{
    const I8Config cfg{variant, bn, split};
    if (variant != kI8Auto && variant != kI8Mma && !i8_umma_config_ok(cfg) && !i8_decode_config_ok(cfg))
        return DGEMM_ERR_INVALID_ARG;
    t_tune = cfg;
    return DGEMM_OK;
}

I8Config i8_take_tune()
{
    const I8Config cfg = t_tune;
    t_tune = {kI8Auto, 0, 1};
    return cfg;
}

}  // namespace dgemm

DGEMM_DEFINE_CHECK_READER(check_status_i8_gemm)
