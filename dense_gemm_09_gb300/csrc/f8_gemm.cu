// f8_gemm.cu -- gemm_f8_tn and gemm_f8_tn_experts: the choice of a kernel, and the
// kernel for operands of any alignment.
//
//   C[m, n] = sum_b sa(m, b) sb(n, b) sum_(k in b) A[m, k] B[n, k] + bias[n] + beta C[m, n]
//
// f8_any_kernel: tiles of 64 tokens x 64 channels.  A block of 128 K values of both
// operands is widened to FP16 (exact for either 8-bit type) into shared memory,
// multiplied by mma.sync with FP32 accumulators, and the block's sums are scaled and
// added to FP32 sums in registers.  It takes what TMA cannot: rows off 16-byte
// boundaries, whose bytes it loads one by one, and is bound by those loads.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "chained.cuh"
#include "dgemm.h"
#include "f8.cuh"
#include "internal.h"

#define DGEMM_UNIT 11
#include "checked.cuh"
#include "f8_tiles.cuh"
#include "rows.cuh"

namespace dgemm {
namespace {

constexpr int kTile = 64;
constexpr int kPitch = kF8Block + 8;  // halves: rows 4 banks apart
constexpr int kThreads = 128;

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// 64 rows x 128 K values of an operand from `row` (rows up to row_end) and k0, as
// FP16; zeros outside.
__device__ __forceinline__ void load_tile(__half *s, const F8Operand &o, const uint8_t *base, int64_t row, int64_t row_end,
                                          int64_t k0, int64_t K)
{
    for (int i = threadIdx.x; i < kTile * kF8Block / 4; i += kThreads) {
        const int r = i / (kF8Block / 4), c = i % (kF8Block / 4) * 4;
        uint32_t w = 0;
        if (row + r < row_end) {
            const uint8_t *src = base + (row + r) * o.ld + k0 + c;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k0 + c + k < K) w |= static_cast<uint32_t>(src[k]) << (8 * k);
        }
        uint32_t *dst = reinterpret_cast<uint32_t *>(s + r * kPitch + c);
        if (!DGEMM_CHECK(r < kTile && c + 4 <= kF8Block)) continue;
        if (o.type == DGEMM_F8_E5M2) {
            dst[0] = f8x2_to_f16x2<true>(w & 0xFFFFu);
            dst[1] = f8x2_to_f16x2<true>(w >> 16);
        } else {
            dst[0] = f8x2_to_f16x2<false>(w & 0xFFFFu);
            dst[1] = f8x2_to_f16x2<false>(w >> 16);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) f8_any_kernel(const F8Params p, uint32_t tiles_n)
{
    __shared__ __align__(16) __half s_a[kTile * kPitch], s_b[kTile * kPitch];
    extern __shared__ uint32_t s_table[];
    const F8Table table{s_table, reinterpret_cast<int32_t *>(s_table + p.experts + 1)};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    chain_wait();
    chain_next();
    if (p.offsets && warp == 0) fill_table(p, kTile, table, lane);
    __syncthreads();
    const uint32_t tiles_t = static_cast<uint32_t>((p.M + kTile - 1) / kTile);  // (of one matrix)
    const uint32_t tiles = (p.offsets ? table.first[p.experts] : tiles_t) * tiles_n;
    const int wr = (warp >> 1) * 32, wc = (warp & 1) * 32;
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const F8Tile tile = find_tile(p, table, tiles_t, tiles_n, kTile, kTile, t);
        const uint8_t *B = p.b.p + tile.expert * p.b_stride;
        const float *sb = p.b.scale + tile.expert * p.sb_stride;
        float acc[2][4][4] = {};
        for (int64_t k0 = 0; k0 < p.K; k0 += kF8Block) {
            __syncthreads();  // the last block has been read
            load_tile(s_a, p.a, p.a.p, tile.t0, tile.t_end, k0, p.K);
            load_tile(s_b, p.b, B, tile.n0, p.N, k0, p.K);
            __syncthreads();
            float part[2][4][4] = {};
#pragma unroll
            for (int k = 0; k < kF8Block; k += 16) {
                uint32_t a[2][4], b[4][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const __half *src = s_a + (wr + i * 16 + g) * kPitch + k + 2 * q;
                    a[i][0] = *reinterpret_cast<const uint32_t *>(src);
                    a[i][1] = *reinterpret_cast<const uint32_t *>(src + 8 * kPitch);
                    a[i][2] = *reinterpret_cast<const uint32_t *>(src + 8);
                    a[i][3] = *reinterpret_cast<const uint32_t *>(src + 8 * kPitch + 8);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __half *src = s_b + (wc + j * 8 + g) * kPitch + k + 2 * q;
                    b[j][0] = *reinterpret_cast<const uint32_t *>(src);
                    b[j][1] = *reinterpret_cast<const uint32_t *>(src + 8);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma16816(part[i][j], a[i], b[j]);
            }
            const int64_t kb = k0 / kF8Block;
            float ra[2][2], cb[4][2];  // scales of this thread's rows and columns (clamped to ones that exist)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t m = min(static_cast<int64_t>(tile.t0) + wr + i * 16 + h * 8 + g, static_cast<int64_t>(tile.t_end - 1));
                    ra[i][h] = p.a.scale[p.a.band(m) * p.a.s_row + kb * p.a.s_blk];
                }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t n = min(tile.n0 + wc + j * 8 + 2 * q + h, p.N - 1);
                    cb[j][h] = sb[p.b.band(n) * p.b.s_row + kb * p.b.s_blk];
                }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        acc[i][j][v] = fmaf(part[i][j][v] * cb[j][v & 1], ra[i][v >> 1], acc[i][j][v]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    // (a tile of an expert that begins anywhere may end past 2^31)
                    const int64_t m = static_cast<int64_t>(tile.t0) + wr + i * 16 + (v >> 1) * 8 + g, n = tile.n0 + wc + j * 8 + 2 * q + (v & 1);
                    if (m >= tile.t_end || n >= p.N || !DGEMM_CHECK(m < p.M)) continue;
                    T *dst = static_cast<T *>(p.C) + m * p.ldc + n;
                    float x = acc[i][j][v];
                    if (p.bias) x += p.bias[n];
                    if (p.beta != 0.f) x = fmaf(p.beta, to_f32(*dst), x);
                    *dst = from_f32<T>(x);
                }
    }
}

thread_local F8Config t_tune = {kF8Auto, 0, 1};

const char *launch_any(const F8Params &p, cudaStream_t stream, const DeviceInfo &dev)
{
    const int64_t tiles_n = (p.N - 1) / kTile + 1, bound = token_tiles_bound(p, kTile);
    const int64_t tiles = tiles_n * bound;
    if (tiles > INT32_MAX) return nullptr;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tiles, static_cast<int64_t>(dev.sm_count) * 8));
    auto kernel = p.c_type == DGEMM_TYPE_F32 ? f8_any_kernel<float>
                  : p.c_type == DGEMM_TYPE_F16 ? f8_any_kernel<__half>
                                               : f8_any_kernel<__nv_bfloat16>;
    const size_t smem = static_cast<size_t>(p.experts + 1) * 8;
    if (launch_chained(kernel, grid, kThreads, smem, stream, 1, p, static_cast<uint32_t>(tiles_n)) != cudaSuccess) return nullptr;
    return "f8_any_64x64";
}

// The kernels' times, fitted to GB300 sweeps: a start, then waves of tiles, each of which takes
// a CTA (pair) `block` for every 128 of K and `tile` besides; never less than the operands'
// bytes.  In microseconds, K = 4096, measured and as estimated here: pair 256 x 256 for 8192 x
// 8192 233 (236), and with a scale a row 355 (357); pair 256 x 128 for 512 x 4096 14.6 (14.4),
// for 2048 x 4096 of 512 values with the old C, to FP32, 19.8 (19.4), where 256 x 256 takes
// 29.8 (28.5); 128 channels x 64 tokens for 128 x 8192 13.5 (13.1), for 256 x 8192 22.4 (21.7);
// x 32 for 20 x 8192 10.8 (11.1), split in two 10.9 (9.9); x 16 for 16 x 8192 11.4 (11.1), split
// in two 10.3 (9.9), for 9 x 512, K = 1664, split in two, as chosen, 5.4 (7.1), in four 5.3
// (7.4); dot products for one token, 8192 channels 8.9 (8.9), 4096 channels 6.4 (7.9).
struct Kernel {
    F8Config cfg;
    int tokens, channels, ctas;  // of a tile
    double block, block_rows;    // with weights in bands of 128 rows, and with a scale a row
    double tile[2][2];           // the stores: [with the old C read][to FP32]
    double join;                 // of split sums, for every doubling of the CTAs
};
// (Narrow tiles first: of kernels that the bytes bound they do best, one token, 8 of 64 experts
// of 4096 x 2048, x 16 11.5 us, x 32 13.0, x 64 15.4.)
constexpr Kernel kKernels[] = {{{kF8Channels, 16, 1}, 16, 128, 1, 0.19, 0.19, {{0.5, 0.5}, {0.9, 0.9}}, 0.8},
                               {{kF8Channels, 32, 1}, 32, 128, 1, 0.19, 0.19, {{0.5, 0.5}, {1.0, 1.0}}, 1.2},
                               {{kF8Channels, 64, 1}, 64, 128, 1, 0.25, 0.25, {{0.6, 0.6}, {2.2, 2.2}}, 0.0},
                               {{kF8Pair, 128, 1}, 256, 128, 2, 0.28, 0.38, {{0.9, 1.1}, {1.8, 2.6}}, 0.0},
                               {{kF8Pair, 256, 1}, 256, 256, 2, 0.47, 0.74, {{1.5, 2.5}, {5.6, 10.1}}, 0.0}};
constexpr double kStart = 4.5, kBytesUs = 6.2e6;

F8Config choose(const F8Params &p, const DeviceInfo &dev)
{
    const double nb = static_cast<double>((p.K + kF8Block - 1) / kF8Block);
    // experts that have rows, at most; rows of each of them, on average
    const double experts = static_cast<double>(p.offsets ? std::min<int64_t>(p.M, p.experts) : 1), rows = static_cast<double>(p.M) / experts;
    const double bytes = (experts * static_cast<double>(p.N) + static_cast<double>(p.M)) * static_cast<double>(p.K);
    F8Config best{};
    double least = 1e300;
    auto offer = [&](const F8Config &cfg, double us) {
        if (us < least) {
            least = us;
            best = cfg;
        }
    };
    for (const Kernel &k : kKernels) {
        // (an expert's last tile is half full on average, if it has more than one)
        const double tiles_t = p.offsets ? experts * (rows <= k.tokens ? 1.0 : rows / k.tokens + 0.5)
                                         : static_cast<double>((p.M + k.tokens - 1) / k.tokens);
        const double tiles = tiles_t * static_cast<double>((p.N + k.channels - 1) / k.channels);
        const double slots = dev.sm_count / k.ctas, block = p.b.block == kF8Block ? k.block : k.block_rows;
        const double tile = k.tile[p.beta != 0.f][p.c_type == DGEMM_TYPE_F32];
        for (int split = 1; split <= 8; split *= 2) {
            if (split > 1 && (k.join == 0.0 || p.offsets || tiles * split > slots || nb < 2 * split)) break;
            const double waves = p.offsets ? std::max(1.0, tiles / slots) : std::ceil(tiles * split / slots);
            const double run = waves * (std::ceil(nb / split) * block + tile) + k.join * std::log2(split);
            offer({k.cfg.variant, k.cfg.bn, split}, kStart + std::max(run, bytes / kBytesUs));
        }
    }
    if (!p.offsets && p.M <= kF8DecodeTokens) {
        const double waves = std::max(1.0, static_cast<double>((p.N + 15) / 16) / (dev.sm_count * 4));
        offer({kF8Decode, 0, 8}, 3.5 + std::max(waves * std::ceil(nb / 8) * 1.1, bytes / kBytesUs));
    }
    return best;
}

const char *kernel_name(const F8Config &cfg)
{
    if (cfg.variant == kF8Decode) return cfg.split == 4 ? "f8_decode_4_warps" : "f8_decode_8_warps";
    if (cfg.variant == kF8Pair) return cfg.bn == 256 ? "f8_pair_256x256" : "f8_pair_256x128";
#define DGEMM_F8_SPLITS(name) {name, name "_split2", name "_split3", name "_split4", name "_split5", name "_split6", name "_split7", name "_split8"}
    static const char *const names[3][8] = {DGEMM_F8_SPLITS("f8_channels_128x16"), DGEMM_F8_SPLITS("f8_channels_128x32"),
                                            DGEMM_F8_SPLITS("f8_channels_128x64")};
#undef DGEMM_F8_SPLITS
    return names[cfg.bn == 16 ? 0 : cfg.bn == 32 ? 1 : 2][cfg.split - 1];
}

}  // namespace

int f8_tune_next(int variant, int bn, int split)
{
    const F8Config cfg{variant, bn, split};
    if (variant != kF8Auto && variant != kF8Any && !f8_umma_config_ok(cfg) && !f8_decode_config_ok(cfg))
        return DGEMM_ERR_INVALID_ARG;
    t_tune = cfg;
    return DGEMM_OK;
}

F8Config f8_take_tune()
{
    const F8Config cfg = t_tune;
    t_tune = {kF8Auto, 0, 1};
    return cfg;
}

const char *launch_gemm_f8(const F8Params &q, const F8Config &tune, cudaStream_t stream, const DeviceInfo &dev)
{
    F8Params p = q;
    // the pitch of a single row is never used
    if (p.M == 1) p.a.ld = (p.K + 15) / 16 * 16;
    if (p.N == 1) p.b.ld = (p.K + 15) / 16 * 16;
    // TMA's conditions, but for C's; the kernels that use it count rows in 32 bits, to the end of a tile
    constexpr int64_t kMost = INT32_MAX - 512;
    const bool tma = p.K > 0 && p.M <= kMost && p.N <= kMost && p.K <= kMost && aligned(p.a.p, p.a.ld, 1, 16) && aligned(p.b.p, p.b.ld, 1, 16) &&
                     (p.experts == 1 || (p.b_stride % 16 == 0 && p.b_stride > 0));
    if (tma && tune.variant != kF8Any) {
        auto run = [&](const F8Config &cfg) {
            return cfg.variant == kF8Decode ? launch_f8_decode(p, cfg, stream) : launch_f8_umma(p, cfg, stream);
        };
        F8Config cfg = tune;
        cfg.split = static_cast<int>(std::min<int64_t>(cfg.split, cfg.variant == kF8Channels ? (p.K - 1) / kF8Block + 1 : 8));
        if (cfg.variant == kF8Auto || !run(cfg)) {
            // (clusters that do not fit the GPU all at once are made smaller)
            for (cfg = choose(p, dev); !run(cfg); cfg.split /= 2)
                if (cfg.split == 1) return launch_any(p, stream, dev);
        }
        return kernel_name(cfg);
    }
    return launch_any(p, stream, dev);
}

}  // namespace dgemm

DGEMM_DEFINE_CHECK_READER(check_status_f8_gemm)
