// f8_rows.cu -- values to 8-bit floating point with a scale for each block of 128,
// and back.
//
//   a = max |y| over a block,  scale = a / top,  Q = f8(y * (top / a))
//
// A block is 128 columns of a row (quantize, swiglu, gather by expert), 128 x 128
// values, or 128 rows of a column (transposed).  All of it is FP32 arithmetic; the
// one rounding to fewer bits is Q's.
//
// The bound is HBM: each value is read once and its byte written once, so a
// block's values stay in registers between its maximum and its bytes.  A block of
// a row is 16 lanes of 8 elements: loads of 16 bytes a lane, the maximum in four
// shuffles, stores of 8 bytes a lane, without shared memory or barriers.
//
// 8192 x 8192, and the time of its bytes at the measured copy rate: bf16 rows 38.1 us
// (30.1), FP32 50.1 (50), gated bf16 59.7 (50), blocks of 128 x 128 bf16 31.3 (29.8) and FP32
// 51 (49.6), transposed bf16 39.3 (30.1), back to bf16 32.3 (30.1); 8192 tokens of 4096 bf16 to
// 8 rows each of an expert order 67.7 (50.9).  Of the 16-bit forms the
// instructions bound the rest: the conversion to 8 bits takes 21 values a clock and SM.
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "dgemm.h"
#include "f8.cuh"
#include "internal.h"

#define DGEMM_UNIT 10
#include "checked.cuh"
#include "rows.cuh"

namespace dgemm {
namespace {

enum { kOpQuantize = 0, kOpSwiglu = 1, kOpGather = 2 };

constexpr int kThreads = 256;
constexpr int kLanes = kF8Block / kVec;  // lanes of a block of a row
static_assert(kLanes == 16, "half a warp");

struct RowParams {
    uint32_t rows, cols, blocks;  // rows * blocks < 2^31
    const void *x, *u;            // u: swiglu's second factor
    int64_t ldx, ldu;
    uint8_t *q;
    int64_t ldq;
    float *scale;
    int64_t s_row, s_blk;
    const int32_t *position;      // gather: the `top` rows of Q that each row goes to,
    int64_t top, out_rows;        // of out_rows
};

template <bool kAligned>
__device__ __forceinline__ void store_bytes(uint8_t *p, int n, uint2 b)
{
    if (kAligned && n == kVec && DGEMM_CHECK((reinterpret_cast<uintptr_t>(p) & 7u) == 0)) {
        *reinterpret_cast<uint2 *>(p) = b;
        return;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? b.x : b.y) >> (8 * (i & 3)));
}

// The largest magnitude of a vector as bits of T, infinities above every finite one and NaNs
// above those: for 16-bit types by integer maxima of two values at a time.
template <typename T>
__device__ __forceinline__ uint32_t max_bits(const Raw<T> &r)
{
    if constexpr (sizeof(T) == 4) {
        float v[kVec];
        unpack(r, v);
        return __float_as_uint(max_abs(0.f, v)) & 0x7FFFFFFFu;
    } else {
        const uint32_t abs = 0x7FFF7FFFu;
        const uint32_t m = __vmaxu2(__vmaxu2(r.w[0].x & abs, r.w[0].y & abs), __vmaxu2(r.w[0].z & abs, r.w[0].w & abs));
        return max(m & 0xFFFFu, m >> 16);
    }
}

// Such bits as FP32's.
template <typename T>
__device__ __forceinline__ uint32_t bits_to_f32(uint32_t bits)
{
    if constexpr (std::is_same<T, float>::value)
        return bits;
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
        return bits << 16;
    else
        return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(bits))));
}

// A warp takes 2 * kMany consecutive blocks, two at a time, all of them loaded before the
// first is worked on.  Their maxima meet in one lane each, which forms the block's scale and
// factor: one division of either kind for all of them.  8192 x 8192, thread blocks an SM as
// the registers fall and six: bf16 rows 40.3 and 38.7 us, FP32 51.9 and 50.0, swiglu of bf16
// 61.3 and 59.5; two blocks a warp step at a time 45.5, sixteen 49.9.
template <int kOp, typename T, bool kAligned, bool kE5, int kMany>
__global__ void __launch_bounds__(kThreads, kAligned && (sizeof(T) == 2 || kOp == kOpQuantize) ? 6 : 2) f8_rows_kernel(const RowParams p)
{
    chain_wait();
    chain_next();
    const int lane = threadIdx.x & (kLanes - 1), half = (threadIdx.x >> 4) & 1;
    const uint32_t warp = threadIdx.x >> 5, total = p.rows * p.blocks;
    const uint32_t first = (blockIdx.x * (kThreads / 32) + warp) * (2 * kMany) + half;
    uint32_t row[kMany], col[kMany];
    int n[kMany];
    Raw<T> x[kMany], u[kMany];
    uint32_t r = first / p.blocks, b = first - r * p.blocks;
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
        row[i] = r;
        col[i] = b * kF8Block + lane * kVec;
        n[i] = r < p.rows && col[i] < p.cols ? static_cast<int>(min(p.cols - col[i], static_cast<uint32_t>(kVec))) : 0;
        x[i] = load_raw<T, kAligned>(static_cast<const T *>(p.x) + static_cast<int64_t>(row[i]) * p.ldx + col[i], n[i]);
        if constexpr (kOp == kOpSwiglu)
            u[i] = load_raw<T, kAligned>(static_cast<const T *>(p.u) + static_cast<int64_t>(row[i]) * p.ldu + col[i], n[i]);
        b += 2;
        while (b >= p.blocks) {
            b -= p.blocks;
            ++r;
        }
    }
    float v[kOp == kOpSwiglu ? kMany : 1][kVec];
    uint32_t mine = 0;  // of block `lane`: its largest magnitude, as bits of T (swiglu: FP32)
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
        uint32_t most;
        if constexpr (kOp == kOpSwiglu) {
            float w[kVec];
            unpack(x[i], v[i]);
            unpack(u[i], w);
#pragma unroll
            for (int k = 0; k < kVec; ++k) v[i][k] = silu(v[i][k]) * w[k];
            most = __float_as_uint(max_abs(0.f, v[i])) & 0x7FFFFFFFu;
        } else {
            most = max_bits(x[i]);
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
        if (lane == i) mine = most;
    }
    const F8Block<kE5> block(kOp == kOpSwiglu ? mine : bits_to_f32<T>(mine));
    const bool some_tiny = __any_sync(0xFFFFFFFFu, lane < kMany && block.tiny);
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
        float (&y)[kVec] = v[kOp == kOpSwiglu ? i : 0];
        if constexpr (kOp != kOpSwiglu) unpack(x[i], y);
        if (some_tiny) {
            const float times = __shfl_sync(0xFFFFFFFFu, block.tiny ? 0x1p100f : 1.f, half * kLanes + i);
#pragma unroll
            for (int k = 0; k < kVec; ++k) y[k] *= times;
        }
        const float inv = __shfl_sync(0xFFFFFFFFu, block.inv, half * kLanes + i);
        const uint2 bytes = f8_eight<kE5>(y, inv);
        const bool in = first + 2 * i < total;
        auto put = [&](int64_t to) {
            if (DGEMM_CHECK(col[i] + n[i] <= p.cols || n[i] == 0)) store_bytes<kAligned>(p.q + to * p.ldq + col[i], n[i], bytes);
            if (lane == i) p.scale[to * p.s_row + (col[i] / kF8Block) * p.s_blk] = block.scale;
        };
        if constexpr (kOp != kOpGather) {
            if (in) put(row[i]);
        } else if (in) {
            for (int64_t j = 0; j < p.top; ++j) {
                const int32_t to = p.position[row[i] * p.top + j];
                if (to >= 0 && to < p.out_rows) put(to);
            }
        }
    }
}

// ---- blocks of 128 x 128, and of 128 rows of a column

struct TileParams {
    int64_t rows, cols;
    const void *x;
    int64_t ldx;
    uint8_t *q;
    int64_t ldq;
    float *scale;
    int64_t s_row, s_blk;
    uint32_t tiles, tiles_c;
};

// 16 bytes from global to shared memory, of which `bytes` are read and the rest are zeros.
__device__ __forceinline__ void copy_async16(uint4 *dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(bytes)
                 : "memory");
}

constexpr int kTileSlots = 3;  // tiles of a thread block in shared memory: one worked on, two on their way

template <typename T>
constexpr size_t tile_smem()
{
    return static_cast<size_t>(kTileSlots) * kF8Block * kF8Block * sizeof(T);
}

// The columns that a thread has of a tile: eight in a row, or (FP32) four and, 64 on, four more,
// so that the 16-byte words of neighbouring threads lie side by side: copies of every other
// word read each sector of L2 twice (16384 x 8192 in blocks 169 us, and 110; 99 with the words'
// places worked out once a tile instead of once a row).
template <typename T>
struct TileCols {
    static constexpr bool kSplit = sizeof(T) == 4;
    static __device__ __forceinline__ int at(int lane, int k) { return kSplit ? (k >> 2) * 64 + lane * 4 + (k & 3) : lane * kVec + k; }
    static __device__ __forceinline__ int lane_of(int c) { return kSplit ? (c & 63) >> 2 : c / kVec; }
};

// A thread's eight bytes of a row at q (column c0 of the tile on, `left` columns there).
template <typename T, bool kAligned>
__device__ __forceinline__ void store_tile_bytes(uint8_t *q, int lane, int left, uint2 b)
{
    if constexpr (!TileCols<T>::kSplit) {
        store_bytes<kAligned>(q + lane * kVec, max(0, min(kVec, left - lane * kVec)), b);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = TileCols<T>::at(lane, 4 * h), n = left - c;
            const uint32_t w = h ? b.y : b.x;
            if (kAligned && n >= 4 && DGEMM_CHECK((reinterpret_cast<uintptr_t>(q + c) & 3u) == 0)) {
                *reinterpret_cast<uint32_t *>(q + c) = w;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < n) q[c + k] = static_cast<uint8_t>(w >> (8 * k));
            }
        }
    }
}

// A thread block takes one tile of 128 x 128 values after another, 8 vectors of it a thread,
// while the next two are on their way to shared memory (each thread fetches the vectors that
// it will use itself; rows off 16 bytes are loaded when their turn comes).
// kTransposed: thread t has rows 8 (t / 16) .. and the columns of t mod 16, so that each of
// its columns is one 8-byte word of a row of Q^T; the words meet in shared memory, word w of
// row c at w ^ (the thread that has it, mod 16), which keeps both the columns' stores and the
// rows' loads on distinct banks.
template <typename T, bool kAligned, bool kAlignedQ, bool kE5, bool kTransposed>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) f8_tile_kernel(const TileParams p)
{
    extern __shared__ uint4 slots[];  // [slot][vector][word][thread]
    using Cols = TileCols<T>;
    constexpr int kWords = Raw<T>::kWords, kPer = 16 / sizeof(T);
    __shared__ uint32_t s_most[kF8Block];
    __shared__ float s_inv[kF8Block];
    __shared__ uint2 s_word[kTransposed ? kF8Block * kLanes : 1];
    const int t = threadIdx.x, lane = t & (kLanes - 1), group = t / kLanes;
    auto row_of = [&](int i) { return kTransposed ? group * 8 + i : i * (kThreads / kLanes) + group; };
    auto origin = [&](uint32_t tile, int64_t &r0, int64_t &c0) {
        r0 = static_cast<int64_t>(tile / p.tiles_c) * kF8Block;
        c0 = static_cast<int64_t>(tile % p.tiles_c) * kF8Block;
    };
    auto slot_of = [&](int slot, int i, int w) { return slots + ((slot * 8 + i) * kWords + w) * kThreads + t; };
    auto fetch = [&](uint32_t tile, int slot) {
        if (kAligned && tile < p.tiles) {
            int64_t r0, c0;
            origin(tile, r0, c0);
            int64_t col[kWords];  // of this thread's words, and the elements there: the same in every row
            int in[kWords];
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                col[w] = c0 + Cols::at(lane, w * kPer);
                const int64_t left = p.cols - col[w];
                in[w] = left >= kPer ? kPer : left > 0 ? static_cast<int>(left) : 0;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t row = r0 + row_of(i);
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    const int n = row < p.rows ? in[w] : 0;
                    const T *src = static_cast<const T *>(p.x) + (n > 0 ? row * p.ldx + col[w] : 0);
                    copy_async16(slot_of(slot, i, w), src, n * static_cast<int>(sizeof(T)));
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    chain_wait();
    chain_next();
    int slot = 0;
    fetch(blockIdx.x, 0);
    fetch(blockIdx.x + gridDim.x, 1);
    for (uint32_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        int64_t r0, c0;
        origin(tile, r0, c0);
        const int cols = static_cast<int>(min(p.cols - c0, static_cast<int64_t>(kF8Block)));  // of the tile
        if (t < kF8Block) s_most[t] = 0u;
        fetch(tile + 2 * gridDim.x, slot >= 1 ? slot - 1 : kTileSlots - 1);  // (the slot of the tile before)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
        Raw<T> x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (kAligned) {
#pragma unroll
                for (int w = 0; w < kWords; ++w) x[i].w[w] = *slot_of(slot, i, w);
            } else {
                const int64_t row = r0 + row_of(i);
                const T *src = static_cast<const T *>(p.x) + (row < p.rows ? row * p.ldx + c0 : 0);
                alignas(16) T e[kVec];
#pragma unroll
                for (int k = 0; k < kVec; ++k)
                    e[k] = row < p.rows && Cols::at(lane, k) < cols ? src[Cols::at(lane, k)] : from_f32<T>(0.f);
#pragma unroll
                for (int w = 0; w < kWords; ++w) x[i].w[w] = reinterpret_cast<const uint4 *>(e)[w];
            }
        }
        slot = slot + 1 == kTileSlots ? 0 : slot + 1;
        __syncthreads();
        // the largest magnitude of the tile, or of each of this thread's columns
        if constexpr (!kTransposed) {
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float v[kVec];
                unpack(x[i], v);
                amax = max_abs(amax, v);
            }
            const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax) & 0x7FFFFFFFu);
            if ((t & 31) == 0) atomicMax(&s_most[0], most);
        } else {
            float most[kVec] = {};
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                float v[kVec], w[kVec];
                unpack(x[i], v);
                unpack(x[i + 1], w);
#pragma unroll
                for (int k = 0; k < kVec; ++k) most[k] = max3_abs(most[k], v[k], w[k]);
            }
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                uint32_t m = __float_as_uint(most[k]) & 0x7FFFFFFFu;
                m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));  // the warp's other eight rows
                if ((t & 16) == 0) atomicMax(&s_most[Cols::at(lane, k)], m);
            }
        }
        __syncthreads();
        if constexpr (!kTransposed) {
            const F8Block<kE5> block(s_most[0]);
            if (t == 0) p.scale[(r0 / kF8Block) * p.s_row + (c0 / kF8Block) * p.s_blk] = block.scale;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t row = r0 + row_of(i);
                float v[kVec];
                unpack(x[i], v);
                if (block.tiny) {
#pragma unroll
                    for (int k = 0; k < kVec; ++k) v[k] *= 0x1p100f;
                }
                if (row < p.rows && DGEMM_CHECK(c0 + cols <= p.cols))
                    store_tile_bytes<T, kAlignedQ>(p.q + row * p.ldq + c0, lane, cols, f8_eight<kE5>(v, block.inv));
            }
            __syncthreads();  // s_most has been read
        } else {
            bool tiny = false;
            if (t < kF8Block) {  // one thread a column: its scale and factor
                const F8Block<kE5> block(s_most[t]);
                s_inv[t] = block.inv;
                tiny = block.tiny;
                if (c0 + t < p.cols) p.scale[(c0 + t) * p.s_row + (r0 / kF8Block) * p.s_blk] = block.scale;
            }
            const bool some_tiny = __syncthreads_or(tiny) != 0;
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                const int c = Cols::at(lane, k);
                float y[kVec];  // the column's eight rows
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float v[kVec];
                    unpack(x[i], v);
                    y[i] = v[k];
                }
                if (some_tiny && __uint_as_float(s_most[c]) < 0x1p-100f) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] *= 0x1p100f;
                }
                s_word[c * kLanes + (group ^ lane)] = f8_eight<kE5>(y, s_inv[c]);
            }
            __syncthreads();
            const int left = vec_len(p.rows, r0 + lane * kVec);  // of this thread's word of each row of Q
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = i * (kThreads / kLanes) + group;
                if (c0 + c < p.cols)
                    store_bytes<kAlignedQ>(p.q + (c0 + c) * p.ldq + r0 + lane * kVec, left, s_word[c * kLanes + (lane ^ Cols::lane_of(c))]);
            }
            // (s_most is written again behind the barrier that the words are written behind; the
            // words behind the next tile's)
        }
    }
}

// ---- back

// `vecs` vectors of 8 elements to a row; rows * vecs < 2^31.
template <typename T, bool kAligned, bool kE5>
__global__ void __launch_bounds__(kThreads)
    f8_dequantize_kernel(uint32_t rows, uint32_t cols, uint32_t vecs, const F8Operand q, int64_t row0, T *x, int64_t ldx)
{
    chain_wait();
    chain_next();
    constexpr int kMany = 4;
    const uint32_t total = rows * vecs;
    const uint32_t first = blockIdx.x * (kThreads * kMany) + threadIdx.x;
    uint32_t row[kMany], col[kMany];
    uint2 b[kMany];
    float s[kMany];
    int n[kMany];
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
        const uint32_t g = first + i * kThreads;
        row[i] = g / vecs;
        col[i] = (g - row[i] * vecs) * kVec;
        n[i] = g < total ? static_cast<int>(min(cols - col[i], static_cast<uint32_t>(kVec))) : 0;
        b[i] = make_uint2(0u, 0u);
        s[i] = 0.f;
        if (n[i] == 0) continue;
        const int64_t r = row0 + row[i];
        const uint8_t *src = q.p + r * q.ld + col[i];
        if (kAligned && n[i] == kVec) {
            b[i] = *reinterpret_cast<const uint2 *>(src);
        } else {
            for (int k = 0; k < n[i]; ++k) {
                const uint32_t v = static_cast<uint32_t>(src[k]) << (8 * (k & 3));
                if (k < 4)
                    b[i].x |= v;
                else
                    b[i].y |= v;
            }
        }
        s[i] = q.scale[q.band(r) * q.s_row + (col[i] / kF8Block) * q.s_blk];
    }
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
        float v[kVec];
#pragma unroll
        for (int k = 0; k < kVec / 2; ++k) {
            const uint32_t h = f8x2_to_f16x2<kE5>(((k < 2 ? b[i].x : b[i].y) >> (16 * (k & 1))) & 0xFFFFu);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            v[2 * k] = f.x * s[i];
            v[2 * k + 1] = f.y * s[i];
        }
        if (n[i] > 0 && DGEMM_CHECK(row[i] < rows && col[i] + n[i] <= cols))
            store_vec<T, kAligned>(x + (row0 + row[i]) * ldx + col[i], n[i], v);
    }
}

// ---- host side

// Blocks of rows one launch takes, so that their number stays in 32 bits.
constexpr int64_t kMostUnits = INT32_MAX - kThreads * 8;

template <int kOp, typename T, bool kAligned, bool kE5>
bool launch_rows(const RowParams &p, cudaStream_t stream)
{
    // several blocks a warp where that leaves enough of them to fill the SMs
    constexpr int kMany = kOp == kOpSwiglu || sizeof(T) == 4 ? 2 : 4;
    const uint32_t total = p.rows * p.blocks;
    auto grid = [&](uint32_t many) { return (total + 2 * many * (kThreads / 32) - 1) / (2 * many * (kThreads / 32)); };
    if (grid(kMany) >= 152 * 4)
        return launch_chained(f8_rows_kernel<kOp, T, kAligned, kE5, kMany>, grid(kMany), kThreads, 0, stream, 1, p) == cudaSuccess;
    return launch_chained(f8_rows_kernel<kOp, T, kAligned, kE5, 1>, grid(1), kThreads, 0, stream, 1, p) == cudaSuccess;
}

template <int kOp, typename T>
const char *launch_rows_typed(int64_t rows, int64_t cols, const void *x, int64_t ldx, const void *u, int64_t ldu,
                              const dgemm_f8 &q, const int32_t *position, int64_t top, int64_t out_rows, cudaStream_t stream)
{
    const int64_t blocks = (cols - 1) / kF8Block + 1, most = kMostUnits / blocks;
    const bool ok = aligned(x, ldx, sizeof(T), 16) && (!u || aligned(u, ldu, sizeof(T), 16)) && aligned(q.data, q.ld, 1, 8);
    const bool e5 = q.type == DGEMM_F8_E5M2;
    for (int64_t r = 0; r < rows; r += most) {
        RowParams p{};
        p.rows = static_cast<uint32_t>(rows - r < most ? rows - r : most);
        p.cols = static_cast<uint32_t>(cols);
        p.blocks = static_cast<uint32_t>(blocks);
        p.x = static_cast<const T *>(x) + r * ldx;
        p.ldx = ldx;
        p.u = u ? static_cast<const T *>(u) + r * ldu : nullptr;
        p.ldu = ldu;
        const int64_t to = kOp == kOpGather ? 0 : r;
        p.q = static_cast<uint8_t *>(q.data) + to * q.ld;
        p.ldq = q.ld;
        p.scale = q.scale + to * q.scale_row;
        p.s_row = q.scale_row;
        p.s_blk = q.scale_blk;
        p.position = position ? position + r * top : nullptr;
        p.top = top;
        p.out_rows = out_rows;
        const bool done = ok ? (e5 ? launch_rows<kOp, T, true, true>(p, stream) : launch_rows<kOp, T, true, false>(p, stream))
                             : (e5 ? launch_rows<kOp, T, false, true>(p, stream) : launch_rows<kOp, T, false, false>(p, stream));
        if (!done) return nullptr;
    }
    return kOp == kOpQuantize ? "f8_quantize_rows" : kOp == kOpSwiglu ? "f8_swiglu_rows" : "f8_gather_rows";
}

template <int kOp>
const char *launch_rows_op(int type, int64_t rows, int64_t cols, const void *x, int64_t ldx, const void *u, int64_t ldu,
                           const dgemm_f8 &q, const int32_t *position, int64_t top, int64_t out_rows, cudaStream_t stream)
{
    switch (type) {
    case DGEMM_TYPE_F32: return launch_rows_typed<kOp, float>(rows, cols, x, ldx, u, ldu, q, position, top, out_rows, stream);
    case DGEMM_TYPE_F16: return launch_rows_typed<kOp, __half>(rows, cols, x, ldx, u, ldu, q, position, top, out_rows, stream);
    case DGEMM_TYPE_BF16: return launch_rows_typed<kOp, __nv_bfloat16>(rows, cols, x, ldx, u, ldu, q, position, top, out_rows, stream);
    default: return nullptr;
    }
}

template <typename T, bool kAligned, bool kAlignedQ, bool kE5, bool kTransposed>
bool launch_tile_kernel(const TileParams &p, cudaStream_t stream)
{
    auto kernel = f8_tile_kernel<T, kAligned, kAlignedQ, kE5, kTransposed>;
    constexpr size_t smem = kAligned ? tile_smem<T>() : 0;
    constexpr uint32_t most = 152 * (sizeof(T) == 2 ? 2 : 1);  // thread blocks that run at once
    if (smem > 0 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return false;
    return launch_chained(kernel, p.tiles < most ? p.tiles : most, kThreads, smem, stream, 1, p) == cudaSuccess;
}

template <typename T, bool kE5, bool kTransposed>
bool launch_tiles_aligned(const TileParams &p, cudaStream_t stream)
{
    const bool x = aligned(p.x, p.ldx, sizeof(T), 16), q = aligned(p.q, p.ldq, 1, 8);
    if (x && q) return launch_tile_kernel<T, true, true, kE5, kTransposed>(p, stream);
    if (x) return launch_tile_kernel<T, true, false, kE5, kTransposed>(p, stream);
    return launch_tile_kernel<T, false, false, kE5, kTransposed>(p, stream);
}

template <typename T>
const char *launch_tiles(int64_t rows, int64_t cols, const void *x, int64_t ldx, const dgemm_f8 &q, bool transposed,
                         cudaStream_t stream)
{
    const int64_t tiles_c = (cols - 1) / kF8Block + 1, tiles_r = (rows - 1) / kF8Block + 1;
    const int64_t most = kMostUnits / tiles_c;  // bands of one launch
    const bool e5 = q.type == DGEMM_F8_E5M2;
    for (int64_t b = 0; b < tiles_r; b += most) {
        const int64_t bands = tiles_r - b < most ? tiles_r - b : most, r = b * kF8Block;
        TileParams p{};
        p.rows = rows - r;
        p.cols = cols;
        p.x = static_cast<const T *>(x) + r * ldx;
        p.ldx = ldx;
        p.q = static_cast<uint8_t *>(q.data) + (transposed ? r : r * q.ld);
        p.ldq = q.ld;
        p.scale = q.scale + b * (transposed ? q.scale_blk : q.scale_row);
        p.s_row = q.scale_row;
        p.s_blk = q.scale_blk;
        p.tiles_c = static_cast<uint32_t>(tiles_c);
        p.tiles = static_cast<uint32_t>(bands * tiles_c);
        const bool done = transposed ? (e5 ? launch_tiles_aligned<T, true, true>(p, stream) : launch_tiles_aligned<T, false, true>(p, stream))
                                     : (e5 ? launch_tiles_aligned<T, true, false>(p, stream) : launch_tiles_aligned<T, false, false>(p, stream));
        if (!done) return nullptr;
    }
    return transposed ? "f8_quantize_transposed" : "f8_quantize_blocks";
}

template <typename T>
const char *launch_dequantize_typed(int64_t rows, int64_t cols, const dgemm_f8 &q, void *x, int64_t ldx, cudaStream_t stream)
{
    const int64_t vecs = (cols - 1) / kVec + 1, most = kMostUnits / vecs;
    const bool ok = aligned(q.data, q.ld, 1, 8) && aligned(x, ldx, sizeof(T), 16), e5 = q.type == DGEMM_F8_E5M2;
    for (int64_t r = 0; r < rows; r += most) {
        const uint32_t n = static_cast<uint32_t>(rows - r < most ? rows - r : most);
        const unsigned grid = static_cast<unsigned>((n * vecs + kThreads * 4 - 1) / (kThreads * 4));
        auto kernel = ok ? (e5 ? f8_dequantize_kernel<T, true, true> : f8_dequantize_kernel<T, true, false>)
                         : (e5 ? f8_dequantize_kernel<T, false, true> : f8_dequantize_kernel<T, false, false>);
        if (launch_chained(kernel, grid, kThreads, 0, stream, 1, n, static_cast<uint32_t>(cols), static_cast<uint32_t>(vecs),
                           f8_operand(q), r, static_cast<T *>(x), ldx) != cudaSuccess)
            return nullptr;
    }
    return "f8_dequantize";
}

}  // namespace

const char *launch_quantize_f8(int64_t rows, int64_t cols, const void *x, int64_t ldx, int type, bool transposed,
                               const dgemm_f8 &q, cudaStream_t stream)
{
    if (!transposed && q.block == 1)
        return launch_rows_op<kOpQuantize>(type, rows, cols, x, ldx, nullptr, 0, q, nullptr, 0, 0, stream);
    switch (type) {
    case DGEMM_TYPE_F32: return launch_tiles<float>(rows, cols, x, ldx, q, transposed, stream);
    case DGEMM_TYPE_F16: return launch_tiles<__half>(rows, cols, x, ldx, q, transposed, stream);
    case DGEMM_TYPE_BF16: return launch_tiles<__nv_bfloat16>(rows, cols, x, ldx, q, transposed, stream);
    default: return nullptr;
    }
}

const char *launch_swiglu_f8(int64_t rows, int64_t cols, const void *g, int64_t ldg, const void *u, int64_t ldu, int type,
                             const dgemm_f8 &q, cudaStream_t stream)
{
    return launch_rows_op<kOpSwiglu>(type, rows, cols, g, ldg, u, ldu, q, nullptr, 0, 0, stream);
}

const char *launch_gather_f8(int64_t tokens, int64_t top, int64_t cols, const void *x, int64_t ldx, int type,
                             const int32_t *position, int64_t rows, const dgemm_f8 &q, cudaStream_t stream)
{
    return launch_rows_op<kOpGather>(type, tokens, cols, x, ldx, nullptr, 0, q, position, top, rows, stream);
}

const char *launch_dequantize_f8(int64_t rows, int64_t cols, const dgemm_f8 &q, void *x, int64_t ldx, int type,
                                 cudaStream_t stream)
{
    switch (type) {
    case DGEMM_TYPE_F32: return launch_dequantize_typed<float>(rows, cols, q, x, ldx, stream);
    case DGEMM_TYPE_F16: return launch_dequantize_typed<__half>(rows, cols, q, x, ldx, stream);
    case DGEMM_TYPE_BF16: return launch_dequantize_typed<__nv_bfloat16>(rows, cols, q, x, ldx, stream);
    default: return nullptr;
    }
}

}  // namespace dgemm

DGEMM_DEFINE_CHECK_READER(check_status_f8_rows)
