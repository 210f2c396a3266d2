// experts.cu -- tokens sorted by expert and back.
//
//   sort     position[t, j] = rank of pair (t, j) by (expert, t, j);  offsets[e]
//   gather   Y[position[t, j]] = X[t]
//   combine  X[t] = sum_j w[t, j] Y[position[t, j]] + beta X[t]
//   grad     dY[position[t, j]] = w[t, j] dX[t],  dw[t, j] = <dX[t], Y[position[t, j]]>
//
// The row movers are bound by HBM.  Each is driven by the tokens: a token's row is
// read (or written) once, whatever the number of its experts, and since the rows
// of different pairs differ, nothing is added atomically and results do not depend
// on timing.  4096 tokens of 8 rows of 4096 bf16: gather 45.9 us (6.6 TB/s), combine
// 44.8 (6.7), grad 93.8 (6.4; reads and writes mixed).  The sort is bound by latency: a
// counting sort in one launch.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "dgemm.h"
#include "f8.cuh"
#include "internal.h"
#include "ptx.cuh"

#define DGEMM_UNIT 13
#include "checked.cuh"
#include "rows.cuh"

namespace dgemm {
namespace {

constexpr int kThreads = 256;

// ---- sort: every warp counts a contiguous range of the pairs, the counts are
// added up over warps, CTAs and experts, and the warp walks its range again.
// Equal experts of 32 pairs find each other by votes, one for each bit of the number, so
// that counts and ranks need no atomics and the order of pairs is kept.  (match.any takes as
// many steps as there are different numbers: 65536 pairs, 64 experts, 18.0 and 8.0 us.)  Many
// pairs are shared by a cluster of 8 CTAs, whose counts meet through distributed shared
// memory: 8192 pairs 4.0 us, by one CTA 7.2.  16 tokens of 8 experts take 1.9 us.

constexpr int kSortHold = 8;       // pairs of a lane that stay in registers between the walks
constexpr int kSortWarps = 32;
constexpr unsigned kSortCluster = 8;
constexpr int64_t kSortFew = 2048;  // pairs up to which one CTA takes them (3.7 us; eight 3.8)

// The lanes of the warp whose keys equal this one's, below their bit `bits`.
__device__ __forceinline__ uint32_t same_key(uint32_t key, uint32_t bits)
{
    uint32_t same = 0xFFFFFFFFu;
    for (uint32_t b = 0; b < bits; ++b) {
        const uint32_t set = __ballot_sync(0xFFFFFFFFu, (key >> b) & 1u);
        same &= (key >> b) & 1u ? set : ~set;
    }
    return same;
}

template <typename Id>
__global__ void __launch_bounds__(kSortWarps * 32)
    sort_kernel(uint32_t n, uint32_t per_warp, uint32_t experts, const Id *ids, int32_t *offsets, int32_t *position)
{
    extern __shared__ uint32_t s[];  // counts of [warp][expert], of the CTA, of all CTAs, first rows
    const uint32_t warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    uint32_t *count = s + warp * experts, *total = s + warps * experts, *all = total + experts, *first = all + experts;
    for (uint32_t i = threadIdx.x; i < warps * experts; i += blockDim.x) s[i] = 0u;
    chain_wait();
    chain_next();
    __syncthreads();
    const uint32_t clusters = ptx::cluster_nctarank(), cta = ptx::cluster_ctarank();
    const uint32_t begin = min(n, (cta * warps + warp) * per_warp), end = min(n, begin + per_warp);
    const uint32_t bits = 32u - static_cast<uint32_t>(__clz(static_cast<int>(experts)));  // (of ~0 they make no expert)
    uint32_t key[kSortHold], same[kSortHold];  // an expert, or ~0; the lanes that have it too
    auto fetch = [&](uint32_t i0) {
#pragma unroll
        for (int k = 0; k < kSortHold; ++k) {
            const uint32_t i = i0 + k * 32 + lane;
            key[k] = ~0u;
            if (i < end) {
                const Id id = ids[i];
                if (id >= 0 && id < static_cast<Id>(experts)) key[k] = static_cast<uint32_t>(id);
            }
        }
    };
    for (uint32_t i0 = begin; i0 < end; i0 += kSortHold * 32) {
        fetch(i0);
#pragma unroll
        for (int k = 0; k < kSortHold; ++k) {
            if (i0 + k * 32 >= end) break;  // warp-uniform
            same[k] = same_key(key[k], bits);
            if (key[k] != ~0u && lane == static_cast<uint32_t>(__ffs(same[k])) - 1) count[key[k]] += __popc(same[k]);
            __syncwarp();
        }
    }
    __syncthreads();
    // the pairs of warps before, and of the CTA
    for (uint32_t e = threadIdx.x; e < experts; e += blockDim.x) {
        uint32_t sum = 0;
        for (uint32_t w = 0; w < warps; ++w) {
            const uint32_t c = s[w * experts + e];
            s[w * experts + e] = sum;
            sum += c;
        }
        total[e] = sum;
    }
    // every CTA's counts, and those of the CTAs before
    if (clusters > 1) {
        ptx::cluster_sync();
        for (uint32_t e = threadIdx.x; e < experts; e += blockDim.x) {
            uint32_t sum = 0, before = 0;
#pragma unroll
            for (uint32_t c = 0; c < kSortCluster; ++c) {
                const uint32_t v = __float_as_uint(ptx::ld_shared_cluster_f32(ptx::mapa(ptx::smem_addr(total + e), c)));
                sum += v;
                if (c < cta) before += v;
            }
            all[e] = sum;
            first[e] = before;
        }
    }
    __syncthreads();
    // experts before: a scan by one warp
    if (warp == 0) {
        uint32_t carry = 0;
        for (uint32_t e0 = 0; e0 < experts; e0 += 32) {
            const uint32_t e = e0 + lane;
            const uint32_t own = e < experts ? clusters > 1 ? all[e] : total[e] : 0u;
            uint32_t up = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, up, o);
                if (lane >= static_cast<uint32_t>(o)) up += v;
            }
            if (e < experts) {
                first[e] = carry + up - own + (clusters > 1 ? first[e] : 0u);
                if (cta == 0) offsets[e] = static_cast<int32_t>(carry + up - own);
            }
            carry += __shfl_sync(0xFFFFFFFFu, up, 31);
        }
        if (cta == 0 && lane == 0) offsets[experts] = static_cast<int32_t>(carry);
    }
    if (clusters > 1)
        ptx::cluster_sync();  // (no CTA leaves while another reads its counts)
    else
        __syncthreads();
    const bool held = end - begin <= kSortHold * 32;  // `key` and `same` still hold the whole range
    for (uint32_t i0 = begin; i0 < end; i0 += kSortHold * 32) {
        if (!held) fetch(i0);
#pragma unroll
        for (int k = 0; k < kSortHold; ++k) {
            if (i0 + k * 32 >= end) break;
            const uint32_t i = i0 + k * 32 + lane;
            if (!held) same[k] = same_key(key[k], bits);
            const uint32_t rank = __popc(same[k] & ((1u << lane) - 1u));
            uint32_t at = 0;
            if (key[k] != ~0u) at = first[key[k]] + count[key[k]] + rank;
            __syncwarp();
            if (key[k] != ~0u && rank == 0) count[key[k]] += __popc(same[k]);
            __syncwarp();
            if (i < end && DGEMM_CHECK(key[k] == ~0u || at < n)) position[i] = key[k] == ~0u ? -1 : static_cast<int32_t>(at);
        }
    }
}

template <typename Id>
bool launch_sort(int64_t n, int experts, const void *ids, int32_t *offsets, int32_t *position, cudaStream_t stream)
{
    const unsigned cluster = n > kSortFew ? kSortCluster : 1;
    // a warp for each 32 pairs, up to all of them
    const unsigned warps = static_cast<unsigned>(std::min<int64_t>(kSortWarps, std::max<int64_t>(4, (n + 31) / 32)));
    const uint32_t per = static_cast<uint32_t>((n + cluster * warps - 1) / (cluster * warps) + 31) / 32 * 32;
    const size_t smem = (static_cast<size_t>(warps) + 3) * experts * 4;
    auto kernel = sort_kernel<Id>;
    if (smem > 48 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (kSortWarps + 3) * kMaxExperts * 4) != cudaSuccess)
        return false;
    return launch_chained(kernel, cluster, warps * 32, smem, stream, cluster, static_cast<uint32_t>(n), per,
                          static_cast<uint32_t>(experts), static_cast<const Id *>(ids), offsets, position) == cudaSuccess;
}

// ---- rows

struct MoveParams {
    uint32_t tokens, cols, vecs;  // vectors of 8 elements to a row; tokens * vecs < 2^31
    int64_t top, rows;            // rows of y
    const void *x;                // a token's row: what gather reads, combine's old X
    int64_t ldx;
    void *y;                      // sorted rows: what gather writes, combine reads
    int64_t ldy;
    void *out;                    // combine: the new X (x's place)
    const int32_t *position;
    const float *weights;
    float beta;
};

// The row of pair j of a token, or -1.
__device__ __forceinline__ int32_t row_of(const int32_t *position, int64_t pair, int64_t rows)
{
    const int32_t r = position[pair];
    return r >= 0 && r < rows ? r : -1;
}

template <typename T, bool kAligned>
__device__ __forceinline__ void store_raw(T *p, int n, const Raw<T> &r)
{
    if (kAligned && n == kVec && DGEMM_CHECK((reinterpret_cast<uintptr_t>(p) & 15u) == 0)) {
#pragma unroll
        for (int i = 0; i < Raw<T>::kWords; ++i) reinterpret_cast<uint4 *>(p)[i] = r.w[i];
        return;
    }
    const T *e = reinterpret_cast<const T *>(r.w);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (i < n) p[i] = e[i];
}

// A thread copies one vector of a token to each of the token's rows.
template <typename T, bool kAligned>
__global__ void __launch_bounds__(kThreads) gather_kernel(const MoveParams p)
{
    chain_wait();
    chain_next();
    const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t t = g / p.vecs, col = (g - t * p.vecs) * kVec;
    if (t >= p.tokens) return;
    const int n = static_cast<int>(min(p.cols - col, static_cast<uint32_t>(kVec)));
    const Raw<T> x = load_raw<T, kAligned>(static_cast<const T *>(p.x) + t * p.ldx + col, n);
    for (int64_t j = 0; j < p.top; ++j) {
        const int32_t r = row_of(p.position, t * p.top + j, p.rows);
        if (r >= 0 && DGEMM_CHECK(col + n <= p.cols)) store_raw<T, kAligned>(static_cast<T *>(p.y) + r * p.ldy + col, n, x);
    }
}

constexpr int kBatch = 8;  // pairs of a token whose rows are loaded together

// A thread adds up one vector of a token over its rows, in the order of the pairs.
template <typename T, bool kAligned>
__global__ void __launch_bounds__(kThreads) combine_kernel(const MoveParams p)
{
    chain_wait();
    chain_next();
    const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t t = g / p.vecs, col = (g - t * p.vecs) * kVec;
    if (t >= p.tokens) return;
    const int n = static_cast<int>(min(p.cols - col, static_cast<uint32_t>(kVec)));
    float sum[kVec] = {};
    for (int64_t j0 = 0; j0 < p.top; j0 += kBatch) {
        Raw<T> y[kBatch];
        float w[kBatch];
        bool in[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t pair = t * p.top + j0 + j;
            const int32_t r = j0 + j < p.top ? row_of(p.position, pair, p.rows) : -1;
            in[j] = r >= 0;
            w[j] = in[j] && p.weights ? p.weights[pair] : 1.f;
            y[j] = load_raw<T, kAligned>(static_cast<const T *>(p.y) + (in[j] ? r * p.ldy + col : 0), in[j] ? n : 0);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            float v[kVec];
            unpack(y[j], v);
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (in[j]) sum[i] = fmaf(w[j], v[i], sum[i]);
        }
    }
    if (p.beta != 0.f) {
        float v[kVec];
        unpack(load_raw<T, kAligned>(static_cast<const T *>(p.x) + t * p.ldx + col, n), v);
#pragma unroll
        for (int i = 0; i < kVec; ++i) sum[i] = fmaf(p.beta, v[i], sum[i]);
    }
    if (DGEMM_CHECK(col + n <= p.cols)) store_vec<T, kAligned>(static_cast<T *>(p.out) + t * p.ldx + col, n, sum);
}

struct GradParams {
    int64_t cols, top, rows;
    const void *dx;
    int64_t lddx;
    const void *y;
    int64_t ldy;
    const int32_t *position;
    const float *weights;
    void *dy;
    int64_t lddy;
    float *dw;
};

// A block takes a token: its gradient row meets the rows of kBatch pairs at a time.
template <typename T, bool kAligned>
__global__ void __launch_bounds__(kThreads) combine_grad_kernel(const GradParams p)
{
    __shared__ float s_dot[kThreads / 32][kBatch];
    chain_wait();
    chain_next();
    const int64_t t = blockIdx.x;
    const int warps = static_cast<int>(blockDim.x) / 32;
    for (int64_t j0 = 0; j0 < p.top; j0 += kBatch) {
        int32_t r[kBatch];
        float w[kBatch], dot[kBatch] = {};
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t pair = t * p.top + j0 + j;
            r[j] = j0 + j < p.top ? row_of(p.position, pair, p.rows) : -1;
            w[j] = r[j] >= 0 ? p.weights[pair] : 0.f;
        }
        for (int64_t c = threadIdx.x * kVec; c < p.cols; c += static_cast<int64_t>(blockDim.x) * kVec) {
            const int n = vec_len(p.cols, c);
            float d[kVec];
            Raw<T> y[kBatch];
            const Raw<T> raw = load_raw<T, kAligned>(static_cast<const T *>(p.dx) + t * p.lddx + c, n);
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                y[j] = load_raw<T, kAligned>(static_cast<const T *>(p.y) + (r[j] >= 0 ? r[j] * p.ldy + c : 0), r[j] >= 0 ? n : 0);
            unpack(raw, d);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (r[j] < 0) continue;  // block-uniform
                float v[kVec], o[kVec];
                unpack(y[j], v);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    dot[j] = fmaf(d[i], v[i], dot[j]);
                    o[i] = w[j] * d[i];
                }
                if (DGEMM_CHECK(c + n <= p.cols)) store_vec<T, kAligned>(static_cast<T *>(p.dy) + r[j] * p.lddy + c, n, o);
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], o);
            if ((threadIdx.x & 31) == 0) s_dot[threadIdx.x >> 5][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < kBatch && j0 + threadIdx.x < p.top) {
            float sum = 0.f;
            for (int v = 0; v < warps; ++v) sum += s_dot[v][threadIdx.x];
            p.dw[t * p.top + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

// ---- host side

template <typename T>
bool launch_moves(bool combine, int64_t tokens, int64_t cols, MoveParams p, cudaStream_t stream)
{
    const int64_t vecs = (cols - 1) / kVec + 1, most = (INT32_MAX - kThreads) / vecs;
    const bool ok = aligned(p.x, p.ldx, sizeof(T), 16) && aligned(p.y, p.ldy, sizeof(T), 16);
    const void *x = p.x;
    const int32_t *position = p.position;
    const float *weights = p.weights;
    for (int64_t t = 0; t < tokens; t += most) {
        p.tokens = static_cast<uint32_t>(std::min(tokens - t, most));
        p.cols = static_cast<uint32_t>(cols);
        p.vecs = static_cast<uint32_t>(vecs);
        p.x = static_cast<const T *>(x) + t * p.ldx;
        p.out = const_cast<void *>(p.x);
        p.position = position + t * p.top;
        p.weights = weights ? weights + t * p.top : nullptr;
        auto kernel = combine ? (ok ? combine_kernel<T, true> : combine_kernel<T, false>)
                              : (ok ? gather_kernel<T, true> : gather_kernel<T, false>);
        const unsigned grid = static_cast<unsigned>((p.tokens * vecs + kThreads - 1) / kThreads);
        if (launch_chained(kernel, grid, kThreads, 0, stream, 1, p) != cudaSuccess) return false;
    }
    return true;
}

template <typename T>
bool launch_grad(int64_t tokens, const GradParams &p, cudaStream_t stream)
{
    const bool ok = aligned(p.dx, p.lddx, sizeof(T), 16) && aligned(p.y, p.ldy, sizeof(T), 16) && aligned(p.dy, p.lddy, sizeof(T), 16);
    const int64_t vecs = (p.cols - 1) / kVec + 1;
    const unsigned threads = static_cast<unsigned>(std::min<int64_t>(kThreads, (vecs + 31) / 32 * 32));
    return launch_chained(ok ? combine_grad_kernel<T, true> : combine_grad_kernel<T, false>, static_cast<unsigned>(tokens),
                          threads, 0, stream, 1, p) == cudaSuccess;
}

}  // namespace

const char *launch_sort_by_expert(int64_t pairs, int experts, const void *ids, int id_bytes, int32_t *offsets,
                                  int32_t *position, cudaStream_t stream)
{
    const bool done = id_bytes == 8 ? launch_sort<int64_t>(pairs, experts, ids, offsets, position, stream)
                                    : launch_sort<int32_t>(pairs, experts, ids, offsets, position, stream);
    return done ? "sort_by_expert" : nullptr;
}

const char *launch_gather(int64_t tokens, int64_t top, int64_t cols, const void *x, int64_t ldx, int type,
                          const int32_t *position, int64_t rows, void *y, int64_t ldy, cudaStream_t stream)
{
    MoveParams p{};
    p.top = top;
    p.rows = rows;
    p.x = x;
    p.ldx = ldx;
    p.y = y;
    p.ldy = ldy;
    p.position = position;
    // (bits are copied: one 16-bit type stands for both)
    const bool done = type == DGEMM_TYPE_F32 ? launch_moves<float>(false, tokens, cols, p, stream)
                                             : launch_moves<__half>(false, tokens, cols, p, stream);
    return done ? "gather_by_expert" : nullptr;
}

const char *launch_combine(int64_t tokens, int64_t top, int64_t cols, const void *y, int64_t ldy, int64_t rows, int type,
                           const int32_t *position, const float *weights, float beta, void *x, int64_t ldx, cudaStream_t stream)
{
    MoveParams p{};
    p.top = top;
    p.rows = rows;
    p.x = x;
    p.ldx = ldx;
    p.y = const_cast<void *>(y);
    p.ldy = ldy;
    p.position = position;
    p.weights = weights;
    p.beta = beta;
    bool done = false;
    switch (type) {
    case DGEMM_TYPE_F32: done = launch_moves<float>(true, tokens, cols, p, stream); break;
    case DGEMM_TYPE_F16: done = launch_moves<__half>(true, tokens, cols, p, stream); break;
    case DGEMM_TYPE_BF16: done = launch_moves<__nv_bfloat16>(true, tokens, cols, p, stream); break;
    }
    return done ? "combine_experts" : nullptr;
}

const char *launch_combine_grad(int64_t tokens, int64_t top, int64_t cols, const void *dx, int64_t lddx, const void *y,
                                int64_t ldy, int64_t rows, int type, const int32_t *position, const float *weights, void *dy,
                                int64_t lddy, float *dw, cudaStream_t stream)
{
    const GradParams p{cols, top, rows, dx, lddx, y, ldy, position, weights, dy, lddy, dw};
    bool done = false;
    switch (type) {
    case DGEMM_TYPE_F32: done = launch_grad<float>(tokens, p, stream); break;
    case DGEMM_TYPE_F16: done = launch_grad<__half>(tokens, p, stream); break;
    case DGEMM_TYPE_BF16: done = launch_grad<__nv_bfloat16>(tokens, p, stream); break;
    }
    return done ? "combine_experts_grad" : nullptr;
}

}  // namespace dgemm

DGEMM_DEFINE_CHECK_READER(check_status_experts)
