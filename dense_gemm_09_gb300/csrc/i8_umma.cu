// i8_umma.cu -- gemm_i8_tn on the tensor cores (tcgen05).
//
//   C[m, n] = scale_a[m] * scale_b[n] * sum_k A[m, k] B[n, k] + bias[n] + beta * C[m, n]
//
// The mathematics.  GB300's integer tensor rate is a small fraction of its
// FP16 rate, but every int8 value is exact in FP16, a product of two is exact
// in FP32, and sums of such products are exact while they stay below 2^24
// (K <= 1024 always; real data far longer), so the product runs on
// kind::f16 with FP32 accumulators in tensor memory and up to there loses nothing
// to an integer one.  Past 2^24 the accumulator truncates at every MMA (16384
// products of one sign: 4.8e-5 of the sum on average, always towards zero).
// Operands stay int8 in HBM and L2 and on their way into the SM; they are
// widened to FP16 inside it.
//
// What bounds it.  The tensor pipe, once shared memory is kept out of the way:
// each SM moves 128 bytes a clock through it, and a K step of 64 costs a CTA of
// a pair (256 x 192 tiles) 14 KB written by TMA, 14 KB read by the
// converters, 12 KB of widened columns written and 12 KB read by the MMAs,
// against 384 clocks of MMA.  So the operand that supplies the MMA's rows
// never goes back to shared memory: its converter warps store it to tensor
// memory (tcgen05.st) and the MMAs take A from there.  That leaves 52 KB, 416
// clocks; with both operands widened in shared memory it would be 84 KB, 672
// clocks.  Measured with operands in place, an MMA of K = 16 takes N / 2 + 10
// clocks with A in tensor memory (N / 2 + 43 with A in shared memory): 848
// clocks for 128 K values at N = 192, and the kernel takes 850.  8192 x 8192 x
// 4096 to bf16: 295 us, 1865 TFLOP/s, 96 % of the measured bf16 GEMM rate
// (up to 327 us in a long run, where the power limit sets the clock: 98 % of
// the rate that is sustained there).
//
// Roles (32 warps, one CTA an SM):
//   warp 0       TMA producer: 128-byte rows (128 K values) of both operands
//                into a ring of raw stages (128-byte swizzle);
//   warps 8-19   row converters, three groups of four that take the halves (64
//                K values) of the raw stages in turn: warp w widens rows 32 (w
//                mod 4) .. into its own TMEM lanes, 32 columns a half;
//   warps 20-31  column converters, in turn too: the other operand, K-major
//                FP16 in shared memory (128-byte swizzle);
//   warp 1       MMA issuer: four tcgen05.mma of K = 16 a half, then a commit that
//                releases the half;
//   warps 4-7    epilogue: accumulator -> scale, bias, beta -> C.
// Two to four converted stages are in flight.  A converter reads and widens
// its part of a stage into registers before it waits for the
// half's last MMAs, so that only the store, the hand-off and the commit lie
// between the release of a half and its next use.  A half takes a converter
// group ~700 clocks from its first wait to its arrival, nearly all of it
// latency; three groups keep a stage at 2/3 of that.
// A CTA pair (cta_group::2) shares one MMA: each CTA widens its own 128 rows
// and half of the columns, and all of the pair's converters arrive on the
// leader's barrier.
//
// "Rows" are A's tokens (kSwap = false) or B's channels (kSwap = true: the
// accumulator holds C^T, for few tokens).  Tiles that all run at once have one
// accumulator of up to 256 columns; a CTA of several tiles has two of up to
// 192, so that one drains while the next fills.
#include <algorithm>
#include <climits>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include <cuda.h>
#include <cuda_runtime.h>

#include "bounded_wait.cuh"
#include "chained.cuh"
#include "dgemm.h"
#include "i8_gemm.h"
#include "internal.h"
#include "ptx.cuh"

#define DGEMM_UNIT 8
#include "checked.cuh"

namespace dgemm {
namespace {

constexpr int kRows = 128;                      // accumulator rows of a CTA: TMEM lanes
constexpr int kRowBytes = 128;                  // K values of a raw stage, one byte each
constexpr int kRawRowsBytes = kRows * kRowBytes;
constexpr int kHalfK = 64;                      // K values of a converted half
constexpr int kMaxBn = 256;                     // tile columns
constexpr int kMaxBn2 = 192;                    // with a second accumulator, for CTAs of several tiles
constexpr int kMaxSplitBn = 128;                // of a single CTA's tile
constexpr int kMaxRaw = 8;                      // raw stages
constexpr int kMaxConv = 4;                     // converted stages, of two halves each
constexpr int kConvCols = kHalfK / 2;           // TMEM columns of a half's rows: two FP16 values a column
constexpr int kTmemCols = 512;                  // one or two accumulators of bn columns, then the converted rows
static_assert(kMaxBn + 2 * 2 * kConvCols <= kTmemCols && 2 * kMaxBn2 + 2 * 2 * kConvCols <= kTmemCols,
              "two converted stages fit beside any accumulators");
constexpr int kBoxBytes = 4096;                 // epilogue staging: 32 rows x 128 bytes
constexpr int kEpiWarps = 4;
constexpr int kConvGroups = 3;                  // converter groups of four warps, of either kind
constexpr int kThreads = 32 * (8 + 2 * 4 * kConvGroups);
static_assert(kThreads <= 1024, "one CTA");
constexpr int kSmemLimit = 227 * 1024;

struct Ctrl {
    uint64_t raw_full[kMaxRaw];    // a raw stage has landed
    uint64_t raw_empty[kMaxRaw];   // its 16 converter warps have read it
    uint64_t conv_full[kMaxConv];  // leader: every converter warp of the pair has stored its part of the stage
    uint64_t conv_empty[2 * kMaxConv];  // the MMAs have read this converted half
    uint64_t acc_full[2];
    uint64_t acc_empty[2];         // leader: every epilogue warp of the pair has read the accumulator
    uint64_t mma_done;
    uint64_t never;                // test hook: a barrier nothing arrives at
    WaitCtl wait;
    uint32_t tmem_base;
    alignas(16) float scale[kMaxBn];  // of the tile's columns
    alignas(16) float bias[kMaxBn];   // (kSwap = false)
};

struct Params {
    I8Params c;
    int64_t rows, cols;            // of the accumulator matrix: (M, N), or (N, M) with kSwap
    uint32_t tiles_r, tiles_c;     // their product is below 2^31
    int bn;                        // tile columns; a CTA of a pair converts half of them
    int num_kb;                    // K blocks of 128
    int raw_stages, raw_bytes;
    int conv_stages;               // 2 .. kMaxConv
    int conv_col;                  // first TMEM column of the converted rows: the accumulators' columns
    int splitk;                    // CTAs of a cluster that share a tile (single CTAs)
    int tma_store;
    uint64_t wait_limit_ns;
    int inject_stall;
};

// ---- PTX beyond ptx.cuh

// As ptx::umma<0> / ptx::umma_pair<0> with A in tensor memory.
template <int kCtas>
__device__ __forceinline__ void umma_a_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate)
{
    if constexpr (kCtas == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Arrive on the barrier at this offset in every CTA of the pair (or in this
// CTA) when the MMAs issued so far by this thread complete.
template <int kCtas>
__device__ __forceinline__ void commit_all(uint32_t bar)
{
    if constexpr (kCtas == 2)
        ptx::umma_commit_pair_multicast(bar, 0x3);
    else
        ptx::umma_commit(bar);
}

__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// Arrive on an mbarrier of another CTA of the cluster with release at CTA
// scope: what it publishes is this CTA's tensor memory and, fenced to the async
// proxy, its shared memory, which this SM's own half of the pair's MMA reads;
// no thread of the other CTA does.  (A release at cluster scope waits ~650
// clocks for every earlier store of the thread to be acknowledged.)
__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// True in one thread of the (converged) warp.  The compiler keeps the operands
// of tcgen05 instructions under this predicate in uniform registers.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Meet the other CTA of the cluster without ordering memory.  (A releasing
// arrival waits for all earlier stores, up to ~1 us.)
__device__ __forceinline__ void cluster_meet()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ void fence_cluster()
{
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

__device__ __forceinline__ void named_barrier(uint32_t id, uint32_t threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---- int8 -> FP16

// Four int8 values as two FP16 pairs, exactly: flipping the sign bit gives
// v + 128 as an unsigned byte; under the exponent byte 0x64 it is the FP16
// number 1024 + (v + 128), from which 1152 is subtracted without rounding.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x5140), b = __byte_perm(u, 0x64646464u, 0x7362);
    const uint32_t bias = 0x64806480u;  // 1152, 1152
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&bias));
    const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), *reinterpret_cast<const __half2 *>(&bias));
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}

// Sixteen int8 values (one chunk of a raw row) as eight FP16 pairs.
__device__ __forceinline__ void widen16(const uint4 &c, uint32_t *out)
{
    widen4(c.x, out[0], out[1]);
    widen4(c.y, out[2], out[3]);
    widen4(c.z, out[4], out[5]);
    widen4(c.w, out[6], out[7]);
}

// ---- schedule

// The work of one CTA (pair): tiles t0, t0 + dt, ..., and of each the raw K
// blocks [kb0, kb1) (all of them, or with split-K the r-th of S near-equal
// ranges for rank r of the cluster).
struct Sched {
    uint32_t t0, dt;
    int kb0, kb1;
};

template <int kCtas>
__device__ __forceinline__ Sched schedule(const Params &p)
{
    Sched s;
    const uint32_t S = kCtas == 1 ? static_cast<uint32_t>(p.splitk) : 1u;
    s.t0 = blockIdx.x;
    s.dt = gridDim.x;
    s.kb0 = 0;
    s.kb1 = p.num_kb;
    if constexpr (kCtas == 2) {
        s.t0 >>= 1;
        s.dt >>= 1;
    } else if (S > 1) {
        const uint32_t r = ptx::cluster_ctarank();
        s.t0 /= S;
        s.dt /= S;
        s.kb0 = static_cast<int>(r * static_cast<uint32_t>(p.num_kb) / S);
        s.kb1 = static_cast<int>((r + 1) * static_cast<uint32_t>(p.num_kb) / S);
    }
    return s;
}

// Tile t in groups of 8 tile columns: tiles in flight together share a few
// bands of either operand.
__device__ __forceinline__ void tile_origin(const Params &p, uint32_t t, int tile_rows, int64_t &r0, int64_t &c0)
{
    constexpr uint32_t kGroup = 8;
    const uint32_t per_group = kGroup * p.tiles_r;
    const uint32_t g = t / per_group, r = t - g * per_group;
    const uint32_t left = p.tiles_c - g * kGroup;
    const uint32_t gc = left < kGroup ? left : kGroup;
    const uint32_t row = r / gc;
    c0 = static_cast<int64_t>(g * kGroup + r - row * gc) * p.bn;
    r0 = static_cast<int64_t>(row) * tile_rows;
}

// ---- roles

// Bounded waits of a whole converged warp.  Every step is decided by a vote, so
// that no branch diverges: a divergent wait (one lane probing, or a per-thread
// loop) costs hundreds of clocks in reconvergence on each half.  False for the
// whole warp on time-out or abort.
template <bool kCluster>
__device__ __forceinline__ bool probe(uint32_t bar, uint32_t parity)
{
    return __all_sync(0xFFFFFFFFu, kCluster ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity));
}

template <bool kCluster>
__device__ __noinline__ bool warp_wait_slow(uint32_t bar, uint32_t parity, WaitCtl *wc)
{
#pragma unroll 1
    for (int i = 0; i < 4; ++i)
        if (probe<kCluster>(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns(), limit = wc->limit_ns;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (probe<kCluster>(bar, parity)) return true;
        if (__any_sync(0xFFFFFFFFu, aborted(wc))) return false;
        if (__any_sync(0xFFFFFFFFu, ptx::globaltimer_ns() - t0 > limit)) {
            raise_abort(wc);
            return false;
        }
    }
}

template <int kCtas>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, WaitCtl *wc)
{
    return probe<kCtas == 2>(bar, parity) || warp_wait_slow<kCtas == 2>(bar, parity, wc);
}

// One raw stage: K block kb of 128 rows from rr and of this CTA's columns from
// cc (by one thread).
__device__ __forceinline__ void load_stage(const CUtensorMap *tmap_r, const CUtensorMap *tmap_c, const Params &p,
                                           uint32_t raw, Ctrl *ctrl, uint32_t stage, int kb, int32_t rr, int32_t cc)
{
    const uint32_t full = ptx::smem_addr(&ctrl->raw_full[stage]);
    const uint32_t dst = raw + stage * static_cast<uint32_t>(p.raw_bytes);
    ptx::mbar_arrive_expect_tx(full, static_cast<uint32_t>(p.raw_bytes));
    // the innermost coordinate is a multiple of 128 bytes
    ptx::tma_load_2d(dst, tmap_r, full, kb * kRowBytes, rr);
    ptx::tma_load_2d(dst + kRawRowsBytes, tmap_c, full, kb * kRowBytes, cc);
}

// The first loads of the CTA, into the empty ring, by the thread that has set
// the ring's barriers up: they are in flight while the rest of the CTA (and
// its pair) starts, ~0.5 us.  Two of them, because the start waits for this
// thread and each takes it ~200 clocks.  Returns their number.
template <int kCtas>
__device__ __forceinline__ int prefill(const CUtensorMap *tmap_r, const CUtensorMap *tmap_c, const Params &p,
                                       uint32_t raw, Ctrl *ctrl, uint32_t rank)
{
    const Sched sc = schedule<kCtas>(p);
    int64_t r0, c0;
    tile_origin(p, sc.t0, kRows * kCtas, r0, c0);
    const int n = min(2, sc.kb1 - sc.kb0);
    for (int i = 0; i < n; ++i)
        load_stage(tmap_r, tmap_c, p, raw, ctrl, i, sc.kb0 + i, static_cast<int32_t>(r0 + rank * kRows),
                   static_cast<int32_t>(c0 + rank * (p.bn / kCtas)));
    return n;
}

// The rest of the loads, after the `done` of prefill.
template <int kCtas>
__device__ __forceinline__ void run_producer(const CUtensorMap *tmap_r, const CUtensorMap *tmap_c, const Params &p,
                                             uint32_t raw, Ctrl *ctrl, uint32_t rank, int done, WaitCtl *wc)
{
    const Sched sc = schedule<kCtas>(p);
    const uint32_t tiles = p.tiles_r * p.tiles_c;
    const int cols = p.bn / kCtas;  // columns this CTA converts
    uint32_t stage = static_cast<uint32_t>(done), phase = 0;
    if (stage == static_cast<uint32_t>(p.raw_stages)) {
        stage = 0;
        phase = 1;
    }
    bool ok = true;
    for (uint32_t t = sc.t0; ok && t < tiles; t += sc.dt) {
        int64_t r0, c0;
        tile_origin(p, t, kRows * kCtas, r0, c0);
        const int32_t rr = static_cast<int32_t>(r0 + rank * kRows), cc = static_cast<int32_t>(c0 + rank * cols);
        for (int kb = t == sc.t0 ? sc.kb0 + done : sc.kb0; kb < sc.kb1; ++kb) {
            ok = warp_wait<1>(ptx::smem_addr(&ctrl->raw_empty[stage]), phase ^ 1u, wc);
            if (!ok) break;
            if (elect_one()) load_stage(tmap_r, tmap_c, p, raw, ctrl, stage, kb, rr, cc);
            __syncwarp();
            if (++stage == static_cast<uint32_t>(p.raw_stages)) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
    // Do not leave while TMA may still be writing into this CTA's memory (after an
    // abort, whoever raised it; else these loads are waited for anyway): stages
    // before `stage` were last filled in this phase, the others (if at all: a
    // barrier's phase 1 counts as over before its first) in the one before.
    if (elect_one())
        for (uint32_t s = 0; s < static_cast<uint32_t>(p.raw_stages); ++s)
            drain_wait(ptx::smem_addr(&ctrl->raw_full[s]), s < stage ? phase : phase ^ 1u);
    __syncwarp();
}

// A converter warp's arrival on a barrier of the pair's leader.
template <int kCtas>
__device__ __forceinline__ void arrive_leader(uint32_t bar)
{
    if constexpr (kCtas == 2)
        arrive_remote(ptx::mapa(bar, 0));
    else
        ptx::mbar_arrive(bar);
}

// Tiles of this CTA (at least one: the grid has no more CTAs than tiles).
__device__ __forceinline__ uint32_t my_tiles(const Params &p, const Sched &sc)
{
    return (p.tiles_r * p.tiles_c - sc.t0 + sc.dt - 1) / sc.dt;
}

// A converter group's walk over the halves of the CTA's raw stages, in the order
// the producer fills them, and the converted stages they go to: group g takes
// halves g, g + 3, ... (two a stage).
struct HalfIter {
    int32_t left;               // stages to go, this one included
    uint32_t half;
    uint32_t stage, phase;      // raw ring
    uint32_t conv, conv_phase;  // converted ring
    uint32_t stages, conv_stages;

    __device__ __forceinline__ HalfIter(const Params &p, const Sched &sc, uint32_t group)
    {
        left = static_cast<int32_t>(my_tiles(p, sc)) * (sc.kb1 - sc.kb0);
        stages = static_cast<uint32_t>(p.raw_stages);
        conv_stages = static_cast<uint32_t>(p.conv_stages);
        stage = phase = conv = conv_phase = 0;
        half = group & 1u;
        advance(group >> 1);
    }
    __device__ __forceinline__ void advance(uint32_t n)  // n <= 2 <= conv_stages, stages
    {
        left -= static_cast<int32_t>(n);
        stage += n;
        if (stage >= stages) {
            stage -= stages;
            phase ^= 1u;
        }
        conv += n;
        if (conv >= conv_stages) {
            conv -= conv_stages;
            conv_phase ^= 1u;
        }
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void next()
    {
        advance(1u + half);
        half ^= 1u;
    }
};
static_assert(kConvGroups == 3, "HalfIter::next steps by three halves");

// Row converters: thread = row.  A raw row is 128 bytes, its 16-byte chunk j
// stored at chunk position j ^ (row mod 8), so that the eight rows of a
// wavefront read distinct banks.
template <int kCtas>
__device__ __forceinline__ void run_row_converter(const Params &p, uint32_t raw, Ctrl *ctrl, uint32_t tmem_base,
                                                  int warp, uint32_t group, int lane, WaitCtl *wc)
{
    const uint32_t quarter = static_cast<uint32_t>(warp & 3);
    const uint32_t row = quarter * 32 + lane;
    const uint32_t lanes = tmem_base + ((quarter * 32u) << 16) + static_cast<uint32_t>(p.conv_col);
    for (HalfIter it(p, schedule<kCtas>(p), group); it.more(); it.next()) {
        if (!warp_wait<1>(ptx::smem_addr(&ctrl->raw_full[it.stage]), it.phase, wc)) return;
        const uint32_t src = raw + it.stage * static_cast<uint32_t>(p.raw_bytes) + row * kRowBytes;
        uint4 c[4];
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) c[j] = ld_shared_v4(src + (((it.half * 4 + j) ^ (row & 7u)) << 4));
        uint32_t w[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) widen16(c[j], w + j * 8);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctrl->raw_empty[it.stage]));
        if (!warp_wait<kCtas>(ptx::smem_addr(&ctrl->conv_empty[2 * it.conv + it.half]), it.conv_phase ^ 1u, wc)) return;
        ptx::tc_fence_after();
        ptx::tmem_st_32x32b_x32(lanes + (2 * it.conv + it.half) * kConvCols, w);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader<kCtas>(ptx::smem_addr(&ctrl->conv_full[it.conv]));
    }
}

// Column converters: a half is the CTA's cols = bn / kCtas columns x 64 K
// values, cols x 4 chunks of 16 bytes, kTasks of them a thread (consecutive
// threads take consecutive columns of one chunk position; where cols is no
// multiple of 32, some chunks are widened twice, to the same words).  A
// widened column is a 128-byte K-major row under the 128-byte swizzle.
template <int kCtas, int kTasks>
__device__ __forceinline__ void run_col_converter(const Params &p, uint32_t raw, uint32_t conv, Ctrl *ctrl, int tid,
                                                  uint32_t group, int lane, WaitCtl *wc)
{
    const int cols = p.bn / kCtas;
    const uint32_t half_bytes = static_cast<uint32_t>(cols) * 128u;
    // offsets of this thread's chunks in a raw stage's first half (the second
    // half's differ in bit 6) and in a converted half (a chunk widens to two
    // 16-byte words: there, and there ^ 16)
    uint32_t src_off[kTasks], dst_off[kTasks];
#pragma unroll
    for (int i = 0; i < kTasks; ++i) {
        const int task = i * 128 + tid;
        const uint32_t col = static_cast<uint32_t>(task % cols), j = static_cast<uint32_t>(task / cols) & 3u;
        src_off[i] = kRawRowsBytes + col * kRowBytes + ((j ^ (col & 7u)) << 4);
        dst_off[i] = col * 128u + (((2 * j) ^ (col & 7u)) << 4);
    }
    for (HalfIter it(p, schedule<kCtas>(p), group); it.more(); it.next()) {
        if (!warp_wait<1>(ptx::smem_addr(&ctrl->raw_full[it.stage]), it.phase, wc)) return;
        const uint32_t src = raw + it.stage * static_cast<uint32_t>(p.raw_bytes);
        uint4 c[kTasks];
        uint32_t w[kTasks][8];
#pragma unroll
        for (int i = 0; i < kTasks; ++i)
            if (DGEMM_CHECK((src_off[i] | 64u) + 16 <= static_cast<uint32_t>(p.raw_bytes)))
                c[i] = ld_shared_v4(src + (src_off[i] ^ (it.half << 6)));
#pragma unroll
        for (int i = 0; i < kTasks; ++i) widen16(c[i], w[i]);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctrl->raw_empty[it.stage]));
        if (!warp_wait<kCtas>(ptx::smem_addr(&ctrl->conv_empty[2 * it.conv + it.half]), it.conv_phase ^ 1u, wc)) return;
        const uint32_t dst = conv + (2 * it.conv + it.half) * half_bytes;
#pragma unroll
        for (int i = 0; i < kTasks; ++i) {
            if (DGEMM_CHECK((dst_off[i] | 16u) + 16 <= half_bytes)) {
                ptx::st_shared_v4(dst + dst_off[i], make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]));
                ptx::st_shared_v4(dst + (dst_off[i] ^ 16u), make_uint4(w[i][4], w[i][5], w[i][6], w[i][7]));
            }
        }
        ptx::fence_proxy_async_smem();  // the MMAs read through the async proxy
        __syncwarp();
        if (lane == 0) arrive_leader<kCtas>(ptx::smem_addr(&ctrl->conv_full[it.conv]));
    }
}

constexpr uint32_t kEpiBarrier = 1;  // named barrier of the epilogue warps

template <int kCtas>
__device__ __forceinline__ void run_mma(const Params &p, uint32_t conv, Ctrl *ctrl, uint32_t tmem_base, WaitCtl *wc)
{
    const Sched sc = schedule<kCtas>(p);
    const uint32_t tiles = p.tiles_r * p.tiles_c;
    const uint32_t half_bytes = static_cast<uint32_t>(p.bn / kCtas) * 128u;
    // D f32, A and B f16 and K-major, N = bn, M = 128 rows a CTA
    const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(p.bn >> 3) << 17) |
                           (static_cast<uint32_t>(kRows * kCtas >> 4) << 24);
    // the descriptor of the first MMA's columns; a half on is half_bytes / 16,
    // an MMA's K step 2, in its address field
    const uint64_t b_desc = ptx::smem_desc(conv, 16, 1024, ptx::kSw128);
    tmem_base = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);  // a uniform value for the compiler
    const uint32_t a_base = tmem_base + static_cast<uint32_t>(p.conv_col);
    uint32_t cs = 0, cphase = 0, acc = 0, acc_phase = 0;
    // test hook: wait on a barrier nothing arrives at, so the wait runs out
    bool ok = !p.inject_stall || warp_wait<1>(ptx::smem_addr(&ctrl->never), 0, wc);
    for (uint32_t t = sc.t0; ok && t < tiles; t += sc.dt) {
        ok = warp_wait<kCtas>(ptx::smem_addr(&ctrl->acc_empty[acc]), acc_phase ^ 1u, wc);
        if (!ok) break;
        const uint32_t d = tmem_base + acc * static_cast<uint32_t>(p.bn);
        for (int kb = sc.kb0; kb < sc.kb1; ++kb) {
            ok = warp_wait<kCtas>(ptx::smem_addr(&ctrl->conv_full[cs]), cphase, wc);
            if (!ok) break;
            ptx::tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h) {
                    const uint32_t a = a_base + (2 * cs + h) * kConvCols;
                    const uint64_t b = b_desc + (2 * cs + h) * (half_bytes >> 4);
#pragma unroll
                    for (int k = 0; k < kHalfK / 16; ++k)
                        umma_a_tmem<kCtas>(d, a + k * 8, b + k * 2, idesc, kb == sc.kb0 && h == 0 && k == 0 ? 0u : 1u);
                    commit_all<kCtas>(ptx::smem_addr(&ctrl->conv_empty[2 * cs + h]));
                }
            }
            __syncwarp();
            if (++cs == static_cast<uint32_t>(p.conv_stages)) {
                cs = 0;
                cphase ^= 1u;
            }
        }
        if (!ok) break;
        if (elect_one()) commit_all<kCtas>(ptx::smem_addr(&ctrl->acc_full[acc]));
        __syncwarp();
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
    }
    __syncwarp();
    // Whatever the epilogue's waits came to, every MMA issued has finished before
    // TMEM is released (the elected thread is the same one each time).
    if (elect_one()) {
        if constexpr (kCtas == 2)
            ptx::umma_commit_pair_multicast(ptx::smem_addr(&ctrl->mma_done), 0x1);
        else
            ptx::umma_commit(ptx::smem_addr(&ctrl->mma_done));
        drain_wait(ptx::smem_addr(&ctrl->mma_done), 0);
    }
    __syncwarp();
}

// ---- epilogues

template <typename T>
__device__ __forceinline__ uint32_t pack_bits(T a, T b)
{
    static_assert(sizeof(T) == 2, "two 16-bit values");
    return static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(&a)) |
           static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(&b)) << 16;
}

// Sixteen accumulator columns from `col` of this lane's row, times the row's
// scale sa and the columns' (in shared memory at `scale`), plus their biases.
// The scales' loads are in flight beside the accumulator's.
__device__ __forceinline__ void load_scaled(const Params &p, uint32_t taddr, uint32_t scale, uint32_t bias, int col,
                                            float sa, float (&v)[16])
{
    uint32_t r[16];
    float4 s[4];
    tmem_ld_32x32b_x16(taddr + col, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = ptx::ld_shared_v4f(scale + static_cast<uint32_t>(col + 4 * i) * 4u);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[4 * i] = __uint_as_float(r[4 * i]) * sa * s[i].x;
        v[4 * i + 1] = __uint_as_float(r[4 * i + 1]) * sa * s[i].y;
        v[4 * i + 2] = __uint_as_float(r[4 * i + 2]) * sa * s[i].z;
        v[4 * i + 3] = __uint_as_float(r[4 * i + 3]) * sa * s[i].w;
    }
    if (!p.c.bias) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 o = ptx::ld_shared_v4f(bias + static_cast<uint32_t>(col + 4 * i) * 4u);
        v[4 * i] += o.x;
        v[4 * i + 1] += o.y;
        v[4 * i + 2] += o.z;
        v[4 * i + 3] += o.w;
    }
}

// v += beta * old for sixteen columns of a row of C (`left` of them in C), whose
// rows start on 16-byte boundaries.
template <typename T>
__device__ __forceinline__ void add_old(const T *c, int64_t left, float beta, float (&v)[16])
{
    if (left >= 16 && DGEMM_CHECK((reinterpret_cast<uintptr_t>(c) & 15u) == 0)) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) {
            constexpr int kPer = 16 / sizeof(T);
            const uint4 w = reinterpret_cast<const uint4 *>(c)[i];
            const T *e = reinterpret_cast<const T *>(&w);
#pragma unroll
            for (int j = 0; j < kPer; ++j) v[i * kPer + j] = fmaf(beta, i8_to_f32(e[j]), v[i * kPer + j]);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (e < left) v[e] = fmaf(beta, i8_to_f32(c[e]), v[e]);
}

// A warp's share of a tile's columns: every step-th piece from `first`, staged
// in `boxes` boxes at `box`.
struct Share {
    int first, step;
    uint32_t box;
    int boxes;
};

// Rows = tokens: the warp's 32 rows x its share of the bn columns from (row0, c0), by boxes of
// 128 bytes of columns staged in shared memory (128-byte swizzle) and stored
// by TMA, or, where TMA cannot describe C, by rows of 32 columns.
template <typename T>
__device__ __forceinline__ void drain_tokens(const Params &p, const CUtensorMap *tmap_o, const Ctrl *ctrl,
                                             uint32_t taddr, int64_t row0, int64_t c0, float sa, const Share &sh,
                                             int lane, uint32_t &nbox)
{
    constexpr int kCols = 128 / sizeof(T);  // columns of a box
    const int64_t row = row0 + lane;
    const float beta = p.c.beta;
    const uint32_t scale = ptx::smem_addr(ctrl->scale), bias = ptx::smem_addr(ctrl->bias);
    T *crow = static_cast<T *>(p.c.C) + row * p.c.ldc;
    if (!DGEMM_CHECK((taddr & 0xFFFFu) + static_cast<uint32_t>(p.bn) <= static_cast<uint32_t>(p.conv_col))) return;
    if (p.tma_store) {
#pragma unroll 1
        for (int b = sh.first; b < p.bn / kCols; b += sh.step) {
            const int64_t col0 = c0 + b * kCols;
            const uint32_t buf = sh.box + (sh.boxes == 2 ? (nbox & 1u) * kBoxBytes : 0u);
            if (row0 >= p.rows || col0 >= p.cols) break;  // warp-uniform: nothing of C here
            if (lane == 0) {  // this box's last store has read it
                if (sh.boxes == 2)
                    ptx::bulk_wait_read<1>();
                else
                    ptx::bulk_wait_read<0>();
            }
            __syncwarp();
            const uint32_t dst = buf + static_cast<uint32_t>(lane) * 128u;
#pragma unroll 1
            for (int part = 0; part < kCols / 16; ++part) {  // (rolled: its code is fetched cold)
                float v[16];
                load_scaled(p, taddr, scale, bias, b * kCols + part * 16, sa, v);
                if (beta != 0.f && row < p.rows) add_old(crow + col0 + part * 16, p.cols - col0 - part * 16, beta, v);
                constexpr int kPer = 16 / sizeof(T);  // values of a 16-byte word
#pragma unroll
                for (int j = 0; j < 16; j += kPer) {
                    uint4 q;
                    if constexpr (sizeof(T) == 2)
                        q = make_uint4(pack_bits(i8_from_f32<T>(v[j]), i8_from_f32<T>(v[j + 1])),
                                       pack_bits(i8_from_f32<T>(v[j + 2]), i8_from_f32<T>(v[j + 3])),
                                       pack_bits(i8_from_f32<T>(v[j + 4]), i8_from_f32<T>(v[j + 5])),
                                       pack_bits(i8_from_f32<T>(v[j + 6]), i8_from_f32<T>(v[j + 7])));
                    else
                        q = make_uint4(__float_as_uint(v[j]), __float_as_uint(v[j + 1]), __float_as_uint(v[j + 2]),
                                       __float_as_uint(v[j + 3]));
                    const uint32_t word = static_cast<uint32_t>((part * 16 + j) / kPer);
                    ptx::st_shared_v4(dst + ((word ^ (static_cast<uint32_t>(lane) & 7u)) << 4), q);
                }
            }
            ptx::fence_proxy_async_smem();  // the TMA store reads through the async proxy
            __syncwarp();
            if (lane == 0 && DGEMM_CHECK(row0 >= 0 && col0 >= 0 && row0 < p.rows && col0 < p.cols)) {
                ptx::tma_store_2d(tmap_o, buf, static_cast<int32_t>(col0), static_cast<int32_t>(row0));
                ptx::bulk_commit();
            }
            ++nbox;
        }
        return;
    }
    // value e of row t sits at word e ^ t of the staged row, so both the
    // row-wise writes and the column-wise reads hit 32 different banks
#pragma unroll 1
    for (int b = sh.first; b < p.bn / 32; b += sh.step) {
        const uint32_t box = sh.box;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            float v[16];
            __syncwarp();
            load_scaled(p, taddr, scale, bias, b * 32 + part * 16, sa, v);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                ptx::st_shared_f32(box + (static_cast<uint32_t>(lane) * 32u + (static_cast<uint32_t>(part * 16 + i) ^ lane)) * 4u,
                                   v[i]);
        }
        __syncwarp();
        const int64_t col = c0 + b * 32 + lane;
#pragma unroll 4
        for (int i = 0; i < 32; ++i) {
            if (row0 + i >= p.rows) break;  // warp-uniform
            float v = ptx::ld_shared_f32(box + (static_cast<uint32_t>(i) * 32u + (lane ^ static_cast<uint32_t>(i))) * 4u);
            if (col < p.cols && DGEMM_CHECK(row0 + i >= 0 && col >= 0)) {
                T *dst = static_cast<T *>(p.c.C) + (row0 + i) * p.c.ldc + col;
                if (beta != 0.f) v = fmaf(beta, i8_to_f32(*dst), v);
                *dst = i8_from_f32<T>(v);
            }
        }
        __syncwarp();  // the buffer is reused by the next chunk
    }
}

// Rows = channels: v[j] is the sum for channel n (this lane's) and token
// m0 + j, whose scale is at sa[j]; for each token the warp's lanes store
// consecutive channels.
template <typename T, int kCount>
__device__ __forceinline__ void store_channels(const Params &p, int64_t n, int64_t m0, uint32_t sa, float sb,
                                               float bias, const float (&v)[kCount])
{
    const int64_t left = p.cols - m0;
    if (n >= p.rows || !DGEMM_CHECK(m0 >= 0 && n >= 0)) return;
    T *dst = static_cast<T *>(p.c.C) + m0 * p.c.ldc + n;
    float x[kCount];
#pragma unroll
    for (int j = 0; j < kCount; j += 4) {
        const float4 s = ptx::ld_shared_v4f(sa + 4u * static_cast<uint32_t>(j));
        x[j] = fmaf(v[j] * s.x, sb, bias);
        x[j + 1] = fmaf(v[j + 1] * s.y, sb, bias);
        x[j + 2] = fmaf(v[j + 2] * s.z, sb, bias);
        x[j + 3] = fmaf(v[j + 3] * s.w, sb, bias);
    }
    if (p.c.beta != 0.f) {
#pragma unroll
        for (int j = 0; j < kCount; ++j)
            if (j < left) x[j] = fmaf(p.c.beta, i8_to_f32(dst[j * p.c.ldc]), x[j]);
    }
#pragma unroll
    for (int j = 0; j < kCount; ++j)
        if (j < left) dst[j * p.c.ldc] = i8_from_f32<T>(x[j]);
}

// The scales (and biases) of the tile's columns, by the 128 epilogue threads;
// whole warps leave together at the named barrier.
template <bool kSwap>
__device__ __forceinline__ void load_column_values(const Params &p, Ctrl *ctrl, int64_t c0, int tid)
{
    for (int c = tid; c < p.bn; c += 32 * kEpiWarps) {
        const bool in = c0 + c < p.cols && c < kMaxBn;
        ctrl->scale[c] = in ? load_f32((kSwap ? p.c.scale_a : p.c.scale_b) + c0 + c) : 0.f;
        if constexpr (!kSwap) ctrl->bias[c] = in && p.c.bias ? load_f32(p.c.bias + c0 + c) : 0.f;
    }
    __syncwarp();
    named_barrier(kEpiBarrier, 32 * kEpiWarps);
}

// One tile's accumulator at taddr (this warp's TMEM lanes) to C.
template <bool kSwap, typename T>
__device__ __forceinline__ void drain(const Params &p, const CUtensorMap *tmap_o, const Ctrl *ctrl, uint32_t taddr,
                                      int64_t row0, int64_t c0, float rs, float rb, const Share &sh, int lane,
                                      uint32_t &nbox)
{
    if constexpr (!kSwap) {
        drain_tokens<T>(p, tmap_o, ctrl, taddr, row0, c0, rs, sh, lane, nbox);
    } else {
#pragma unroll 1
        for (int b = 16 * sh.first; b < p.bn; b += 16 * sh.step) {
            uint32_t r[16];
            __syncwarp();
            tmem_ld_32x32b_x16(taddr + b, r);
            ptx::tmem_ld_wait();
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
            store_channels<T>(p, row0 + lane, c0 + b, ptx::smem_addr(ctrl->scale + b), rs, rb, v);
        }
    }
}

// This lane's row of the accumulator: a token's scale, or a channel's scale
// and bias.
template <bool kSwap>
__device__ __forceinline__ void load_row_values(const Params &p, int64_t row, float &rs, float &rb)
{
    rs = row < p.rows ? load_f32((kSwap ? p.c.scale_b : p.c.scale_a) + row) : 0.f;
    rb = kSwap && p.c.bias && row < p.rows ? load_f32(p.c.bias + row) : 0.f;
}

// The CTA's tiles but the last, while the MMAs of the next one run; then the
// column values of the last and the wait for its accumulator.
template <int kCtas, bool kSwap, typename T>
__device__ __forceinline__ void run_epilogue(const Params &p, const CUtensorMap *tmap_o, Ctrl *ctrl,
                                             uint32_t tmem_base, uint32_t box, uint32_t rank, int warp, int lane,
                                             WaitCtl *wc)
{
    const Sched sc = schedule<kCtas>(p);
    const uint32_t tiles = p.tiles_r * p.tiles_c;
    const uint32_t quarter = static_cast<uint32_t>(warp & 3);  // the TMEM lanes this warp may read
    const Share sh{0, 1, box + quarter * 2 * kBoxBytes, 2};
    uint32_t acc = 0, acc_phase = 0, nbox = 0;
    for (uint32_t t = sc.t0; t < tiles; t += sc.dt) {
        int64_t r0, c0;
        tile_origin(p, t, kRows * kCtas, r0, c0);
        const int64_t row0 = r0 + rank * kRows + quarter * 32;
        __syncwarp();
        named_barrier(kEpiBarrier, 32 * kEpiWarps);  // the last tile's values have been read
        load_column_values<kSwap>(p, ctrl, c0, quarter * 32 + lane);
        float rs, rb;  // loaded while the MMAs run
        load_row_values<kSwap>(p, row0 + lane, rs, rb);
        bool ok = warp_wait<kCtas>(ptx::smem_addr(&ctrl->acc_full[acc]), acc_phase, wc);
        if (t + sc.dt >= tiles) break;  // drain_last's, whether it came or not
        // every epilogue warp leaves together, so none waits for another at
        // the named barrier
        __syncwarp();
        ok = !ptx::bar_red_or(kEpiBarrier, 32 * kEpiWarps, !ok);
        if (!ok) break;
        ptx::tc_fence_after();
        drain<kSwap, T>(p, tmap_o, ctrl, tmem_base + ((quarter * 32u) << 16) + acc * static_cast<uint32_t>(p.bn), row0, c0,
                        rs, rb, sh, lane, nbox);
        ptx::tc_fence_before();
        __syncwarp();
        // (the accumulator's next tile; an arrival that nothing waits for could
        // reach a CTA that has left)
        if (lane == 0 && t + 2 * sc.dt < tiles) arrive_leader<kCtas>(ptx::smem_addr(&ctrl->acc_empty[acc]));
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
    }
}

// The last (with split-K: the only) tile of the CTA as a draining warp sees it.
struct LastTile {
    int64_t row0, c0;   // first row of the warp's 32, first column of the tile
    float rs, rb;       // this lane's row values
    uint32_t acc;       // accumulator
};

template <int kCtas, bool kSwap>
__device__ __forceinline__ LastTile last_tile(const Params &p, uint32_t rank, int warp, int lane)
{
    const Sched sc = schedule<kCtas>(p);
    const uint32_t n = my_tiles(p, sc);
    LastTile l;
    int64_t r0;
    tile_origin(p, sc.t0 + (n - 1) * sc.dt, kRows * kCtas, r0, l.c0);
    l.row0 = r0 + rank * kRows + static_cast<uint32_t>(warp & 3) * 32;
    l.acc = (n - 1) & 1u;
    load_row_values<kSwap>(p, l.row0 + lane, l.rs, l.rb);
    return l;
}

// The last tile of the CTA, after a barrier of all its warps: no MMAs are left
// to hide the drain behind, so 16 warps share it (the epilogue's and the row
// converters', group g of four taking every fourth piece of columns).  The
// converters' warps stage in the raw ring, which is idle now.
template <int kCtas, bool kSwap, typename T>
__device__ __forceinline__ void drain_last(const Params &p, const CUtensorMap *tmap_o, const Ctrl *ctrl,
                                           const LastTile &l, uint32_t tmem_base, uint32_t box, uint32_t raw, int warp,
                                           int lane, WaitCtl *wc)
{
    if (__any_sync(0xFFFFFFFFu, aborted(wc))) {
        if (lane == 0) ptx::bulk_wait<0>();  // earlier tiles' stores
        if (kCtas == 2) fence_cluster();     // and arrivals (see the call)
        return;
    }
    ptx::tc_fence_after();
    const int group = (warp - 4) >> 2;
    const uint32_t quarter = static_cast<uint32_t>(warp & 3);
    const Share sh{group, 1 + kConvGroups,
                   group == 0 ? box + quarter * 2 * kBoxBytes : raw + ((group - 1) * 4 + quarter) * kBoxBytes, 1};
    uint32_t nbox = 0;
    drain<kSwap, T>(p, tmap_o, ctrl, tmem_base + ((quarter * 32u) << 16) + l.acc * static_cast<uint32_t>(p.bn), l.row0,
                    l.c0, l.rs, l.rb, sh, lane, nbox);
    if (lane == 0) ptx::bulk_wait<0>();  // stores done before the CTA leaves
}

// ---- split-K (kSwap, single CTAs): the S CTAs of a cluster have each summed
// a K range of one tile.  Groups of 8 columns are owned round-robin by the
// ranks; each CTA pushes the groups it does not own into the owner's idle raw
// ring, [sender slot][owned group][column quad][row] in 16-byte units, and
// the owner adds the partials in rank order, so the sum does not depend on
// timing.

__device__ __forceinline__ uint32_t recv_offset(uint32_t groups, uint32_t slot, uint32_t idx, uint32_t S, int q,
                                                int row)
{
    const uint32_t owned = (groups + S - 1) / S;
    return (((slot * owned + idx) * 2u + static_cast<uint32_t>(q)) * kRows + static_cast<uint32_t>(row)) * 16u;
}

__device__ __forceinline__ void splitk_push(const Params &p, uint32_t tmem_base, uint32_t raw, int warp, int lane,
                                            WaitCtl *wc)
{
    if (__any_sync(0xFFFFFFFFu, aborted(wc))) return;
    ptx::tc_fence_after();
    const uint32_t quarter = static_cast<uint32_t>(warp & 3);
    const uint32_t S = static_cast<uint32_t>(p.splitk), rank = ptx::cluster_ctarank();
    const uint32_t groups = static_cast<uint32_t>(p.bn) / 8;
    const int row = static_cast<int>(quarter * 32 + lane);
#pragma unroll 1
    for (uint32_t g = static_cast<uint32_t>(warp - 4) >> 2; g < groups; g += 1 + kConvGroups) {  // shared as in drain_last
        const uint32_t owner = g % S;
        if (owner == rank) continue;
        uint32_t r[8];
        __syncwarp();
        tmem_ld_32x32b_x8(tmem_base + ((quarter * 32u) << 16) + g * 8, r);
        ptx::tmem_ld_wait();
        const uint32_t slot = rank < owner ? rank : rank - 1;
        if (!DGEMM_CHECK(recv_offset(groups, slot, g / S, S, 1, row) + 16 <= static_cast<uint32_t>(p.raw_stages * p.raw_bytes))) continue;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            ptx::st_shared_cluster_v4(ptx::mapa(raw + recv_offset(groups, slot, g / S, S, q, row), owner),
                                      make_float4(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]),
                                                  __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3])));
    }
}

template <typename T>
__device__ __forceinline__ void splitk_reduce(const Params &p, const Ctrl *ctrl, const LastTile &l, uint32_t tmem_base,
                                              uint32_t raw, int warp, int lane, WaitCtl *wc)
{
    if (__any_sync(0xFFFFFFFFu, aborted(wc))) return;
    ptx::tc_fence_after();
    const uint32_t quarter = static_cast<uint32_t>(warp & 3);
    const uint32_t S = static_cast<uint32_t>(p.splitk), rank = ptx::cluster_ctarank();
    const uint32_t groups = static_cast<uint32_t>(p.bn) / 8;
    const int row = static_cast<int>(quarter * 32 + lane);
#pragma unroll 1
    for (uint32_t g = rank + S * (static_cast<uint32_t>(warp - 4) >> 2); g < groups; g += S * (1 + kConvGroups)) {
        uint32_t own[8];
        __syncwarp();
        tmem_ld_32x32b_x8(tmem_base + ((quarter * 32u) << 16) + g * 8, own);
        ptx::tmem_ld_wait();
        float v[8] = {};
        for (uint32_t s = 0; s < S; ++s) {
            if (s == rank) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += __uint_as_float(own[j]);
                continue;
            }
            const uint32_t slot = s < rank ? s : s - 1;
            if (!DGEMM_CHECK(recv_offset(groups, slot, g / S, S, 1, row) + 16 <= static_cast<uint32_t>(p.raw_stages * p.raw_bytes))) continue;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float4 f = ptx::ld_shared_v4f(raw + recv_offset(groups, slot, g / S, S, q, row));
                v[4 * q] += f.x;
                v[4 * q + 1] += f.y;
                v[4 * q + 2] += f.z;
                v[4 * q + 3] += f.w;
            }
        }
        store_channels<T>(p, l.row0 + lane, l.c0 + g * 8, ptx::smem_addr(ctrl->scale + g * 8), l.rs, l.rb, v);
    }
}

template <int kCtas, bool kSwap, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    i8_umma_kernel(const __grid_constant__ CUtensorMap tmap_r, const __grid_constant__ CUtensorMap tmap_c,
                   const __grid_constant__ CUtensorMap tmap_o, const Params p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    // converted columns | epilogue boxes (kSwap: none) | raw ring | control
    const uint32_t conv = ptx::smem_addr(smem);
    const uint32_t box = conv + static_cast<uint32_t>(p.conv_stages * 2 * (p.bn / kCtas) * 128);
    const uint32_t raw = box + (kSwap ? 0 : kEpiWarps * 2 * kBoxBytes);
    Ctrl *ctrl = reinterpret_cast<Ctrl *>(smem + (raw - conv) + p.raw_stages * p.raw_bytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = kCtas == 2 ? (ptx::cluster_ctarank() & 1u) : 0u;
    const bool leader = rank == 0;
    int loaded = 0;  // raw stages already under way (warp 0)

    if (warp == 0) {
        if (elect_one()) {
            for (int s = 0; s < kMaxRaw; ++s) {
                ptx::mbar_init(ptx::smem_addr(&ctrl->raw_full[s]), 1);
                ptx::mbar_init(ptx::smem_addr(&ctrl->raw_empty[s]), 16);
            }
            ptx::fence_mbarrier_init();
            chain_wait();  // (everything below reads or writes the call's operands)
            loaded = prefill<kCtas>(&tmap_r, &tmap_c, p, raw, ctrl, rank);
        }
        loaded = __reduce_max_sync(0xFFFFFFFFu, loaded);
    } else if (warp == 1) {
        if constexpr (kCtas == 2) {
            ptx::tmem_alloc_pair(ptx::smem_addr(&ctrl->tmem_base), kTmemCols);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(ptx::smem_addr(&ctrl->tmem_base), kTmemCols);
            ptx::tmem_relinquish();
        }
    } else if (warp == 2 && elect_one()) {
        for (int s = 0; s < kMaxConv; ++s) ptx::mbar_init(ptx::smem_addr(&ctrl->conv_full[s]), 16 * kCtas);
        for (int s = 0; s < 2 * kMaxConv; ++s) ptx::mbar_init(ptx::smem_addr(&ctrl->conv_empty[s]), 1);
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(ptx::smem_addr(&ctrl->acc_full[a]), 1);
            ptx::mbar_init(ptx::smem_addr(&ctrl->acc_empty[a]), kEpiWarps * kCtas);
        }
        ptx::mbar_init(ptx::smem_addr(&ctrl->mma_done), 1);
        ptx::mbar_init(ptx::smem_addr(&ctrl->never), 1);
        ctrl->wait.abort = 0;
        ctrl->wait.limit_ns = p.wait_limit_ns;
        ptx::fence_mbarrier_init();
        if (p.tma_store) ptx::prefetch_tmap(&tmap_o);
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    // both CTAs' barriers exist (fence_mbarrier_init above) before any
    // cross-CTA signal
    if constexpr (kCtas == 2) cluster_meet();
    ptx::tc_fence_after();
    chain_wait();
    chain_next();
    const uint32_t tmem_base = ctrl->tmem_base;
    WaitCtl *wc = &ctrl->wait;

    if (warp == 0) {
        run_producer<kCtas>(&tmap_r, &tmap_c, p, raw, ctrl, rank, loaded, wc);
    } else if (warp == 1) {
        if (leader) run_mma<kCtas>(p, conv, ctrl, tmem_base, wc);
    } else if (warp >= 8 + 4 * kConvGroups) {
        const int tid = threadIdx.x & 127, group = (warp - 8 - 4 * kConvGroups) >> 2;
        switch ((p.bn / kCtas + 31) / 32) {  // chunks a thread takes; uniform
        case 1: run_col_converter<kCtas, 1>(p, raw, conv, ctrl, tid, group, lane, wc); break;
        case 2: run_col_converter<kCtas, 2>(p, raw, conv, ctrl, tid, group, lane, wc); break;
        case 3: run_col_converter<kCtas, 3>(p, raw, conv, ctrl, tid, group, lane, wc); break;
        default: run_col_converter<kCtas, 4>(p, raw, conv, ctrl, tid, group, lane, wc);
        }
    } else if (warp >= 8) {
        run_row_converter<kCtas>(p, raw, ctrl, tmem_base, warp, (warp - 8) >> 2, lane, wc);
    } else if (warp >= 4) {
        if (kCtas == 1 && p.splitk > 1) {
            int64_t r0, c0;
            tile_origin(p, blockIdx.x / p.splitk, kRows, r0, c0);
            load_column_values<kSwap>(p, ctrl, c0, threadIdx.x & 127);
            wait_bounded(ptx::smem_addr(&ctrl->acc_full[0]), 0, wc);  // a time-out raises the abort flag
        } else
            run_epilogue<kCtas, kSwap, T>(p, &tmap_o, ctrl, tmem_base, box, rank, warp, lane, wc);
    }

    const bool drains = warp >= 4 && warp < 8 + 4 * kConvGroups;  // (warp-uniform)
    LastTile last{};
    if (drains) last = last_tile<kCtas, kSwap>(p, rank, warp, lane);  // its loads are in flight across the barrier
    __syncwarp();  // the barriers below are warp-aligned: reconverge the single-lane roles
    ptx::tc_fence_before();
    if (kCtas == 1 && kSwap && p.splitk > 1) {  // uniform over the cluster
        ptx::cluster_sync();  // every CTA's sums are complete: the raw rings are idle
        if (drains) splitk_push(p, tmem_base, raw, warp, lane, wc);
        __syncwarp();
        ptx::tc_fence_before();
        ptx::cluster_sync();  // every partial has landed in its owner
        if (drains) splitk_reduce<T>(p, ctrl, last, tmem_base, raw, warp, lane, wc);
    } else {
        __syncthreads();  // every role of this CTA is done
        // after an abort, arrivals on the leader's barriers that nothing has waited
        // for may be under way: they come before this CTA's part in the meeting below
        if (kCtas == 2 && !drains && __any_sync(0xFFFFFFFFu, aborted(wc))) fence_cluster();
        if (drains) drain_last<kCtas, kSwap, T>(p, &tmap_o, ctrl, last, tmem_base, box, raw, warp, lane, wc);
    }
    __syncwarp();
    ptx::tc_fence_before();
    if constexpr (kCtas == 2)
        cluster_meet();  // no CTA leaves while the other may still signal or read it
    else
        __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        if constexpr (kCtas == 2)
            ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
        else
            ptx::tmem_dealloc(tmem_base, kTmemCols);
    }
}

// ---- host side

// Dynamic shared memory of a launch, and its rings.  Converted stages first:
// between the release of one and its next MMAs lie ~1500 clocks of hand-offs,
// so more of them pay until TMEM or the raw ring runs short (it keeps at least
// three stages).
int set_rings(Params &p, int ctas, bool swap)
{
    const int conv_bytes = 2 * (p.bn / ctas) * 128;
    p.raw_bytes = kRawRowsBytes + p.bn / ctas * kRowBytes;
    const int space = kSmemLimit - (swap ? 0 : kEpiWarps * 2 * kBoxBytes) - 1024 - static_cast<int>(sizeof(Ctrl));
    p.conv_stages = std::min({kMaxConv, (kTmemCols - p.conv_col) / (2 * kConvCols), (space - 3 * p.raw_bytes) / conv_bytes});
    p.raw_stages = std::min(kMaxRaw, (space - p.conv_stages * conv_bytes) / p.raw_bytes);
    return kSmemLimit - space + p.conv_stages * conv_bytes + p.raw_stages * p.raw_bytes;
}

// CTAs (kCtas == 1) or clusters of `cluster` CTAs of the kernel that can be
// resident at once on the current device, cached; 0 if it cannot run.
template <int kCtas, bool kSwap, typename T>
int capacity(int cluster)
{
    constexpr int kMaxDevices = 64;
    static int cached[kMaxDevices][9];
    static std::once_flag once[kMaxDevices];
    int dev = 0;
    if (cluster < 1 || cluster > 8 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    std::call_once(once[dev], [dev] {
        auto kernel = i8_umma_kernel<kCtas, kSwap, T>;
        int sms = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) == cudaSuccess &&
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) {
            cached[dev][1] = sms;
            for (int s = 2; s <= (kCtas == 2 ? 2 : 8); ++s) {
                cudaLaunchConfig_t cfg = {};
                cudaLaunchAttribute attr[1];
                attr[0].id = cudaLaunchAttributeClusterDimension;
                attr[0].val.clusterDim.x = static_cast<unsigned>(s);
                attr[0].val.clusterDim.y = 1;
                attr[0].val.clusterDim.z = 1;
                cfg.gridDim = dim3(static_cast<unsigned>(sms - sms % s));
                cfg.blockDim = dim3(kThreads);
                cfg.dynamicSmemBytes = kSmemLimit;
                cfg.attrs = attr;
                cfg.numAttrs = 1;
                int n = 0;
                if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) n = 0;
                cached[dev][s] = n;
            }
        }
        cudaGetLastError();  // a failed query leaves no sticky error behind
    });
    return cached[dev][cluster];
}

template <int kCtas, bool kSwap, typename T>
bool launch(const I8Params &c, int bn, int splitk, cudaStream_t stream)
{
    Params p{};
    p.c = c;
    p.rows = kSwap ? c.N : c.M;
    p.cols = kSwap ? c.M : c.N;
    p.bn = bn;
    const int64_t tiles_r = (p.rows + kRows * kCtas - 1) / (kRows * kCtas), tiles_c = (p.cols + bn - 1) / bn;
    const int64_t tiles = tiles_r * tiles_c;
    if (tiles > INT32_MAX / 16) return false;  // (32-bit tile arithmetic, with room for a group of tile columns)
    p.tiles_r = static_cast<uint32_t>(tiles_r);
    p.tiles_c = static_cast<uint32_t>(tiles_c);
    p.num_kb = static_cast<int>((c.K + kRowBytes - 1) / kRowBytes);
    p.splitk = std::min(splitk, p.num_kb);
    const int cluster = kCtas == 2 ? 2 : p.splitk;
    const int fit = capacity<kCtas, kSwap, T>(cluster);
    // CTAs of one tile need one accumulator
    if (tiles > fit && bn > kMaxBn2) return false;
    p.conv_col = tiles > fit ? 2 * bn : bn;
    const int smem = set_rings(p, kCtas, kSwap);
    if (fit < 1 || p.raw_stages < 2 || p.conv_stages < 2 || (p.splitk > 1 && tiles > fit)) return false;
    CUtensorMap mr{}, mc{}, mo{};
    const void *pr = kSwap ? c.B : c.A, *pc = kSwap ? c.A : c.B;
    const int64_t ldr = kSwap ? c.ldb : c.lda, ldc = kSwap ? c.lda : c.ldb;
    if (!encode_tiled_2d(&mr, CU_TENSOR_MAP_DATA_TYPE_UINT8, pr, c.K, p.rows, ldr, kRowBytes, kRows,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tiled_2d(&mc, CU_TENSOR_MAP_DATA_TYPE_UINT8, pc, c.K, p.cols, ldc, kRowBytes, bn / kCtas,
                         CU_TENSOR_MAP_SWIZZLE_128B))
        return false;
    if constexpr (!kSwap) {
        constexpr int kCols = 128 / sizeof(T);
        const CUtensorMapDataType dt = std::is_same<T, float>::value    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                       : std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                        : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        p.tma_store = bn % kCols == 0 && aligned16(c.C) && c.ldc * sizeof(T) % 16 == 0 &&
                      encode_tiled_2d(&mo, dt, c.C, c.N, c.M, c.ldc * sizeof(T), kCols, 32,
                                      CU_TENSOR_MAP_SWIZZLE_128B);
    }
    const uint64_t stall = take_injected_stall();
    p.inject_stall = stall ? 1 : 0;
    p.wait_limit_ns = stall ? stall : kWaitLimitNs;
    if (launch_chained(i8_umma_kernel<kCtas, kSwap, T>, static_cast<unsigned>(cluster * std::min<int64_t>(tiles, fit)), kThreads,
                       smem, stream, static_cast<unsigned>(cluster), mr, mc, mo, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return true;
}

template <typename T>
bool launch_typed(const I8Params &c, const I8Config &cfg, cudaStream_t stream)
{
    switch (cfg.variant) {
    case kI8PairTokens: return launch<2, false, T>(c, cfg.bn, 1, stream);
    case kI8PairChannels: return launch<2, true, T>(c, cfg.bn, 1, stream);
    case kI8Split: return launch<1, true, T>(c, cfg.bn, cfg.split, stream);
    default: return false;
    }
}

}  // namespace

bool i8_umma_config_ok(const I8Config &cfg)
{
    switch (cfg.variant) {
    case kI8PairTokens: return cfg.bn == 64 || cfg.bn == 128 || cfg.bn == 192 || cfg.bn == 256;
    case kI8PairChannels: return cfg.bn >= 32 && cfg.bn <= kMaxBn && cfg.bn % 32 == 0;
    case kI8Split: return cfg.bn >= 16 && cfg.bn <= kMaxSplitBn && cfg.bn % 16 == 0 && cfg.split >= 1 && cfg.split <= 8;
    default: return false;
    }
}

bool launch_i8_umma(const I8Params &c, int c_type, const I8Config &cfg, cudaStream_t stream)
{
    if (!i8_umma_config_ok(cfg)) return false;
    switch (c_type) {
    case DGEMM_TYPE_F32: return launch_typed<float>(c, cfg, stream);
    case DGEMM_TYPE_F16: return launch_typed<__half>(c, cfg, stream);
    case DGEMM_TYPE_BF16: return launch_typed<__nv_bfloat16>(c, cfg, stream);
    default: return false;
    }
}

bool i8_umma_fits(const I8Params &c, const I8Config &cfg)
{
    if (cfg.variant == kI8Split && cfg.split > 1) {
        const int64_t tiles = (c.N + kRows - 1) / kRows * ((c.M + cfg.bn - 1) / cfg.bn);
        const int fit = capacity<1, true, float>(cfg.split);
        return fit == 0 || tiles <= fit;
    }
    if ((cfg.variant == kI8PairTokens || cfg.variant == kI8PairChannels) && cfg.bn > kMaxBn2) {
        const bool tokens = cfg.variant == kI8PairTokens;
        const int64_t tiles = ((tokens ? c.M : c.N) + 2 * kRows - 1) / (2 * kRows) *
                              (((tokens ? c.N : c.M) + cfg.bn - 1) / cfg.bn);
        const int fit = capacity<2, false, float>(2);
        return fit == 0 || tiles <= fit;
    }
    return true;
}

int i8_read_status(int clear)
{
    return read_wait_status(clear);
}

}  // namespace dgemm

DGEMM_DEFINE_CHECK_READER(check_status_i8_umma)
