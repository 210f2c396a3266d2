// f8_umma.cu -- gemm_f8_tn and gemm_f8_tn_experts on the tensor cores (tcgen05).
//
//   C[m, n] = sum_b sa(m, b) sb(n, b) sum_(k in b) A[m, k] B[n, k] + bias[n] + beta C[m, n]
//
// The mathematics.  A block b is 128 K values, one 128-byte swizzled row of either
// operand: four MMAs of kind::f8f6f4 (K = 32) sum it into an accumulator in tensor
// memory, from zero.  The scales are any FP32 numbers, so they cannot join the MMA;
// the accumulator is read back block by block, multiplied by its row's and column's
// scales and added to sums in registers, in FP32, while the MMAs fill the next one.
//
// What bounds it.  For many tokens the epilogue: 8192 x 8192 x 4096 takes 233 us (2360 TFLOP/s),
// ~1000 clocks a block of a 256 x 256 tile, where the MMAs alone take 512 (8192 products a clock
// and SM) and the packed FMAs of a CTA 256 beside them; each of eight warps reads its 128 columns
// in eight dependent pieces.  In a long run the card's power limit takes the clock to 1957 of
// 2070 MHz, 248 us; zeros, which stay below the limit (740 of 1400 W), take 230 all the same.
// Of 137 us for 4864 x 8192 x 4096, 32 go without the FMAs and another 2 without reading the
// accumulators (1.25 x the time of the operations).  Larger pieces of the accumulator read at
// once, or the next block's first piece ahead, spilled sums (145 to 159 us).
// For few tokens the weights' bytes: there the channels are the MMA's rows and the tokens its
// columns (kSwap), so that no row of the tensor cores' work is padding that is loaded: 16
// tokens, 8 of 64 experts of 4096 x 2048 take 66 us, 7.2 TB/s (reads alone go faster than copies).
//
// Roles (12 warps):
//   warp 0      TMA producer: 128 bytes of K of both operands a stage;
//   warp 1      MMA issuer (in a pair's other CTA it tells the leader which of its own
//               stages have landed);
//   warp 2      the blocks' scales, into a ring;
//   warp 3      the table of tiles, at the start; then MMA issuer of the second half of
//               tiles of 256 columns;
//   warps 4-11  two groups of four: group g has columns g bn / 2 .. of the tile, warp w
//               of it the accumulator's rows 32 w ..: sums in registers, then C.
#include <algorithm>
#include <climits>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "bounded_wait.cuh"
#include "box_edge.cuh"
#include "chained.cuh"
#include "dgemm.h"
#include "f8.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "umma_warp.cuh"

#define DGEMM_UNIT 12
#include "checked.cuh"
#include "f8_tiles.cuh"
#include "rows.cuh"

namespace dgemm {
namespace {

constexpr int kRows = 128;                     // accumulator rows of a CTA: TMEM lanes
constexpr int kRowBytes = kF8Block;            // a block of K, one byte a value
constexpr int kRowsBytes = kRows * kRowBytes;
constexpr int kMaxStages = 12;
constexpr int kMaxAccs = 8;
constexpr int kSpan = 8;                        // blocks whose scales go together (a wait costs ~100 clocks)
constexpr int kScaleSlots = 2;
constexpr int kRowPitch = kSpan + 4;            // floats: 16-byte words, the rows of eight lanes on distinct banks
constexpr int kBoxBytes = 4096;                // epilogue staging: 32 rows x 128 bytes
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (4 + kEpiWarps);
constexpr int kSmemLimit = 227 * 1024;

struct Ctrl {
    uint64_t full[kMaxStages];       // a stage of this CTA has landed
    uint64_t peer_full[kMaxStages];  // leader: the other CTA's has
    uint64_t empty[kMaxStages];      // the MMAs have read it
    uint64_t acc_full[kMaxAccs];     // the MMAs of a block (a half of it: [half][slot]) are done
    uint64_t acc_empty[kMaxAccs];    // leader: every epilogue warp of the pair that reads them has
    uint64_t sc_full[kScaleSlots], sc_empty[kScaleSlots];
    uint64_t mma_done[2];
    uint64_t old_full[kEpiWarps];    // an epilogue warp's old C has landed in its boxes
    uint64_t never;                  // test hook: a barrier nothing arrives at
    uint32_t stop, limit_us;         // a wait ran out; a wait's limit, in 1024 ns (adjacent, see role_wait)
    uint32_t tmem_base;
};

struct Params {
    F8Params c;
    uint32_t tiles_n;      // tiles of channels
    uint32_t tiles_t;      // tiles of tokens, of one matrix (experts: in the table)
    int num_kb;            // blocks of K
    int stages;
    int boxes;             // staging boxes of an epilogue warp
    int splitk;            // CTAs of a cluster that share a tile (kSwap)
    int one_row;           // the tile's rows share their scales
    int a_words, b_words;  // an operand's scales along K lie in 16-byte words
    int tma_store;
    int tma_old;           // tiles of 128 columns: the old C comes by TMA too, into the two boxes
    int tok_rows, chan_rows;  // of a load's box: no more than the operand has
    uint32_t idesc;
    uint32_t wait_limit_us;
    int inject_stall;
};

// One kernel: kCtas CTAs share an MMA; kSwap: the rows are channels and the columns
// tokens; kBn columns to a tile; kUniform: the scales of a group's columns are one number
// (bands of 128 channels); kExtra: the call may have a bias or a beta (a kernel of their own
// for the CTA pairs: without, the sums of 256 columns just fit the registers, and 8 bytes a
// thread that do not cost 8192 x 8192 x 4096 20 of 237 us; with it 256 columns spill 44 bytes, or
// 64 with a scale a row, and a bias takes 269 us where 233 are without, 397 where 355).
template <int kCtas_, bool kSwap_, int kBn_, bool kUniform_, bool kExtra_>
struct Shape {
    static constexpr int kCtas = kCtas_, kBn = kBn_;
    static constexpr bool kSwap = kSwap_, kUniform = kUniform_, kExtra = kExtra_;
    static constexpr int kWgCols = kBn / 2;                     // columns of an epilogue group
    static constexpr int kTileRows = kRows * kCtas;
    static constexpr int kTokens = kSwap ? kBn : kTileRows, kChannels = kSwap ? kRows : kBn;  // of a tile
    // blocks that go from role to role together: a hand-over costs a role some hundred clocks,
    // which a block of few columns does not take
    static constexpr int kGroup = !kSwap ? 1 : kBn == 16 ? 4 : 2;
    static constexpr int kBlockBytes = kRowsBytes + kBn / kCtas * kRowBytes;
    static constexpr int kStageBytes = kGroup * kBlockBytes;
    // tiles of 256 columns: an MMA for each epilogue group's half, with accumulators and
    // barriers of its own, so that one group reads while the other's half is multiplied
    static constexpr int kHalves = kBn == 256 ? 2 : 1;
    static constexpr int kAccCols = kGroup * kBn;
    static constexpr int kAccs = 512 / kAccCols < kMaxAccs ? 512 / kAccCols : kMaxAccs;  // of either half
    static constexpr int kTmemCols = kAccs * kAccCols;
    // a slot of scales: [row][block], then [group][block] or [block][column]
    static constexpr int kSlotBytes = (kRowPitch * kRows + kSpan * (kUniform ? 2 : kBn)) * 4;
    static constexpr int kScaleBytes = kScaleSlots * kSlotBytes;
    // arrivals that a slot of scales takes: one for each lane's asynchronous copies, and where the
    // columns go through registers one that releases their stores
    static constexpr uint32_t kScaleArrivals = 32 + (kSwap ? 1 : 0);
    // sums of 128 columns and 32 more on their way do not fit the 168 registers a thread that
    // 384 threads share alike: the four other warps give 112 each of theirs
    static constexpr bool kMoveRegs = kWgCols >= 128;
    static_assert(!kMoveRegs || 128 * 56 + 256 * 224 <= 384 * 168, "what is taken was given");
    static_assert(kTmemCols >= 32 && (kTmemCols & (kTmemCols - 1)) == 0 && kTmemCols <= 512, "TMEM");
    static_assert(kSpan % kGroup == 0, "a group's scales are in one slot");
};

// ---- PTX

template <int kCtas>
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (kCtas == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// kChunk columns of this lane's row; the values are there after tmem_wait.
template <int kChunk>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[kChunk])
{
    if constexpr (kChunk == 32)
        ptx::tmem_ld_32x32b_x32(taddr, r);
    else if constexpr (kChunk == 16)
        tmem_ld_32x32b_x16(taddr, r);
    else
        tmem_ld_32x32b_x8(taddr, r);
}

// Wait for the loads of r; its values pass through the assembly, so that no use of them
// moves before the wait.
template <int kChunk>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[kChunk])
{
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < kChunk; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                     "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// 4 or 16 bytes from global to shared memory, without a register in between.
__device__ __forceinline__ void copy_async4(uint32_t dst, const float *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_async16(uint32_t dst, const float *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// One lane's arrival, without a branch around it.
__device__ __forceinline__ void arrive_if(bool yes, uint32_t bar)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
                 "r"(static_cast<uint32_t>(yes))
                 : "memory");
}

// The same on the barrier of a cluster's CTA (as arrive_remote).
__device__ __forceinline__ void arrive_remote_if(bool yes, uint32_t cluster_addr)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t@q mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];\n\t}" ::"r"(
            cluster_addr),
        "r"(static_cast<uint32_t>(yes))
        : "memory");
}

// Whether the phase of this parity is over, without waiting.
__device__ __forceinline__ bool test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// warp_wait, in line (a call would have to save the epilogue's sums around itself, and
// functions do not go with setmaxnreg), with the wait control at a shared-memory address.
__device__ __forceinline__ bool stopped(uint32_t wc)
{
    uint32_t v;
    asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(v) : "r"(wc) : "memory");
    return v != 0;
}

template <int kCtas>
__device__ __forceinline__ bool role_wait(uint32_t bar, uint32_t parity, uint32_t wc)
{
    if (probe<kCtas == 2>(bar, parity)) return true;
    uint32_t began = 0;  // in microseconds
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (probe<kCtas == 2>(bar, parity)) return true;
        if (__any_sync(0xFFFFFFFFu, stopped(wc))) return false;
        const uint32_t now = static_cast<uint32_t>(ptx::globaltimer_ns() >> 10) | 1u;
        if (began == 0) began = now;
        uint32_t limit;
        asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(limit) : "r"(wc + 4u) : "memory");
        if (__any_sync(0xFFFFFFFFu, now - began > limit)) {
            atomicExch(&g_wait_status, DGEMM_ERR_TIMEOUT);
            asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(wc), "r"(1u) : "memory");
            return false;
        }
    }
}

__device__ __forceinline__ bool role_drain(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, parity))
        if (ptx::globaltimer_ns() - t0 > kDrainLimitNs) return false;
    return true;
}

// ---- schedule

// The work of one CTA (pair, or cluster that splits K): tiles t0, t0 + dt, ... below
// `tiles`, and of each the blocks [kb0, kb1).
struct Sched {
    uint32_t t0, dt, tiles;
    int kb0, kb1;
    // groups of blocks this CTA works on in all
    __device__ __forceinline__ uint32_t groups(int of) const
    {
        return t0 < tiles ? ((tiles - t0 + dt - 1) / dt) * static_cast<uint32_t>((kb1 - kb0 + of - 1) / of) : 0u;
    }
};

template <typename S>
__device__ __forceinline__ Sched schedule(const Params &p, const F8Table &table)
{
    Sched s;
    const uint32_t n = S::kCtas == 2 ? 2u : static_cast<uint32_t>(p.splitk);
    s.t0 = blockIdx.x / n;
    s.dt = gridDim.x / n;
    s.tiles = (p.c.offsets ? table.first[p.c.experts] : p.tiles_t) * p.tiles_n;
    s.kb0 = 0;
    s.kb1 = p.num_kb;
    if (S::kCtas == 1 && n > 1) {
        const uint32_t r = ptx::cluster_ctarank();
        s.kb0 = static_cast<int>(r * static_cast<uint32_t>(p.num_kb) / n);
        s.kb1 = static_cast<int>((r + 1) * static_cast<uint32_t>(p.num_kb) / n);
    }
    return s;
}

template <typename S>
__device__ __forceinline__ F8Tile tile_at(const Params &p, const F8Table &table, uint32_t t)
{
    return find_tile(p.c, table, p.tiles_t, p.tiles_n, S::kTokens, S::kChannels, t);
}

// A ring's position: slot and the parity of its turn.
struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t slots)
    {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// ---- roles

// One stage: blocks kb .. kb_end (a group at most) of this CTA's part of the pair's tile, 128
// of its rows and half of its columns (by one thread).  Boxes that hold no row of the operand
// are left out (loads out of range cost TMA more than loads; what the stage holds in their
// place meets sums that are not stored).
template <typename S>
__device__ __forceinline__ void load_stage(const CUtensorMap *tmap_t, const CUtensorMap *tmap_w, const Params &p, uint32_t ring,
                                           Ctrl *ctrl, uint32_t slot, const F8Tile &tile, uint32_t rank, int kb, int kb_end)
{
    const int32_t tok = tile.t0 + static_cast<int32_t>(rank) * (S::kSwap ? S::kBn / S::kCtas : kRows);
    const int32_t chan = static_cast<int32_t>(tile.n0) + static_cast<int32_t>(rank) * (S::kSwap ? kRows : S::kBn / S::kCtas / S::kHalves);
    const bool toks = tok < p.c.M, chans[2] = {chan < p.c.N, S::kHalves == 2 && chan + 128 < p.c.N};
    const uint32_t full = ptx::smem_addr(&ctrl->full[slot]);
    const int n = min(S::kGroup, kb_end - kb);
    const int rows = (toks ? p.tok_rows : 0) + (chans[0] ? p.chan_rows : 0) + (chans[1] ? p.chan_rows : 0);
    ptx::mbar_arrive_expect_tx(full, n * rows * kRowBytes);
#pragma unroll
    for (int g = 0; g < S::kGroup; ++g) {
        if (g >= n) break;
        const uint32_t dst = ring + slot * S::kStageBytes + g * S::kBlockBytes;
        const int32_t k = (kb + g) * kRowBytes;  // (the innermost coordinate, a multiple of 128 bytes)
        if (toks) ptx::tma_load_3d(dst + (S::kSwap ? kRowsBytes : 0), tmap_t, full, k, tok, 0);
        // (with halves: of each half's 128 columns, this CTA's 64)
#pragma unroll
        for (int h = 0; h < S::kHalves; ++h)
            if (chans[h])
                ptx::tma_load_3d(dst + (S::kSwap ? 0 : kRowsBytes) + h * 64 * kRowBytes, tmap_w, full, k, chan + h * 128, tile.expert);
    }
}

// The first loads of the CTA, into the empty ring, by the thread that has set the ring's
// barriers up: they are in flight while the rest of the CTA (and its pair) starts.  Of one
// matrix only (the tiles of experts take the table).  Returns the number of stages.
template <typename S>
__device__ __forceinline__ int prefill(const CUtensorMap *tmap_t, const CUtensorMap *tmap_w, const Params &p, const F8Table &table,
                                       uint32_t ring, Ctrl *ctrl, uint32_t rank)
{
    const Sched sc = schedule<S>(p, table);
    const F8Tile tile = tile_at<S>(p, table, sc.t0);
    int n = 0;
    for (int kb = sc.kb0; kb < sc.kb1 && n < p.stages; kb += S::kGroup, ++n)
        load_stage<S>(tmap_t, tmap_w, p, ring, ctrl, n, tile, rank, kb, sc.kb1);
    return n;
}

// The rest of the loads, after the `done` stages of prefill.
template <typename S>
__device__ __forceinline__ void run_producer(const CUtensorMap *tmap_t, const CUtensorMap *tmap_w, const Params &p,
                                             const F8Table &table, uint32_t ring, Ctrl *ctrl, uint32_t rank, int done, uint32_t wc)
{
    const Sched sc = schedule<S>(p, table);
    const uint32_t stages = static_cast<uint32_t>(p.stages);
    Ring st;
    for (int i = 0; i < done; ++i) st.next(stages);
    bool ok = true;
    for (uint32_t t = sc.t0; ok && t < sc.tiles; t += sc.dt) {
        const F8Tile tile = tile_at<S>(p, table, t);
        for (int kb = sc.kb0 + (t == sc.t0 ? done * S::kGroup : 0); kb < sc.kb1; kb += S::kGroup) {
            ok = role_wait<1>(ptx::smem_addr(&ctrl->empty[st.slot]), st.phase ^ 1u, wc);
            if (!ok) break;
            if (elect_one()) load_stage<S>(tmap_t, tmap_w, p, ring, ctrl, st.slot, tile, rank, kb, sc.kb1);
            __syncwarp();
            st.next(stages);
        }
    }
    // Do not leave while TMA may still be writing into this CTA's memory, or the MMAs'
    // commits may still arrive here: stages before the current one were last filled in
    // this phase, the others (if at all: a barrier's phase 1 counts as over before its
    // first) in the one before.
    if (elect_one())
        for (uint32_t s = 0; s < stages; ++s) {
            role_drain(ptx::smem_addr(&ctrl->full[s]), s < st.slot ? st.phase : st.phase ^ 1u);
            if (ok) ok = role_drain(ptx::smem_addr(&ctrl->empty[s]), s < st.slot ? st.phase : st.phase ^ 1u);
        }
    __syncwarp();
}

// The other CTA of a pair: each stage that has landed here is the leader's to use.
template <typename S>
__device__ __forceinline__ void run_forwarder(const Params &p, const F8Table &table, Ctrl *ctrl, int lane, uint32_t wc)
{
    Ring st;
    for (uint32_t n = schedule<S>(p, table).groups(S::kGroup); n > 0; --n) {
        if (!role_wait<1>(ptx::smem_addr(&ctrl->full[st.slot]), st.phase, wc)) return;
        if (lane == 0) arrive_remote(ptx::mapa(ptx::smem_addr(&ctrl->peer_full[st.slot]), 0));
        __syncwarp();
        st.next(static_cast<uint32_t>(p.stages));
    }
}

// The MMAs of a block, or with kHalves == 2 those of the half that this warp issues.
template <typename S>
__device__ __forceinline__ void run_mma(const Params &p, const F8Table &table, uint32_t ring, Ctrl *ctrl, uint32_t tmem_base,
                                        uint32_t half, uint32_t wc)
{
    tmem_base = __shfl_sync(0xFFFFFFFFu, tmem_base, 0) + half * (S::kBn / 2);  // a uniform value for the compiler
    // descriptors of the first stage; a stage on is kStageBytes / 16, an MMA's K step 2, in
    // their address fields
    const uint64_t row_desc = ptx::smem_desc(ring, 16, 1024, ptx::kSw128);
    const uint64_t col_desc = ptx::smem_desc(ring + kRowsBytes + half * (S::kBn / S::kCtas / 2) * kRowBytes, 16, 1024, ptx::kSw128);
    const uint32_t idesc = p.idesc;
    const uint32_t full = ptx::smem_addr(ctrl->full), peer = ptx::smem_addr(ctrl->peer_full), empty = ptx::smem_addr(ctrl->empty);
    const uint32_t acc_full = ptx::smem_addr(ctrl->acc_full) + half * S::kAccs * 8, acc_empty = ptx::smem_addr(ctrl->acc_empty) + half * S::kAccs * 8;
    Ring st, acc;
    bool landed = false, both = S::kCtas == 1;  // this CTA's and the other's stage, as a look ahead saw them
    // test hook: wait on a barrier nothing arrives at, so the wait runs out
    bool ok = !p.inject_stall || role_wait<1>(ptx::smem_addr(&ctrl->never), 0, wc);
    const Sched sc = schedule<S>(p, table);
    int left = sc.kb1 - sc.kb0;  // blocks of the tile
    for (uint32_t n = sc.groups(S::kGroup); ok && n > 0; --n) {
        ok = (__all_sync(0xFFFFFFFFu, landed) || role_wait<1>(full + st.slot * 8, st.phase, wc)) &&
             (__all_sync(0xFFFFFFFFu, both) || role_wait<2>(peer + st.slot * 8, st.phase, wc)) &&
             role_wait<S::kCtas>(acc_empty + acc.slot * 8, acc.phase ^ 1u, wc);
        if (!ok) break;
        ptx::tc_fence_after();
        if (elect_one()) {
#pragma unroll
            for (int g = 0; g < S::kGroup; ++g) {
                if (g >= left) break;
                const uint32_t d = tmem_base + acc.slot * S::kAccCols + g * S::kBn, at = (st.slot * S::kStageBytes + g * S::kBlockBytes) / 16;
#pragma unroll
                for (int k = 0; k < kRowBytes / 32; ++k)
                    umma_f8<S::kCtas>(d, row_desc + at + k * 2, col_desc + at + k * 2, idesc, k == 0 ? 0u : 1u);
            }
            commit_all<S::kCtas>(acc_full + acc.slot * 8);
            commit_all<S::kCtas>(empty + st.slot * 8);
        }
        __syncwarp();
        left -= S::kGroup;
        if (left <= 0) left = sc.kb1 - sc.kb0;
        st.next(static_cast<uint32_t>(p.stages));
        acc.next(S::kAccs);
        landed = test(full + st.slot * 8, st.phase);
        if constexpr (S::kCtas == 2) both = test(peer + st.slot * 8, st.phase);
    }
    // Whatever the epilogue's waits came to, every MMA issued has finished before TMEM is
    // released (the elected thread is the same one each time).
    if (elect_one()) {
        if constexpr (S::kCtas == 2)
            ptx::umma_commit_pair_multicast(ptx::smem_addr(&ctrl->mma_done[half]), 0x1);
        else
            ptx::umma_commit(ptx::smem_addr(&ctrl->mma_done[half]));
        role_drain(ptx::smem_addr(&ctrl->mma_done[half]), 0);
    }
    __syncwarp();
}

// A row's scales of n blocks (kSpan at most) from p on; `words`: they lie in 16-byte words.
__device__ __forceinline__ void load_span(const float *p, int64_t blk, bool words, int n, float (&v)[kSpan])
{
    if (words && n == kSpan) {
#pragma unroll
        for (int j = 0; j < kSpan; j += 4) {
            const uint4 w = load_v4(p + j);
            v[j] = __uint_as_float(w.x);
            v[j + 1] = __uint_as_float(w.y);
            v[j + 2] = __uint_as_float(w.z);
            v[j + 3] = __uint_as_float(w.w);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < kSpan; ++j) v[j] = j < n ? load_f32(p + j * blk) : 0.f;
}

// The scales of kSpan blocks at a time: the CTA's 128 rows' (or the one number that they
// share: channels in bands of 128), then the tile's columns' (kUniform: one for each group
// of columns).  By asynchronous copies, each of which takes ~6 clocks a lane, also where all
// lanes read one address: so what rows share is copied once, and the columns of narrow tiles
// go through registers.  Rows past the operand have none, for sums that are not stored.
template <typename S>
__device__ __forceinline__ void run_scales(const Params &p, const F8Table &table, uint32_t scales, Ctrl *ctrl, uint32_t rank,
                                           int lane, uint32_t wc)
{
    const Sched sc = schedule<S>(p, table);
    const F8Operand &ro = S::kSwap ? p.c.b : p.c.a, &co = S::kSwap ? p.c.a : p.c.b;
    const bool in_words = sc.kb0 % 4 == 0;
    const bool row_words = in_words && (S::kSwap ? p.b_words : p.a_words), col_words = in_words && (S::kSwap ? p.a_words : p.b_words);
    Ring st;
    bool ok = true;
    for (uint32_t t = sc.t0; ok && t < sc.tiles; t += sc.dt) {
        const F8Tile tile = tile_at<S>(p, table, t);
        // of row (column) i of the tile: its scales from block kb on, or null
        auto place = [&](const F8Operand &o, bool token, int i, int kb) -> const float * {
            const int64_t at = token ? static_cast<int64_t>(tile.t0) + i : tile.n0 + i;
            if (at >= (token ? p.c.M : p.c.N)) return nullptr;
            return o.scale + (token ? 0 : tile.expert * p.c.sb_stride) + o.band(at) * o.s_row + kb * o.s_blk;
        };
        for (int kb = sc.kb0; kb < sc.kb1; kb += kSpan) {
            ok = role_wait<1>(ptx::smem_addr(&ctrl->sc_empty[st.slot]), st.phase ^ 1u, wc);
            if (!ok) break;
            const uint32_t dst = scales + st.slot * S::kSlotBytes, cols = dst + kRows * kRowPitch * 4;
            const int n = min(kSpan, sc.kb1 - kb);
            if (p.one_row) {
                if (lane < n) copy_async4(dst + lane * 4, place(ro, !S::kSwap, 0, kb + lane));
            } else {
#pragma unroll 1
                for (int i = 0; i < kRows; i += 32) {
                    const float *src = place(ro, !S::kSwap, static_cast<int>(rank) * kRows + i + lane, kb);
                    const uint32_t to = dst + (i + lane) * kRowPitch * 4;
                    if (!src) continue;
                    if (row_words && n == kSpan) {
#pragma unroll
                        for (int j = 0; j < kSpan; j += 4) copy_async16(to + j * 4, src + j);
                    } else {
                        for (int j = 0; j < n; ++j) copy_async4(to + j * 4, src + j * ro.s_blk);
                    }
                }
                __syncwarp();
            }
            if constexpr (S::kUniform) {
                const int j = lane % kSpan, group = lane / kSpan;
                if (group < 2 && j < n)
                    if (const float *src = place(co, S::kSwap, group * S::kWgCols, kb + j))
                        copy_async4(cols + (group * kSpan + j) * 4, src);
            } else if constexpr (!S::kSwap) {
#pragma unroll 1
                for (int i = 0; i < S::kBn; i += 32)
                    if (const float *src = place(co, S::kSwap, i + lane, kb))
                        for (int j = 0; j < n; ++j) copy_async4(cols + (j * S::kBn + i + lane) * 4, src + j * co.s_blk);
            } else {
#pragma unroll 1
                for (int i = 0; i < S::kBn; i += 64) {
                    float v[2][kSpan];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int c = i + h * 32 + lane;
                        if (c < S::kBn)
                            if (const float *src = place(co, S::kSwap, c, kb)) load_span(src, co.s_blk, col_words, n, v[h]);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int c = i + h * 32 + lane;
                        if (c >= S::kBn) continue;
#pragma unroll
                        for (int j = 0; j < kSpan; ++j) ptx::st_shared_f32(cols + (j * S::kBn + c) * 4, v[h][j]);
                    }
                }
            }
            __syncwarp();
            // (announces the lane's asynchronous copies and nothing else that it wrote)
            ptx::cp_async_mbar_arrive_noinc(ptx::smem_addr(&ctrl->sc_full[st.slot]));
            // the lanes' own stores are behind the __syncwarp, and one arrival releases them
            if constexpr (S::kSwap) arrive_if(lane == 0, ptx::smem_addr(&ctrl->sc_full[st.slot]));
            st.next(kScaleSlots);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---- epilogue

// What one epilogue warp keeps from tile to tile.
struct Epi {
    Ring acc, sc;
    uint32_t left;  // blocks to go
    uint32_t nbox;
    uint32_t old_phase;  // of the old C's barrier
    bool old_coming;     // loads of it that nothing has waited for
};

// The sums of one tile (or of this CTA's blocks of it), two columns a word.  A look at a
// barrier takes ~100 clocks to come back, so those of the next block are taken, and its
// scales fetched, beside the sums of this one.
template <typename S>
__device__ __forceinline__ bool sum_blocks(const Params &p, Ctrl *ctrl, uint32_t scales, uint32_t taddr, int row, int group,
                                           int blocks, int lane, Epi &e, uint64_t (&sum)[S::kWgCols / 2], uint32_t wc)
{
    constexpr int kChunk = S::kWgCols >= 128 ? 16 : S::kWgCols < 32 ? S::kWgCols : 32, kChunks = S::kWgCols / kChunk;
#pragma unroll
    for (int i = 0; i < S::kWgCols / 2; ++i) sum[i] = 0ull;
    const uint32_t acc_full = ptx::smem_addr(ctrl->acc_full) + (S::kHalves == 2 ? group * S::kAccs : 0) * 8;
    uint32_t acc_empty = ptx::smem_addr(ctrl->acc_empty) + (S::kHalves == 2 ? group * S::kAccs : 0) * 8;
    if constexpr (S::kCtas == 2) acc_empty = ptx::mapa(acc_empty, 0);
    const uint32_t sc_full = ptx::smem_addr(ctrl->sc_full), sc_empty = ptx::smem_addr(ctrl->sc_empty);
    if (!role_wait<1>(sc_full + e.sc.slot * 8, e.sc.phase, wc)) return false;
    uint32_t slot = scales + e.sc.slot * S::kSlotBytes;  // of this block's scales
    float r = ptx::ld_shared_f32(slot + row * (kRowPitch * 4)), c = 1.f;
    if constexpr (S::kUniform) c = ptx::ld_shared_f32(slot + kRows * kRowPitch * 4 + group * (kSpan * 4));
    bool ready = false;  // the block's accumulator, as the look ahead saw it
    int j = 0;           // the block's place in its span
    for (int left = blocks; left > 0; --left) {
        if (!__all_sync(0xFFFFFFFFu, ready) && !role_wait<1>(acc_full + e.acc.slot * 8, e.acc.phase, wc)) return false;
        ptx::tc_fence_after();
        const uint32_t src = taddr + e.acc.slot * S::kAccCols, release = acc_empty + e.acc.slot * 8;
        uint32_t d[kChunks > 1 ? 2 : 1][kChunk];
        tmem_load<kChunk>(src, d[0]);
        e.acc.next(S::kAccs);
        ready = test(acc_full + e.acc.slot * 8, e.acc.phase);
        // (the scales' product has to be a normal number, or 0: a multiplication of every value by
        // either scale takes 334 us for 8192 x 8192 x 4096, and a choice between the two, for each
        // block or for eight, 272 to 293 for 234, since its code moves this loop's registers)
        const float rc = S::kUniform ? r * c : r;
        const uint64_t r2 = pack2(rc, rc);
        const uint32_t cols = slot + (kRows * kRowPitch + j * S::kBn + group * S::kWgCols) * 4;
        const bool last = j == kSpan - 1 || left == 1;  // of its span
        bool more = false;
        if (!last) {
            r = ptx::ld_shared_f32(slot + (row * kRowPitch + j + 1) * 4);
            if constexpr (S::kUniform) c = ptx::ld_shared_f32(slot + (kRows * kRowPitch + group * kSpan + j + 1) * 4);
        } else if (left > 1) {
            const uint32_t n = e.sc.slot + 1 == kScaleSlots ? 0u : e.sc.slot + 1;
            more = test(sc_full + n * 8, e.sc.phase ^ (n == 0 ? 1u : 0u));
        }
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            uint32_t(&v)[kChunk] = d[k & 1];
            tmem_wait<kChunk>(v);  // (of the whole warp)
            if (k + 1 < kChunks) {
                tmem_load<kChunk>(src + (k + 1) * kChunk, d[(k + 1) & 1]);
            } else {
                ptx::tc_fence_before();
                // (an arrival that nothing waits for could reach a CTA that has left)
                const bool yes = lane == 0 && e.left > S::kAccs;
                if constexpr (S::kCtas == 2)
                    arrive_remote_if(yes, release);
                else
                    arrive_if(yes, release);
                --e.left;
            }
#pragma unroll
            for (int i = 0; i < kChunk; i += 4) {
                uint64_t x = pack2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                uint64_t y = pack2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                if constexpr (!S::kUniform) {
                    const float4 f = ptx::ld_shared_v4f(cols + (k * kChunk + i) * 4);
                    x = mul2(x, pack2(f.x, f.y));
                    y = mul2(y, pack2(f.z, f.w));
                }
                const int at = (k * kChunk + i) / 2;
                sum[at] = fma2(x, r2, sum[at]);
                sum[at + 1] = fma2(y, r2, sum[at + 1]);
            }
        }
        ++j;
        if (last) {
            __syncwarp();
            arrive_if(lane == 0, sc_empty + e.sc.slot * 8);
            e.sc.next(kScaleSlots);
            if (left > 1) {
                if (!__all_sync(0xFFFFFFFFu, more) && !role_wait<1>(sc_full + e.sc.slot * 8, e.sc.phase, wc)) return false;
                slot = scales + e.sc.slot * S::kSlotBytes;
                r = ptx::ld_shared_f32(slot + row * (kRowPitch * 4));
                if constexpr (S::kUniform) c = ptx::ld_shared_f32(slot + (kRows * kRowPitch + group * kSpan) * 4);
                j = 0;
            }
        }
    }
    return true;
}

// The same by groups of blocks: a group's accumulators are read together.
template <typename S>
__device__ __forceinline__ bool sum_groups(const Params &p, Ctrl *ctrl, uint32_t scales, uint32_t taddr, int row, int group,
                                           int blocks, int lane, Epi &e, uint64_t (&sum)[S::kWgCols / 2], uint32_t wc)
{
    constexpr int kChunk = S::kWgCols < 32 ? S::kWgCols : 32;
    static_assert(S::kWgCols <= 32 && !S::kUniform && S::kCtas == 1, "narrow tiles of single CTAs");
#pragma unroll
    for (int i = 0; i < S::kWgCols / 2; ++i) sum[i] = 0ull;
    const uint32_t acc_full = ptx::smem_addr(ctrl->acc_full), acc_empty = ptx::smem_addr(ctrl->acc_empty);
    const uint32_t sc_full = ptx::smem_addr(ctrl->sc_full), sc_empty = ptx::smem_addr(ctrl->sc_empty);
    int j = 0;  // the group's place in its span of scales
    for (int left = blocks; left > 0; left -= S::kGroup) {
        if (j == 0 && !role_wait<1>(sc_full + e.sc.slot * 8, e.sc.phase, wc)) return false;
        const uint32_t slot = scales + e.sc.slot * S::kSlotBytes;
        float r[S::kGroup];
#pragma unroll
        for (int g = 0; g < S::kGroup; ++g) r[g] = ptx::ld_shared_f32(slot + (row * kRowPitch + j + g) * 4);
        if (!role_wait<1>(acc_full + e.acc.slot * 8, e.acc.phase, wc)) return false;
        ptx::tc_fence_after();
        uint32_t d[S::kGroup][kChunk];
#pragma unroll
        for (int g = 0; g < S::kGroup; ++g)  // (past the last block: what an earlier one left, not used)
            tmem_load<kChunk>(taddr + e.acc.slot * S::kAccCols + g * S::kBn, d[g]);
#pragma unroll
        for (int g = 0; g < S::kGroup; ++g) tmem_wait<kChunk>(d[g]);
        ptx::tc_fence_before();
        // (an arrival that nothing waits for could reach a CTA that has left)
        arrive_if(lane == 0 && e.left > S::kAccs, acc_empty + e.acc.slot * 8);
#pragma unroll
        for (int g = 0; g < S::kGroup; ++g) {
            if (g >= left) break;  // uniform
            const uint64_t r2 = pack2(r[g], r[g]);
            const uint32_t cols = slot + (kRows * kRowPitch + (j + g) * S::kBn + group * S::kWgCols) * 4;
#pragma unroll
            for (int i = 0; i < kChunk; i += 4) {
                const float4 f = ptx::ld_shared_v4f(cols + i * 4);
                const uint64_t x = pack2(__uint_as_float(d[g][i]), __uint_as_float(d[g][i + 1]));
                const uint64_t y = pack2(__uint_as_float(d[g][i + 2]), __uint_as_float(d[g][i + 3]));
                sum[i / 2] = fma2(mul2(x, pack2(f.x, f.y)), r2, sum[i / 2]);
                sum[i / 2 + 1] = fma2(mul2(y, pack2(f.z, f.w)), r2, sum[i / 2 + 1]);
            }
        }
        --e.left;
        e.acc.next(S::kAccs);
        j += S::kGroup;
        if (j == kSpan || left <= S::kGroup) {
            __syncwarp();
            arrive_if(lane == 0, sc_empty + e.sc.slot * 8);
            e.sc.next(kScaleSlots);
            j = 0;
        }
    }
    return true;
}

template <typename S>
__device__ __forceinline__ bool sum_tile(const Params &p, Ctrl *ctrl, uint32_t scales, uint32_t taddr, int row, int group,
                                         int blocks, int lane, Epi &e, uint64_t (&sum)[S::kWgCols / 2], uint32_t wc)
{
    if constexpr (S::kGroup > 1)
        return sum_groups<S>(p, ctrl, scales, taddr, row, group, blocks, lane, e, sum, wc);
    else
        return sum_blocks<S>(p, ctrl, scales, taddr, row, group, blocks, lane, e, sum, wc);
}

template <typename T>
__device__ __forceinline__ uint32_t pack_bits(float a, float b)
{
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Rows = tokens: the bias added to this lane's sums, if the call has one.  (Apart from the
// stores, whose code, fetched anew for each tile, is a tenth of this.)
template <int kCols>
__device__ __forceinline__ void add_bias(const Params &p, uint64_t (&sum)[kCols / 2], int64_t col0)
{
    if (!p.c.bias) return;
#pragma unroll
    for (int i = 0; i < kCols; i += 2) {
        const int64_t c = col0 + i;
        sum[i / 2] = add2(sum[i / 2], pack2(c < p.c.N ? p.c.bias[c] : 0.f, c + 1 < p.c.N ? p.c.bias[c + 1] : 0.f));
    }
}

// Brings the old C of a warp's 32 rows x kCols columns into L2, ahead of their sums.
template <int kCols>
__device__ __forceinline__ void prefetch_old(const Params &p, int64_t row, int64_t row_end, int64_t col0)
{
    const int e = p.c.c_type == DGEMM_TYPE_F32 ? 4 : 2;
    if (row >= row_end) return;
    const char *src = static_cast<const char *>(p.c.C) + (row * p.c.ldc + col0) * e;
    for (int b = 0; b < kCols * e && col0 + b / e < p.c.N; b += 128) ptx::prefetch_l2(src + b);
}

// The old C of a box (32 rows of 128 bytes from row0 and column c) into it, 8 lanes a row.
template <typename T, int kCols>
__device__ __forceinline__ void load_old_box(const Params &p, uint32_t buf, int64_t row0, int64_t row_end, int64_t c, bool words, int lane)
{
    constexpr int kPer = 16 / sizeof(T);
    const T *const C = static_cast<const T *>(p.c.C);
    const uint32_t w = lane & 7u;
    const int64_t cw = c + w * kPer;
    constexpr int kMany = kCols <= 64 ? 8 : 4;  // words of a lane on their way (as the sums leave registers)
#pragma unroll 1
    for (int i = 0; i < 32; i += 4 * kMany) {
        uint4 q[kMany];
#pragma unroll
        for (int h = 0; h < kMany; ++h) {
            const int64_t m = row0 + i + h * 4 + (lane >> 3);
            const T *src = C + m * p.c.ldc + cw;
            if (m < row_end && words && cw + kPer <= p.c.N) {
                q[h] = *reinterpret_cast<const uint4 *>(src);
            } else {
                alignas(16) T v[kPer];
#pragma unroll
                for (int k = 0; k < kPer; ++k) v[k] = m < row_end && cw + k < p.c.N ? src[k] : from_f32<T>(0.f);
                q[h] = *reinterpret_cast<const uint4 *>(v);
            }
        }
#pragma unroll
        for (int h = 0; h < kMany; ++h) {
            const uint32_t r = i + h * 4 + (lane >> 3);
            ptx::st_shared_v4(buf + r * 128u + ((w ^ (r & 7u)) << 4), q[h]);
        }
    }
    __syncwarp();
}

// Rows = tokens, tiles of 128 columns: the old C of a warp's 32 rows x kCols columns on its way
// into the boxes that the sums will be stored from (what lies past C's edges arrives as zeros).
template <int kCols>
__device__ __forceinline__ void load_old(const Params &p, const CUtensorMap *tmap_o, int64_t row0, int64_t row_end, int64_t col0,
                                         uint32_t box, uint32_t bar, int lane, Epi &e)
{
    if (row0 >= row_end || col0 >= p.c.N || !DGEMM_CHECK(row0 >= 0 && col0 >= 0 && row0 < p.c.M)) return;  // warp-uniform
    e.old_coming = true;
    if (lane == 0) {
        const int cols = p.c.c_type == DGEMM_TYPE_F32 ? 32 : 64, n = col0 + cols < p.c.N ? kCols / cols : 1;
        ptx::bulk_wait_read<0>();  // the boxes' last stores have read them
        ptx::mbar_arrive_expect_tx(bar, n * kBoxBytes);
        for (int b = 0; b < n; ++b)
            ptx::tma_load_2d(box + ((e.nbox + b) & 1u) * kBoxBytes, tmap_o, bar, static_cast<int32_t>(col0) + b * cols,
                             static_cast<int32_t>(row0));
    }
    __syncwarp();
}

// Rows = tokens: beta times the old C added to a warp's sums, box by box through shared
// memory (the stores' box, whose last store has to have read it).
template <typename T, int kCols>
__device__ __forceinline__ void add_old(const Params &p, uint64_t (&sum)[kCols / 2], int64_t row0, int64_t row_end, int64_t col0,
                                        uint32_t box, int lane)
{
    constexpr int kPer = 16 / sizeof(T), kBoxCols = 128 / sizeof(T);
    const float beta = p.c.beta;
    if (beta == 0.f) return;
    const bool words = (reinterpret_cast<uintptr_t>(p.c.C) & 15u) == 0 && p.c.ldc % kPer == 0;
    if (lane == 0) ptx::bulk_wait_read<0>();
#pragma unroll
    for (int b = 0; b < kCols / kBoxCols; ++b) {
        const int64_t c = col0 + b * kBoxCols;
        if (c >= p.c.N) return;
        __syncwarp();
        load_old_box<T, kCols>(p, box, row0, row_end, c, words, lane);
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const uint4 q = ld_shared_v4(box + lane * 128u + ((w ^ (lane & 7u)) << 4));
            const T *o = reinterpret_cast<const T *>(&q);
#pragma unroll
            for (int i = 0; i < kPer; i += 2) {
                uint64_t &s = sum[(b * kBoxCols + w * kPer + i) / 2];
                s = fma2(pack2(to_f32(o[i]), to_f32(o[i + 1])), pack2(beta, beta), s);
            }
        }
    }
    __syncwarp();
}

// Rows = tokens: a warp's 32 rows from `row0` (up to row_end) x kCols columns from col0.  Boxes
// of 128 bytes of columns are staged in shared memory (128-byte swizzle: word w of row r at
// w ^ (r mod 8)) and stored by TMA, or, where the box holds rows that are not the expert's
// or TMA cannot describe C, word by word, 8 lanes a row.
template <typename T, int kCols, bool kExtra>
__device__ __forceinline__ void store_tokens(const Params &p, const CUtensorMap *tmap_o, uint64_t (&sum)[kCols / 2], int64_t row0,
                                             int64_t row_end, int64_t col0, uint32_t box, int lane, uint32_t bar, uint32_t wc, Epi &e)
{
    constexpr int kPer = 16 / sizeof(T), kBoxCols = 128 / sizeof(T);  // values of a word, of a row of the box
    uint32_t &nbox = e.nbox;
    if (row0 >= row_end) return;  // warp-uniform
    const bool in_box = kExtra && kCols == 64 && e.old_coming;  // the old C is where the sums go
    if constexpr (kExtra) {
        add_bias<kCols>(p, sum, col0);
        if (in_box) {
            if (!role_wait<1>(bar, e.old_phase, wc)) return;
            e.old_coming = false;
            e.old_phase ^= 1u;
        } else {
            add_old<T, kCols>(p, sum, row0, row_end, col0, box, lane);
        }
    }
    T *const C = static_cast<T *>(p.c.C);
    const bool whole = p.tma_store && (!p.c.offsets || row0 + 32 <= row_end);
    const bool words = (reinterpret_cast<uintptr_t>(C) & 15u) == 0 && p.c.ldc % kPer == 0;
#pragma unroll
    for (int b = 0; b < kCols / kBoxCols; ++b) {
        const int64_t c = col0 + b * kBoxCols;
        if (c >= p.c.N) return;
        const uint32_t buf = box + (p.boxes == 2 ? (nbox & 1u) * kBoxBytes : 0u);
        if (lane == 0) {  // this box's last store has read it
            if (p.boxes == 2)
                ptx::bulk_wait_read<1>();
            else
                ptx::bulk_wait_read<0>();
        }
        __syncwarp();
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            float v[kPer];
#pragma unroll
            for (int i = 0; i < kPer; i += 2) unpack2(sum[(b * kBoxCols + w * kPer + i) / 2], v[i], v[i + 1]);
            const uint32_t word = buf + lane * 128u + ((w ^ (lane & 7u)) << 4);
            uint4 q;
            if (in_box) {
                q = ld_shared_v4(word);
                const T *o = reinterpret_cast<const T *>(&q);
#pragma unroll
                for (int i = 0; i < kPer; ++i) v[i] = fmaf(p.c.beta, to_f32(o[i]), v[i]);
            }
            if constexpr (sizeof(T) == 2)
                q = make_uint4(pack_bits<T>(v[0], v[1]), pack_bits<T>(v[2], v[3]), pack_bits<T>(v[4], v[5]), pack_bits<T>(v[6], v[7]));
            else
                q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            ptx::st_shared_v4(word, q);
        }
        if (whole && !box_edge(c, kBoxCols, p.c.N, sizeof(T))) {
            ptx::fence_proxy_async_smem();  // the TMA store reads through the async proxy
            __syncwarp();
            if (lane == 0 && DGEMM_CHECK(row0 >= 0 && c >= 0 && row0 < p.c.M && c < p.c.N)) {
                ptx::tma_store_2d(tmap_o, buf, static_cast<int32_t>(c), static_cast<int32_t>(row0));
                ptx::bulk_commit();
            }
            ++nbox;
            continue;
        }
        if (DGEMM_CHECK(row_end <= p.c.M)) store_box(C, p.c.ldc, row_end, p.c.N, row0, c, words, buf, lane);
        if (kExtra && kCols == 64 && p.tma_old) {
            // a later tile's old C comes into this box by TMA, behind what the lanes wrote and read here
            ptx::fence_proxy_async_smem();
            __syncwarp();
        }
    }
}

// Rows = channels: this lane's channel n of tokens m0 .. m_end; the warp's lanes store
// consecutive channels.
template <typename T, int kCols>
__device__ __forceinline__ void store_channels(const Params &p, const uint64_t (&sum)[kCols / 2], int64_t n, int64_t m0, int64_t m_end)
{
    if (n >= p.c.N) return;
    constexpr int kMany = kCols == 16 ? 16 : 8;  // old values on their way together
    const float bias = p.c.bias ? p.c.bias[n] : 0.f;
    T *dst = static_cast<T *>(p.c.C) + m0 * p.c.ldc + n;
#pragma unroll
    for (int j0 = 0; j0 < kCols; j0 += kMany) {
        T old[kMany];
        if (p.c.beta != 0.f) {
#pragma unroll
            for (int j = 0; j < kMany; ++j)
                if (m0 + j0 + j < m_end) old[j] = dst[(j0 + j) * p.c.ldc];
        }
#pragma unroll
        for (int j = 0; j < kMany; j += 2) {
            float v[2];
            unpack2(sum[(j0 + j) / 2], v[0], v[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (m0 + j0 + j + i >= m_end || !DGEMM_CHECK(m0 + j0 + j + i < p.c.M)) continue;
                float x = v[i] + bias;
                if (p.c.beta != 0.f) x = fmaf(p.c.beta, to_f32(old[j + i]), x);
                dst[(j0 + j + i) * p.c.ldc] = from_f32<T>(x);
            }
        }
    }
}

// Brings a warp's old C (32 channels of kCols tokens) into L2, ahead of the sums.
template <int kCols>
__device__ __forceinline__ void prefetch_channels(const Params &p, int64_t n, int64_t m0, int64_t m_end, int lane)
{
    const int e = p.c.c_type == DGEMM_TYPE_F32 ? 4 : 2;
    if (n < p.c.N && lane < kCols && m0 + lane < m_end)
        ptx::prefetch_l2(static_cast<const char *>(p.c.C) + ((m0 + lane) * p.c.ldc + n) * e);
}

template <typename S, int kCols>
__device__ __forceinline__ void store_channels_any(const Params &p, const uint64_t (&sum)[kCols / 2], int64_t n, int64_t m0, int64_t m_end)
{
    switch (p.c.c_type) {
    case DGEMM_TYPE_F32: return store_channels<float, kCols>(p, sum, n, m0, m_end);
    case DGEMM_TYPE_F16: return store_channels<__half, kCols>(p, sum, n, m0, m_end);
    default: return store_channels<__nv_bfloat16, kCols>(p, sum, n, m0, m_end);
    }
}

// Split-K: the S CTAs of a cluster have each summed a range of one tile's blocks.  Groups of
// 8 columns are owned round-robin by the ranks; each CTA pushes the groups it does not own
// into the owner's idle stage ring, [sender slot][owned group][column quad][row] in 16-byte
// units, and the owner adds the partials in rank order, so the sum does not depend on timing.
__device__ __forceinline__ uint32_t recv_offset(uint32_t groups, uint32_t slot, uint32_t idx, uint32_t S, int q, int row)
{
    const uint32_t owned = (groups + S - 1) / S;
    return (((slot * owned + idx) * 2u + static_cast<uint32_t>(q)) * kRows + static_cast<uint32_t>(row)) * 16u;
}

template <typename S>
__device__ __forceinline__ void join_split(const Params &p, const F8Tile &tile, uint32_t ring, int row, int group, int64_t n,
                                           const uint64_t (&sum)[S::kWgCols / 2], uint32_t wc)
{
    constexpr uint32_t kGroups = S::kBn / 8, kMine = S::kWgCols / 8;  // of the tile, of this thread
    const uint32_t N = static_cast<uint32_t>(p.splitk), rank = ptx::cluster_ctarank();
    const uint32_t bytes = static_cast<uint32_t>(p.stages) * S::kStageBytes;
    ptx::cluster_sync();  // every CTA's sums are complete: the rings are idle
    const bool stop = __any_sync(0xFFFFFFFFu, stopped(wc));
    if (!stop) {
#pragma unroll
        for (uint32_t i = 0; i < kMine; ++i) {
            const uint32_t g = group * kMine + i, owner = g % N;
            if (owner == rank) continue;
            const uint32_t slot = rank < owner ? rank : rank - 1;
            if (!DGEMM_CHECK(recv_offset(kGroups, slot, g / N, N, 1, row) + 16 <= bytes)) continue;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float4 f;
                unpack2(sum[i * 4 + q * 2], f.x, f.y);
                unpack2(sum[i * 4 + q * 2 + 1], f.z, f.w);
                ptx::st_shared_cluster_v4(ptx::mapa(ring + recv_offset(kGroups, slot, g / N, N, q, row), owner), f);
            }
        }
    }
    __syncwarp();
    ptx::cluster_sync();  // every partial has landed in its owner
    if (stop) return;
#pragma unroll
    for (uint32_t i = 0; i < kMine; ++i) {
        const uint32_t g = group * kMine + i;
        if (g % N != rank) continue;
        uint64_t total[4] = {};
        for (uint32_t s = 0; s < N; ++s) {
            const uint32_t slot = s < rank ? s : s - 1;
            if (s != rank && !DGEMM_CHECK(recv_offset(kGroups, slot, g / N, N, 1, row) + 16 <= bytes)) continue;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint64_t a = sum[i * 4 + q * 2], b = sum[i * 4 + q * 2 + 1];
                if (s != rank) {
                    const float4 f = ptx::ld_shared_v4f(ring + recv_offset(kGroups, slot, g / N, N, q, row));
                    a = pack2(f.x, f.y);
                    b = pack2(f.z, f.w);
                }
                total[q * 2] = add2(total[q * 2], a);
                total[q * 2 + 1] = add2(total[q * 2 + 1], b);
            }
        }
        store_channels_any<S, 8>(p, total, n, tile.t0 + g * 8, tile.t_end);
    }
}

template <typename S>
__device__ __forceinline__ void run_epilogue(const Params &p, const CUtensorMap *tmap_o, const F8Table &table, uint32_t ring,
                                             uint32_t box, uint32_t scales, Ctrl *ctrl, uint32_t tmem_base, uint32_t rank,
                                             int warp, int lane, uint32_t wc)
{
    const Sched sc = schedule<S>(p, table);
    const int quarter = warp & 3, group = (warp - 4) >> 2, row = quarter * 32 + lane;
    const int sc_row = S::kSwap && p.one_row ? 0 : row;
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + group * S::kWgCols;
    const uint32_t my_box = box + static_cast<uint32_t>(warp - 4) * p.boxes * kBoxBytes, bar = ptx::smem_addr(&ctrl->old_full[warp - 4]);
    Epi e{{}, {}, sc.groups(S::kGroup), 0, 0, false};
    uint64_t sum[S::kWgCols / 2];
    if (S::kSwap && p.splitk > 1) {  // one tile, uniform over the cluster
        const F8Tile tile = tile_at<S>(p, table, sc.t0);
        if (p.c.beta != 0.f)
            prefetch_channels<S::kWgCols>(p, tile.n0 + quarter * 32, tile.t0 + group * S::kWgCols, tile.t_end, lane);
        sum_tile<S>(p, ctrl, scales, taddr, sc_row, group, sc.kb1 - sc.kb0, lane, e, sum, wc);  // (a time-out raises the abort flag)
        __syncwarp();
        if constexpr (S::kSwap) join_split<S>(p, tile, ring, row, group, tile.n0 + row, sum, wc);
        return;
    }
    for (uint32_t t = sc.t0; t < sc.tiles; t += sc.dt) {
        if (S::kExtra && p.c.beta != 0.f) {
            const F8Tile tile = tile_at<S>(p, table, t);
            if constexpr (S::kSwap)
                prefetch_channels<S::kWgCols>(p, tile.n0 + quarter * 32, tile.t0 + group * S::kWgCols, tile.t_end, lane);
            else if (S::kBn == 128 && p.tma_old)
                load_old<S::kWgCols>(p, tmap_o, static_cast<int64_t>(tile.t0) + rank * kRows + quarter * 32, tile.t_end,
                                     tile.n0 + group * S::kWgCols, my_box, bar, lane, e);
            else
                prefetch_old<S::kWgCols>(p, static_cast<int64_t>(tile.t0) + rank * kRows + row, tile.t_end, tile.n0 + group * S::kWgCols);
        }
        if (!sum_tile<S>(p, ctrl, scales, taddr, sc_row, group, sc.kb1 - sc.kb0, lane, e, sum, wc)) break;
        const F8Tile tile = tile_at<S>(p, table, t);
        if constexpr (S::kSwap) {
            store_channels_any<S, S::kWgCols>(p, sum, tile.n0 + rank * kRows + row, tile.t0 + group * S::kWgCols, tile.t_end);
        } else {
            const int64_t row0 = tile.t0 + rank * kRows + quarter * 32, col0 = tile.n0 + group * S::kWgCols;
            switch (p.c.c_type) {
            case DGEMM_TYPE_F32: store_tokens<float, S::kWgCols, S::kExtra>(p, tmap_o, sum, row0, tile.t_end, col0, my_box, lane, bar, wc, e); break;
            case DGEMM_TYPE_F16: store_tokens<__half, S::kWgCols, S::kExtra>(p, tmap_o, sum, row0, tile.t_end, col0, my_box, lane, bar, wc, e); break;
            default: store_tokens<__nv_bfloat16, S::kWgCols, S::kExtra>(p, tmap_o, sum, row0, tile.t_end, col0, my_box, lane, bar, wc, e);
            }
            if (e.old_coming) break;  // its wait ran out
        }
        __syncwarp();
    }
    if (!S::kSwap && lane == 0) {
        if (e.old_coming) role_drain(bar, e.old_phase);  // (after an abort)
        ptx::bulk_wait<0>();                             // loads and stores done before the CTA leaves
    }
}

template <typename S>
__global__ void __launch_bounds__(kThreads, 1)
    f8_umma_kernel(const __grid_constant__ CUtensorMap tmap_t, const __grid_constant__ CUtensorMap tmap_w,
                   const __grid_constant__ CUtensorMap tmap_o, const Params p)
{
    // stage ring | staging boxes | scales | control | table of tiles
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t ring = ptx::smem_addr(smem);
    const uint32_t box = ring + static_cast<uint32_t>(p.stages) * S::kStageBytes;
    const uint32_t scales = box + (S::kSwap ? 0u : static_cast<uint32_t>(kEpiWarps * p.boxes) * kBoxBytes);
    Ctrl *ctrl = reinterpret_cast<Ctrl *>(smem + (scales - ring) + S::kScaleBytes);
    uint32_t *words = reinterpret_cast<uint32_t *>(ctrl + 1);
    const F8Table table{words, reinterpret_cast<int32_t *>(words + p.c.experts + 1)};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = S::kCtas == 2 ? (ptx::cluster_ctarank() & 1u) : 0u;

    int loaded = 0;  // stages already under way (warp 0)
    if (warp == 0) {
        if (elect_one()) {
            for (int s = 0; s < kMaxStages; ++s) {
                ptx::mbar_init(ptx::smem_addr(&ctrl->full[s]), 1);
                ptx::mbar_init(ptx::smem_addr(&ctrl->empty[s]), S::kHalves);
            }
            ptx::fence_mbarrier_init();
            chain_wait();  // (what follows reads the call's operands)
            if (!p.c.offsets) loaded = prefill<S>(&tmap_t, &tmap_w, p, table, ring, ctrl, rank);
        }
        loaded = __reduce_max_sync(0xFFFFFFFFu, loaded);
    } else if (warp == 1) {
        if constexpr (S::kCtas == 2) {
            ptx::tmem_alloc_pair(ptx::smem_addr(&ctrl->tmem_base), S::kTmemCols);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(ptx::smem_addr(&ctrl->tmem_base), S::kTmemCols);
            ptx::tmem_relinquish();
        }
    } else if (warp == 2 && elect_one()) {
        for (int s = 0; s < kMaxStages; ++s) ptx::mbar_init(ptx::smem_addr(&ctrl->peer_full[s]), 1);
        for (int a = 0; a < kMaxAccs; ++a) {
            ptx::mbar_init(ptx::smem_addr(&ctrl->acc_full[a]), 1);
            ptx::mbar_init(ptx::smem_addr(&ctrl->acc_empty[a]), kEpiWarps / S::kHalves * S::kCtas);
        }
        for (int s = 0; s < kScaleSlots; ++s) {
            ptx::mbar_init(ptx::smem_addr(&ctrl->sc_full[s]), S::kScaleArrivals);
            ptx::mbar_init(ptx::smem_addr(&ctrl->sc_empty[s]), kEpiWarps);
        }
        for (int h = 0; h < 2; ++h) ptx::mbar_init(ptx::smem_addr(&ctrl->mma_done[h]), 1);
        for (int w = 0; w < kEpiWarps; ++w) ptx::mbar_init(ptx::smem_addr(&ctrl->old_full[w]), 1);
        ptx::mbar_init(ptx::smem_addr(&ctrl->never), 1);
        ctrl->stop = 0u;
        ctrl->limit_us = p.wait_limit_us;
        ptx::fence_mbarrier_init();
        if (p.tma_store) ptx::prefetch_tmap(&tmap_o);
    }
    __syncwarp();
    const uint32_t wc = ptx::smem_addr(&ctrl->stop);
    chain_wait();  // (everything below reads or writes the call's operands)
    chain_next();
    if (warp == 3 && p.c.offsets) fill_table(p.c, S::kTokens, table, lane);
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    // both CTAs' barriers exist (fence_mbarrier_init above) before any cross-CTA signal
    if constexpr (S::kCtas == 2) cluster_meet();
    ptx::tc_fence_after();
    const uint32_t tmem_base = ctrl->tmem_base;

    if (warp < 4) {
        if constexpr (S::kMoveRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {
            run_producer<S>(&tmap_t, &tmap_w, p, table, ring, ctrl, rank, loaded, wc);
        } else if (warp == 1 || (S::kHalves == 2 && warp == 3)) {
            if (rank == 0)
                run_mma<S>(p, table, ring, ctrl, tmem_base, warp >> 1, wc);
            else if (warp == 1)
                run_forwarder<S>(p, table, ctrl, lane, wc);
        } else if (warp == 2) {
            run_scales<S>(p, table, scales, ctrl, rank, lane, wc);
        }
        __syncwarp();
        if (S::kSwap && p.splitk > 1) {  // (join_split's barriers)
            ptx::cluster_sync();
            ptx::cluster_sync();
        }
    } else {
        if constexpr (S::kMoveRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        run_epilogue<S>(p, &tmap_o, table, ring, box, scales, ctrl, tmem_base, rank, warp, lane, wc);
    }

    __syncwarp();  // the barriers below are warp-aligned: reconverge the single-lane roles
    ptx::tc_fence_before();
    __syncthreads();  // every role of this CTA is done
    if constexpr (S::kCtas == 2) {
        // after an abort, arrivals on the leader's barriers that nothing has waited for may be
        // under way: they come before this CTA's part in the meeting
        if (__any_sync(0xFFFFFFFFu, stopped(wc))) fence_cluster();
        cluster_meet();  // no CTA leaves while the other may still signal or read it
    }
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        if constexpr (S::kCtas == 2)
            ptx::tmem_dealloc_pair(tmem_base, S::kTmemCols);
        else
            ptx::tmem_dealloc(tmem_base, S::kTmemCols);
    }
}

// ---- host side

// Dynamic shared memory of a launch, and its rings: two boxes a warp if that leaves five
// stages, else one.
template <typename S>
int set_rings(Params &p)
{
    const int fixed = S::kScaleBytes + static_cast<int>(sizeof(Ctrl)) + 8 * (p.c.experts + 1);
    p.boxes = 0;
    if (!S::kSwap) p.boxes = (kSmemLimit - fixed - 2 * kEpiWarps * kBoxBytes) / S::kStageBytes >= 5 ? 2 : 1;
    const int boxes = kEpiWarps * p.boxes * kBoxBytes;
    p.stages = std::min(kMaxStages, (kSmemLimit - fixed - boxes) / S::kStageBytes);
    return fixed + boxes + p.stages * S::kStageBytes;
}

// CTAs (or clusters of `cluster`) of the kernel that can be resident at once on the
// current device, cached; 0 if it cannot run.
template <typename S>
int capacity(int cluster)
{
    constexpr int kMaxDevices = 64;
    static int cached[kMaxDevices][9];
    static std::once_flag once[kMaxDevices];
    int dev = 0;
    if (cluster < 1 || cluster > 8 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    std::call_once(once[dev], [dev] {
        auto kernel = f8_umma_kernel<S>;
        int sms = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) == cudaSuccess &&
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) {
            cached[dev][1] = sms;
            for (int s = 2; s <= (S::kCtas == 2 ? 2 : 8); ++s) {
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

template <typename S>
bool launch(const F8Params &c, int splitk, cudaStream_t stream)
{
    Params p{};
    p.c = c;
    const int64_t tiles_n = (c.N + S::kChannels - 1) / S::kChannels, tiles = tiles_n * token_tiles_bound(c, S::kTokens);
    if (tiles > INT32_MAX / 16) return false;  // (32-bit tile arithmetic, with room for a group of tile columns)
    p.tiles_n = static_cast<uint32_t>(tiles_n);
    p.tiles_t = static_cast<uint32_t>((c.M + S::kTokens - 1) / S::kTokens);
    p.num_kb = static_cast<int>((c.K + kRowBytes - 1) / kRowBytes);
    p.splitk = splitk;
    if (tiles / 76 * p.num_kb > INT32_MAX) return false;  // blocks of one CTA
    const int cluster = S::kCtas == 2 ? 2 : p.splitk;
    const int fit = capacity<S>(cluster);
    const int smem = set_rings<S>(p);
    if (fit < 1 || p.stages < 2 || (p.splitk > 1 && tiles > fit)) return false;
    constexpr int kTokBox = S::kSwap ? S::kBn / S::kCtas : kRows, kChanBox = S::kSwap ? kRows : S::kBn / S::kCtas / S::kHalves;
    p.one_row = S::kSwap && c.b.block == kF8Block;
    p.a_words = c.a.s_blk == 1 && c.a.s_row % 4 == 0 && aligned16(c.a.scale);
    p.b_words = c.b.s_blk == 1 && c.b.s_row % 4 == 0 && c.sb_stride % 4 == 0 && aligned16(c.b.scale);
    const uint64_t k = static_cast<uint64_t>(c.K), m = static_cast<uint64_t>(c.M), n = static_cast<uint64_t>(c.N);
    p.tok_rows = static_cast<int>(std::min<int64_t>(kTokBox, c.M));
    p.chan_rows = static_cast<int>(std::min<int64_t>(kChanBox, c.N));
    CUtensorMap mt{}, mw{}, mo{};
    if (!encode_tiled_3d(&mt, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.a.p, {k, m, 1}, {static_cast<uint64_t>(c.a.ld), m * c.a.ld},
                         {kRowBytes, static_cast<uint32_t>(p.tok_rows), 1}, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tiled_3d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.b.p, {k, n, static_cast<uint64_t>(c.experts)},
                         {static_cast<uint64_t>(c.b.ld), c.experts > 1 ? static_cast<uint64_t>(c.b_stride) : n * c.b.ld},
                         {kRowBytes, static_cast<uint32_t>(p.chan_rows), 1}, CU_TENSOR_MAP_SWIZZLE_128B))
        return false;
    if (!S::kSwap) {
        const int e = c.c_type == DGEMM_TYPE_F32 ? 4 : 2;
        const CUtensorMapDataType dt = c.c_type == DGEMM_TYPE_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                       : c.c_type == DGEMM_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        p.tma_store = aligned16(c.C) && c.ldc * e % 16 == 0 &&
                      encode_tiled_2d(&mo, dt, c.C, n, m, static_cast<uint64_t>(c.ldc) * e, static_cast<uint32_t>(128 / e), 32,
                                      CU_TENSOR_MAP_SWIZZLE_128B);
    }
    p.tma_old = p.tma_store && p.boxes == 2;
    // D f32; the types of the rows' and the columns' operand; both K-major; N = kBn (or a half), M = 128 rows a CTA
    const uint32_t rows_type = static_cast<uint32_t>((S::kSwap ? c.b : c.a).type), cols_type = static_cast<uint32_t>((S::kSwap ? c.a : c.b).type);
    p.idesc = (1u << 4) | (rows_type << 7) | (cols_type << 10) | (static_cast<uint32_t>(S::kBn / S::kHalves >> 3) << 17) |
              (static_cast<uint32_t>(S::kTileRows >> 4) << 24);
    const uint64_t stall = take_injected_stall();
    p.inject_stall = stall ? 1 : 0;
    p.wait_limit_us = static_cast<uint32_t>(std::min<uint64_t>((stall ? stall : kWaitLimitNs) >> 10, UINT32_MAX / 2));
    if (launch_chained(f8_umma_kernel<S>, static_cast<unsigned>(cluster * std::min<int64_t>(tiles, fit)), kThreads, smem, stream,
                       static_cast<unsigned>(cluster), mt, mw, mo, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return true;
}

template <int kBn>
bool launch_pair(const F8Params &c, cudaStream_t stream)
{
    const bool uniform = c.b.block == kF8Block, extra = c.bias || c.beta != 0.f;
    if (uniform)
        return extra ? launch<Shape<2, false, kBn, true, true>>(c, 1, stream) : launch<Shape<2, false, kBn, true, false>>(c, 1, stream);
    return extra ? launch<Shape<2, false, kBn, false, true>>(c, 1, stream) : launch<Shape<2, false, kBn, false, false>>(c, 1, stream);
}

}  // namespace

bool f8_umma_config_ok(const F8Config &cfg)
{
    switch (cfg.variant) {
    case kF8Pair: return cfg.bn == 128 || cfg.bn == 256;
    case kF8Channels:
        return (cfg.bn == 16 || cfg.bn == 32 || cfg.bn == 64) && cfg.split >= 1 && cfg.split <= 8;
    default: return false;
    }
}

bool launch_f8_umma(const F8Params &c, const F8Config &cfg, cudaStream_t stream)
{
    if (!f8_umma_config_ok(cfg) || (cfg.split > 1 && (c.offsets || cfg.split > (c.K - 1) / kF8Block + 1))) return false;
    if (cfg.variant == kF8Pair) return cfg.bn == 256 ? launch_pair<256>(c, stream) : launch_pair<128>(c, stream);
    switch (cfg.bn) {
    case 16: return launch<Shape<1, true, 16, false, true>>(c, cfg.split, stream);
    case 32: return launch<Shape<1, true, 32, false, true>>(c, cfg.split, stream);
    default: return launch<Shape<1, true, 64, false, true>>(c, cfg.split, stream);
    }
}

int f8_read_status(int clear)
{
    return read_wait_status(clear);
}

}  // namespace dgemm

DGEMM_DEFINE_CHECK_READER(check_status_f8_umma)
