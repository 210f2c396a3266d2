// f8_tiles.cuh -- the output tiles of an 8-bit floating-point product, for one
// matrix or for rows sorted by expert, as the kernels walk them.
//
// A tile is `tile` tokens of one expert (from the expert's first row on) times a
// number of channels.  How many tokens an expert has is known on the GPU alone, so
// every CTA forms the table of the experts' first tiles for itself, in shared
// memory; one matrix is one expert with all the rows, without a table.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "f8.cuh"

namespace dgemm {
namespace {

// The table: first[e] tiles of tokens before expert e, start[e] its first row
// (experts + 1 entries each; the last ones: all tiles, the end of the last expert).
struct F8Table {
    uint32_t *first;
    int32_t *start;
};

// By one whole warp.  Offsets out of order are raised to the one before them, and
// all are kept within 0 .. M.
__device__ __forceinline__ void fill_table(const F8Params &p, int tile, const F8Table &table, int lane)
{
    const int32_t most = static_cast<int32_t>(p.M);
    int32_t before = 0;   // the offset before this batch, in order
    uint32_t tiles = 0;   // of the experts before this batch
    for (int e0 = 0; e0 <= p.experts; e0 += 32) {
        const int e = e0 + lane;
        int32_t at = e <= p.experts ? min(max(p.offsets[e], 0), most) : 0;
        if (lane == 0) at = max(at, before);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xFFFFFFFFu, at, o);
            if (lane >= o) at = max(at, v);
        }
        // this lane's expert begins at `at` and the expert before it began at `prev`
        int32_t prev = __shfl_up_sync(0xFFFFFFFFu, at, 1);
        if (lane == 0) prev = e0 == 0 ? at : before;
        uint32_t up = (static_cast<uint32_t>(at - prev) + static_cast<uint32_t>(tile - 1)) / static_cast<uint32_t>(tile);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, up, o);
            if (lane >= o) up += v;
        }
        if (e <= p.experts) {
            table.start[e] = at;
            table.first[e] = tiles + up;
        }
        before = __shfl_sync(0xFFFFFFFFu, at, 31);
        tiles += __shfl_sync(0xFFFFFFFFu, up, 31);
    }
}

// Upper bound of the tiles of tokens (at least one).
inline int64_t token_tiles_bound(const F8Params &p, int tile)
{
    if (!p.offsets) return (p.M + tile - 1) / tile;
    const int64_t some = p.M < p.experts ? p.M : p.experts;
    return p.M / tile + some > 0 ? p.M / tile + some : 1;
}

struct F8Tile {
    int expert;
    int32_t t0, t_end;  // its first token, and the end of its expert
    int64_t n0;         // its first channel
};

// Tile t, in groups of 8 tile columns (of channels) over all of the expert's tokens,
// so that tiles in flight together share a few bands of either operand.
__device__ __forceinline__ F8Tile find_tile(const F8Params &p, const F8Table &table, uint32_t all_tiles_t, uint32_t tiles_n,
                                            int tile, int bn, uint32_t t)
{
    F8Tile r;
    uint32_t first = 0, tiles_t = all_tiles_t;
    int32_t begin = 0;
    r.expert = 0;
    r.t_end = static_cast<int32_t>(p.M);
    if (p.offsets) {
        const uint32_t of_tokens = t / tiles_n;
        int lo = 0, hi = p.experts;  // the last expert whose first tile is not past it (so it has tiles)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (table.first[mid] <= of_tokens)
                lo = mid;
            else
                hi = mid;
        }
        r.expert = lo;
        first = table.first[lo];
        tiles_t = table.first[lo + 1] - first;
        begin = table.start[lo];
        r.t_end = table.start[lo + 1];
    }
    constexpr uint32_t kGroup = 8;
    const uint32_t local = t - first * tiles_n, per_group = kGroup * tiles_t;
    const uint32_t g = local / per_group, in = local - g * per_group;
    const uint32_t left = tiles_n - g * kGroup, gc = left < kGroup ? left : kGroup;
    const uint32_t band = in / gc;
    r.n0 = static_cast<int64_t>(g * kGroup + in - band * gc) * bn;
    r.t0 = begin + static_cast<int32_t>(band) * tile;
    return r;
}

}  // namespace
}  // namespace dgemm
