// box_edge.cuh -- the boxes at C's right edge that a TMA store would write past.
//
// A TMA store leaves out whole 16-byte words outside the tensor, not elements: where N
// elements end inside a word, the rest of that word is written too (N = 257 to FP32 at a
// pitch of 272: three elements a row), which may be a neighbouring matrix's.  Storing such
// boxes by their warp costs 300 x 257 x 512 in bf16 0.8 of 6.6 us and 2048 x 2047 x 512 0.2 to
// 0.9 of 10 to 11; a tensor of N's whole words and the last word's elements by the lanes of their
// rows was slower (4096 x 4097 x 2048 of 8 bits to FP32, with the old C, 81.9 for 76.3 us), the
// loop below unrolled or called no faster.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace dgemm {
namespace {

// Whether the box of `cols` columns from column c on ends in such a word.
__device__ __forceinline__ bool box_edge(int64_t c, int cols, int64_t N, int elem)
{
    return c + cols > N && (N * elem & 15) != 0;
}

// A warp's staged box (32 rows of 128 bytes, 16-byte word w of row r at w ^ (r mod 8)) to C's rows
// from row0 (up to row_end) and columns from c, 8 lanes a row.  `words`: C's rows lie on
// 16-byte boundaries.  All lanes call it, after their part of the box is written.
template <typename E>
__device__ __forceinline__ void store_box(E *C, int64_t ldc, int64_t row_end, int64_t N, int64_t row0, int64_t c, bool words,
                                          uint32_t box, int lane)
{
    constexpr int kPer = 16 / sizeof(E);  // values of a word
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < 32; i += 4) {
        const uint32_t r = static_cast<uint32_t>(i) + (static_cast<uint32_t>(lane) >> 3), w = static_cast<uint32_t>(lane) & 7u;
        const int64_t m = row0 + r, cw = c + w * kPer;
        if (m >= row_end || cw >= N) continue;
        const float4 f = ptx::ld_shared_v4f(box + r * 128u + ((w ^ (r & 7u)) << 4));
        const uint4 q = make_uint4(__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(f.z), __float_as_uint(f.w));
        E *dst = C + m * ldc + cw;
        if (words && cw + kPer <= N) {
            *reinterpret_cast<uint4 *>(dst) = q;
        } else {
            const E *v = reinterpret_cast<const E *>(&q);
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (cw + k < N) dst[k] = v[k];
        }
    }
    __syncwarp();  // the box is written again
}

}  // namespace
}  // namespace dgemm
