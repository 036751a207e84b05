// mx_shape.h -- plain arithmetic of the grouped MXFP4 product that its kernel
// and its launch share with the checks on the host: what a load may read, the
// count of items, and which form of the kernel a call takes.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmoe {

// A byte offset behind every buffer (buffers are shorter than 2^31 bytes).
constexpr uint32_t kMxOutside = 0x80000000u;

// Bytes of a buffer of `bytes` that are left from byte `at` on.  A load's descriptor starts at its
// step's first byte and holds these, so the hardware compares a lane's whole remaining offset with
// what is left, and a step behind the buffer's end, or of no tile, reads nothing: with the step in the
// instruction's scalar offset this would hang on whether and how that offset enters the comparison.
// Both are below 2^31, so their difference has a sign, and the scalar units can do all of it.
__host__ __device__ inline uint32_t mx_bytes_left(uint32_t bytes, uint32_t at)
{
    const int32_t left = (int32_t)(bytes - at);
    return left > 0 ? (uint32_t)left : 0u;
}

// Largest rows * N of a call: items (tiles of 32 x 64 or more) then count in 32 bits.
constexpr int64_t kMxMaxOutputs = int64_t(1) << 40;

// Items of `tiles` m-tiles of `bm` rows with n_tiles column tiles each.  Experts whose offsets do not
// decrease have at most one partial tile each; a table with more tiles than that decreases somewhere, and
// could count past 32 bits and lead the search for an item outside the output: it gets no items.
__host__ __device__ inline int mx_items(int tiles, int n_tiles, int rows, int bm, int E)
{
    return tiles <= rows / bm + (E < rows ? E : rows) ? tiles * n_tiles : 0;
}

constexpr int kMxCUs = 256;

// Tile rows x columns and LDS stages.
enum class MxTile { k32x64s4, k64x128s4, k128x128s4, k64x128s2, k128x128s2, k256x256s2 };

// Tile by the rows an expert gets if all of them (or, of fewer rows, one a row)
// share alike, by how many tiles that makes for 256 CUs, and in the end by the
// rounds that they take.  The host knows the offsets' sizes only, so routes that
// meet in a few of many experts get the tile of an even spread: 8192 rows all on
// 4 of 512 experts, N 4096, K 2048 take 126 us, on 4 of 128 experts 63, and with
// those 4 experts alone 49.  Measured in us, weights out of cache, stages in
// brackets:
//                                32x64 [4]  64x128 [4]  64x128 [2]  128x128 [2]
//   E 1, N 4096, K 14336, rows 64   18.8       30.5        45.4        48.7
//                        rows 1024  92.3       59.6        53.5        53.7 (43.4 with four stages)
//   E 1, N 4096, K 4096, rows 256   10.1       11.5        13.3        15.2
//                        rows 512   15.5       12.2        13.9        15.5
//   E 8, N 4096, K 4096, rows 256   21.6       17.8        20.5        21.9
//                        rows 512   30.1       23.7        23.1        27.7
//                        rows 1024  42.7       34.5        38.2        29.9
//   E 8, N 2048, K 4096, rows 1024   -         23.6        22.9        20.9 (18.0)
//   E 8, N 4096, K 2048, rows 128   10.6        -          12.3        13.2
//                        rows 1024   -          -          22.8        19.0
//   E 512, N 1536, K 2048, rows 60  20.8        -          21.0        23.9
//   E 512, N 2048, K 768, rows 512  50.3 [2]    -          49.1        52.9
// The four-stage forms load up to a tile ahead, so K must make two groups.
// A round of 256 x 256 (one a CU) takes 1.6 times as long as one of 128 x 128
// (two a CU), for twice the work; rounds of either, and the time of both:
//   E 8, N 4096, K 2048:  rows 4096: 2 and 3, 43.0 and 37.2;  rows 8192: 3 and 5, 65.4 and 64.3
//   E 8, N 8192, K 4096:  rows 2048: 2 and 3, 71.1 and 67.5;  rows 4096: 3 and 5, 99.8 and 115.7
//   E 1, N 4096, K 4096:  rows 4096: 1 and 2, 40.5 and 43.9;  rows 8192: 2 and 4, 71.5 and 81.2
//   E 1, N 8192, K 8192:  rows 4096: 2 and 4, 133.5 and 182.1
inline MxTile mx_tile(int E, int N, int K, int rows)
{
    const int64_t experts = E < rows ? E : rows;
    const int64_t mean = rows / experts;
    auto tiles = [&](int bm, int bn) {  // of several experts, each one's last tile counts half
        const int64_t m = experts == 1 ? (rows + bm - 1) / bm : rows / bm + (experts + 1) / 2;
        return m * ((N + bn - 1) / bn);
    };
    const int64_t middle = tiles(128, 128);
    if (K > 1024) {
        if (mean <= 16 || tiles(32, 64) <= 2 * kMxCUs) return MxTile::k32x64s4;
        if (tiles(64, 128) <= kMxCUs) return MxTile::k64x128s4;
        if (mean > 64 && middle <= kMxCUs) return MxTile::k128x128s4;
    }
    if (mean <= 64 || middle < kMxCUs) return MxTile::k64x128s2;
    const int64_t middle_rounds = (middle + 2 * kMxCUs - 1) / (2 * kMxCUs);
    const int64_t large_rounds = (tiles(256, 256) + kMxCUs - 1) / kMxCUs;
    if (8 * large_rounds > 5 * middle_rounds) return MxTile::k128x128s2;
    return MxTile::k256x256s2;
}

// Whether K fills whole groups of steps (of two stages, whole halves) and the scale rows are 16-byte
// aligned: scales then take the direct path to LDS, and no step has a tail.
inline bool mx_whole(int stages, int K, const void* a_scales, const void* w_scales)
{
    return K % (stages == 2 && K > 512 ? 512 : 1024) == 0 && reinterpret_cast<uintptr_t>(a_scales) % 16 == 0 &&
           reinterpret_cast<uintptr_t>(w_scales) % 16 == 0;
}

// Whether a tile ends behind half a group of its four steps of 256 values.
__host__ __device__ inline bool mx_half_group(int stages, int K)
{
    const int filled = (K + 255) / 256;
    return stages == 2 && filled > 2 && (filled - 1) % 4 < 2;
}

}  // namespace qmoe
