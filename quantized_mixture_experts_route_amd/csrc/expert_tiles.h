// expert_tiles.h -- tiles of a grouped product over the rows of each expert:
// the list of m-tiles that a table of offsets makes, and the tile of an item.
// Shared by the grouped products (mx_matmul.hip, fp8_matmul.hip).
#pragma once

#include "mx_shape.h"
#include "qmoe_device.h"
#include "rowio.h"

namespace qmoe {

constexpr int kMaxExperts = 1024;

template <int DT>
__device__ inline uint32_t pack_pair(float lo, float hi)
{
    if constexpr (DT == kBF16) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
    } else {
        return pack2(Dt<kF16>::from_float(lo), Dt<kF16>::from_float(hi));
    }
}

// Stores 16 rows of 32 columns of 16-bit values: lane l's v holds the eight columns from
// 8 (l / 32) + 16 (l / 16 % 2) on of row l % 16.  `out` is the first row and column; rows and cols say how
// many of them exist (WHOLE: all).
template <bool WHOLE>
__device__ inline void store_sixteen(uint16_t* out, int N, int rows, int cols, u32x4 v, int lane)
{
    const int row = lane & 15, col = 8 * (lane >> 5) + 16 * ((lane >> 4) & 1);
    uint16_t* p = out + (int64_t)row * N + col;
    if (WHOLE && (((uintptr_t)out | (uintptr_t)N << 1) & 2)) {
        // rows that start between two words: they are stored one column on, in whole words, with
        // the first column of the neighbour's eight at the end; columns 0 and 31 on their own
        // (MXFP4, 18498 rows of 2175 columns: 90 us, with 16-byte stores that split words 105)
        const uint32_t next = (uint32_t)__shfl((int)v[0], lane < 32 ? lane + 32 : lane - 16, kWave);
        const bool odd = (uintptr_t)p & 2;
        if (odd) {
            if (col == 0) p[0] = (uint16_t)v[0];
            if (col == 24) p[7] = (uint16_t)(v[3] >> 16);
            v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16 | next << 16};
        }
        __builtin_memcpy(p + odd, &v, 12);
        if (!odd || col < 24) __builtin_memcpy(p + odd + 6, (const char*)&v + 12, 4);
        return;
    }
    if (!WHOLE && row >= rows) return;
    if (WHOLE || col + 8 <= cols) {
        __builtin_memcpy(p, &v, 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (col + i < cols) p[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// m-tiles of each expert in LDS: first[e] .. first[e + 1] of the tile list.
// Offsets are clamped to [0, rows] and mx_items() bounds the count, so no table
// content leads outside the output.  scratch: E + 1 words of LDS.
template <int BM, int THREADS>
__device__ void build_tile_list(int* first, int* scratch, const int32_t* offsets, int E, int rows)
{
    for (int e = threadIdx.x; e <= E; e += THREADS) {
        scratch[e] = offsets ? min(max(offsets[e], 0), rows) : e * rows;
    }
    __syncthreads();
    if (threadIdx.x < kWave) {
        const int lane = threadIdx.x, per = (E + kWave - 1) / kWave;  // consecutive experts a lane
        auto tiles = [&](int e) { return e < E ? (max(scratch[e + 1] - scratch[e], 0) + BM - 1) / BM : 0; };
        int sum = 0;
        for (int i = 0; i < per; ++i) sum += tiles(lane * per + i);
        int incl = sum;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int y = __shfl_up(incl, d, kWave);
            if (lane >= d) incl += y;
        }
        int run = incl - sum;
        for (int i = 0; i < per; ++i) {
            const int e = lane * per + i;
            if (e < E) first[e] = run;
            run += tiles(e);
        }
        if (lane == kWave - 1) first[E] = run;
    }
    __syncthreads();
}

// Reads through it are scalar and wait for no vector memory; what it points to does not change
// while the kernel runs.
__device__ inline const __attribute__((address_space(4))) int32_t* constant(const int32_t* p)
{
    return (const __attribute__((address_space(4))) int32_t*)p;
}

// The workgroups that run on a die at a time (32 of the largest tile) share rows and weights in its
// L2: bands of 8 m-tiles make that about 8 row blocks and 4 weight blocks, in place of one column of
// 32 (8192^3: 281 -> 246 us; bands of 4 and of 12 were slower).
constexpr int kBand = 8;

struct TileItem {
    int expert;
    int row0;
    int n;   // rows; 0: no item
    int n0;  // first column
};

// offset(e) gives expert e's clamped offset.
template <int BM, int BN, class Offset>
__device__ TileItem item_at(const int* first, Offset offset, int E, int n_tiles, int item, int end)
{
    if (item >= end) return TileItem{0, 0, 0, 0};
    int lo = 0, hi = E - 1;  // the last expert whose first item is <= item
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] * n_tiles <= item) lo = mid; else hi = mid - 1;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    const int base = __builtin_amdgcn_readfirstlane(first[lo]);
    const int m_tiles = __builtin_amdgcn_readfirstlane(first[lo + 1]) - base;
    // bands of up to kBand m-tiles, in a band neighbouring items share the weights
    int local = item - base * n_tiles;
    int m0 = 0, band = m_tiles;
    if (m_tiles > kBand) {
        const int bands = (m_tiles + kBand - 1) / kBand;
        band = (m_tiles + bands - 1) / bands;
        m0 = local / (band * n_tiles) * band;
        local -= m0 * n_tiles;
        band = min(band, m_tiles - m0);
    }
    const int nt = local / band;
    const int r_lo = offset(lo), r_hi = offset(lo + 1);
    const int row0 = r_lo + (m0 + local - nt * band) * BM;
    return TileItem{lo, row0, min(BM, r_hi - row0), nt * BN};
}

}  // namespace qmoe
