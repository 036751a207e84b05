// fp8_convert.hip -- conversion to and from 8-bit floating point (e4m3) with a
// float32 scale for each block of 128 values of a row, or for each square of
// 128 x 128 of a matrix (weights; then the transposed matrix has the same codes
// and scales at their transposed places).  fp8_block.h defines scale and code.
//
// Every value is read and written once with a few operations: bound by HBM, of which a copy reaches 5.1 TB/s (out
// of the cache: 4096 x 4096 bf16 to codes 12.7 us, 4.0 TB/s, and back 11.2, 4.5 TB/s; 4096 x 4096 f32 to codes and
// back 30 us, 5.6 TB/s; 8 matrices of 2048 x 2048 f16, transposed, 24 us, 4.2 TB/s).
#include <algorithm>

#include "fp8_block.h"
#include "qmoe_internal.h"

namespace qmoe {
namespace {

constexpr int kThreads = 256;

// Eight values a thread, 16 threads a block; consecutive threads take consecutive eights, so loads and
// stores are whole lines.  blocks: of a row.
template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const void* __restrict__ x, int64_t row_stride,
                                                           int64_t threads, int blocks, int K,
                                                           uint8_t* __restrict__ codes, float* __restrict__ scales)
{
    typedef typename RowType<DT>::Raw Raw;
    // a multiple of 16: a block's threads stay together
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < threads; i += (int64_t)gridDim.x * kThreads) {
        const int64_t block = i >> 4, row = block / blocks;
        const int k = (int)(block - row * blocks) * kFp8Block + (int)(i & 15) * 8;
        const bool in = k < K;
        float v[8] = {};
        if (in) {
            const auto raw = load_vec<Raw, 8>((const Raw*)x + row * row_stride + k);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = RowType<DT>::value(raw.v[q]);
        }
        fp8_store_block(v, in, codes + row * K + k, scales + block);
    }
}

// One square a workgroup, so that its maximum is one exchange of four words and no value is read again: thread (r, c)
// of 16 x 16 holds rows 8 r .. 8 r + 7, columns 8 c .. 8 c + 7.
// Transposed, the codes pass through LDS, so that a column's 128 bytes leave as one line.
template <int DT, bool TRANSPOSE>
__global__ __launch_bounds__(kThreads) void quantize_squares_kernel(const void* __restrict__ x, int rows, int K,
                                                                   uint8_t* __restrict__ codes,
                                                                   float* __restrict__ scales)
{
    typedef typename RowType<DT>::Raw Raw;
    constexpr int kPitch = kFp8Block + 16;
    __shared__ uint32_t tops[kThreads / kWave];
    __shared__ __align__(16) uint8_t staged[TRANSPOSE ? kFp8Block * kPitch : 16];
    const int64_t e = blockIdx.z;
    const int r0 = blockIdx.y * kFp8Block + (threadIdx.x >> 4) * 8, k0 = blockIdx.x * kFp8Block + (threadIdx.x & 15) * 8;
    const Raw* p = (const Raw*)x + (e * rows + r0) * (int64_t)K + k0;
    float v[8][8];  // [row][column]
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        if (r0 + r < rows && k0 + 8 <= K) {
            const auto raw = load_vec<Raw, 8>(p + (int64_t)r * K);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[r][q] = RowType<DT>::value(raw.v[q]);
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                v[r][q] = r0 + r < rows && k0 + q < K ? RowType<DT>::value(p[(int64_t)r * K + q]) : 0.0f;
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) top = max(top, magnitude_bits(v[r][q]));
    }
    top = wave_max_u32(top);
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    const uint32_t bits = fp8_scale_bits(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
    const bool finite = bits != 0x7fc00000u;
    const float inv = fp8_inverse(bits);
    const int row_blocks = (rows + kFp8Block - 1) / kFp8Block, k_blocks = (K + kFp8Block - 1) / kFp8Block;
    if constexpr (!TRANSPOSE) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const u32x2 c = finite ? u32x2{fp8_encode4(v[r], inv), fp8_encode4(v[r] + 4, inv)} : u32x2{};
            // K is a multiple of 16: eight columns lie inside or outside together
            if (r0 + r < rows && k0 < K) *reinterpret_cast<u32x2*>(codes + (e * rows + r0 + r) * (int64_t)K + k0) = c;
        }
        if (threadIdx.x == 0) {
            scales[(e * row_blocks + blockIdx.y) * k_blocks + blockIdx.x] = __builtin_bit_cast(float, bits);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float column[8] = {v[0][q], v[1][q], v[2][q], v[3][q], v[4][q], v[5][q], v[6][q], v[7][q]};
            const u32x2 c = finite ? u32x2{fp8_encode4(column, inv), fp8_encode4(column + 4, inv)} : u32x2{};
            *reinterpret_cast<u32x2*>(staged + ((threadIdx.x & 15) * 8 + q) * kPitch + (threadIdx.x >> 4) * 8) = c;
        }
        __syncthreads();
        const int part = (threadIdx.x & 7) * 16;  // 16 rows of x, of one column
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int column = j * 32 + (threadIdx.x >> 3);
            const int64_t k = blockIdx.x * kFp8Block + column;
            const int r = blockIdx.y * kFp8Block + part;
            // rows is a multiple of 16
            if (k < K && r < rows) {
                *reinterpret_cast<u32x4*>(codes + (e * K + k) * (int64_t)rows + r) =
                    *reinterpret_cast<const u32x4*>(staged + column * kPitch + part);
            }
        }
        if (threadIdx.x == 0) {
            scales[(e * k_blocks + blockIdx.x) * row_blocks + blockIdx.y] = __builtin_bit_cast(float, bits);
        }
    }
}

// Eight codes a thread.  code * scale is rounded to float32 (exact for a power of two) and to the type.
template <int DT>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t* __restrict__ codes,
                                                             const float* __restrict__ scales, int64_t eights,
                                                             int eights_per_row, int blocks, int64_t rows,
                                                             int block_rows, void* __restrict__ out)
{
    typedef typename RowType<DT>::Raw Raw;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < eights; i += (int64_t)gridDim.x * kThreads) {
        const int64_t row = i / eights_per_row;
        const int block = (int)(i - row * eights_per_row) >> 4;
        int64_t scale_row = row;
        if (block_rows != 1) {
            const int64_t e = row / rows, row_blocks = (rows + block_rows - 1) / block_rows;
            scale_row = e * row_blocks + (row - e * rows) / block_rows;
        }
        const u32x2 c = reinterpret_cast<const u32x2*>(codes)[i];
        const float scale = scales[scale_row * blocks + block];
        RowVec<Raw, 8> y;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], true);
            y.v[4 * h] = RowType<DT>::round(lo[0] * scale);
            y.v[4 * h + 1] = RowType<DT>::round(lo[1] * scale);
            y.v[4 * h + 2] = RowType<DT>::round(hi[0] * scale);
            y.v[4 * h + 3] = RowType<DT>::round(hi[1] * scale);
        }
        store_vec<Raw, 8>((Raw*)out + i * 8, y);
    }
}

// A launch has fewer than 2^32 threads; those of more run through several items.
unsigned blocks_for(int64_t n) { return (unsigned)std::min((n + kThreads - 1) / kThreads, int64_t(1) << 23); }

int block_count(int n) { return (n + kFp8Block - 1) / kFp8Block; }

}  // namespace

hipError_t launch_fp8_quantize(const void* x, int64_t row_stride, int64_t rows, int K, int dtype, uint8_t* codes,
                               float* scales, hipStream_t s)
{
    const int64_t threads = rows * block_count(K) * 16;
    auto go = [&](auto kernel) {
        launch(kernel, dim3(blocks_for(threads)), dim3(kThreads), s, x, row_stride, threads, block_count(K), K, codes,
               scales);
    };
    if (dtype == kF32) go(quantize_kernel<kF32>);
    else if (dtype == kBF16) go(quantize_kernel<kBF16>);
    else go(quantize_kernel<kF16>);
    return hipGetLastError();
}

hipError_t launch_fp8_quantize_weights(const void* x, int E, int rows, int K, int dtype, bool transpose, uint8_t* codes,
                                       float* scales, hipStream_t s)
{
    const dim3 grid((unsigned)block_count(K), (unsigned)block_count(rows), (unsigned)E);
    auto go = [&](auto kernel) { launch(kernel, grid, dim3(kThreads), s, x, rows, K, codes, scales); };
    if (transpose) {
        if (dtype == kF32) go(quantize_squares_kernel<kF32, true>);
        else if (dtype == kBF16) go(quantize_squares_kernel<kBF16, true>);
        else go(quantize_squares_kernel<kF16, true>);
    } else {
        if (dtype == kF32) go(quantize_squares_kernel<kF32, false>);
        else if (dtype == kBF16) go(quantize_squares_kernel<kBF16, false>);
        else go(quantize_squares_kernel<kF16, false>);
    }
    return hipGetLastError();
}

hipError_t launch_fp8_dequantize(const uint8_t* codes, const float* scales, int E, int64_t rows, int K, int block_rows,
                                 int dtype, void* out, hipStream_t s)
{
    const int64_t eights = E * rows * (K / 8);
    auto go = [&](auto kernel) {
        launch(kernel, dim3(blocks_for(eights)), dim3(kThreads), s, codes, scales, eights, K / 8, block_count(K), rows,
               block_rows, out);
    };
    if (dtype == kF32) go(dequantize_kernel<kF32>);
    else if (dtype == kBF16) go(dequantize_kernel<kBF16>);
    else go(dequantize_kernel<kF16>);
    return hipGetLastError();
}

}  // namespace qmoe
