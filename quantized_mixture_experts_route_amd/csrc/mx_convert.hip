// mx_convert.hip -- conversion to and from microscaled 4-bit floating point
// (MXFP4): blocks of 32 values, each an e2m1 code (sign, 2 exponent bits,
// 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) times one
// power of two per block, stored as a byte with bias 127.
//
// Quantisation of a block with m = max |x|: the scale's exponent is
// floor(log2 m) - 2 (2 is e2m1's largest exponent), at least -127; a code is
// x / scale rounded to the nearest e2m1 value, ties to the even code, 6 at
// most.  A block holding a NaN or an infinity gets the scale byte 255, which
// stands for NaN, and codes 0.  The division by a power of two is an exact
// float32 product, so rounding to e2m1 is the only rounding.
//
// Both directions read and write every value once with a few operations per
// value: bound by HBM.  4096 x 4096 bf16 values out of cache: 10.5 us to codes
// (4.0 TB/s; 8.8 us where the cache holds them), 8.9 us back (4.8 TB/s); 8 x
// 2048 x 2048 f16 values to codes of the transposes 18.1 us (4.7 TB/s; 14.4).
#include "expert_ops.h"
#include "qmoe_internal.h"
#include "rowio.h"

namespace qmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 32;

// Scale byte of a block whose largest magnitude has the float32 bits `top`
// (NaN and infinities are the largest patterns).
__device__ inline uint32_t scale_byte(uint32_t top)
{
    const uint32_t e = top >> 23;
    return e == 255 ? 255 : e < 2 ? 0 : e - 2;
}

// 2^-(byte - 127) for a scale byte of a finite block (at most 252).
__device__ inline float inverse_scale(uint32_t byte)
{
    return __builtin_bit_cast(float, (254u - byte) << 23);
}

// 8 values over the scale -> 8 codes, value i at bits [4i, 4i + 4).
__device__ inline uint32_t encode8(const float* v, float inv)
{
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * inv, v[1] * inv, 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * inv, v[3] * inv, 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * inv, v[5] * inv, 1.0f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * inv, v[7] * inv, 1.0f, 3);
    return c;
}

__device__ inline uint32_t magnitude(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

// Eight values a thread, four threads a block; consecutive threads take
// consecutive eights, so loads and stores are whole lines.
template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const void* __restrict__ x, int64_t row_stride,
                                                           int64_t eights, int eights_per_row, int contiguous,
                                                           uint8_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales)
{
    typedef typename RowType<DT>::Raw Raw;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= eights) return;  // eights is a multiple of 4: a block's threads leave together
    int64_t at = i * 8;
    if (!contiguous) {
        const int64_t row = i / eights_per_row;
        at = row * row_stride + (i - row * eights_per_row) * 8;
    }
    const auto in = load_vec<Raw, 8>((const Raw*)x + at);
    float v[8];
    uint32_t top = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        v[q] = RowType<DT>::value(in.v[q]);
        top = max(top, magnitude(v[q]));
    }
    top = max(top, dpp_u32<kDppXor1>(top));
    top = max(top, dpp_u32<kDppXor2>(top));
    const uint32_t byte = scale_byte(top);
    const uint32_t c = byte == 255 ? 0u : encode8(v, inverse_scale(byte));
    reinterpret_cast<uint32_t*>(codes)[i] = c;
    if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
}

// Blocks along the rows of x [E, rows, K]; codes [E, K, rows/2], scales
// [E, K, rows/32].  A workgroup takes 64 columns and 256 rows: each of its 8
// wavefronts reads 32 rows of 64 neighbouring values, a lane one column's block.
// The codes pass through LDS, so that a column's 128 bytes leave as one line
// (8192 x 8192 float32 values 63 us, 4.8 TB/s; with 16 bytes a lane straight
// from the registers 74 us).
constexpr int kColumns = 64;
constexpr int kColumnBlocks = 8;
template <int DT>
__global__ __launch_bounds__(64 * kColumnBlocks) void quantize_columns_kernel(const void* __restrict__ x, int rows,
                                                                             int K, uint8_t* __restrict__ codes,
                                                                             uint8_t* __restrict__ scales)
{
    typedef typename RowType<DT>::Raw Raw;
    __shared__ u32x4 staged[kColumns][kColumnBlocks + 1];  // one spare: columns start in different banks
    __shared__ uint8_t staged_scale[kColumns][kColumnBlocks];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int k0 = blockIdx.x * kColumns, block0 = blockIdx.y * kColumnBlocks;
    const int64_t e = blockIdx.z;
    const int blocks = rows / kBlock;
    const int k = k0 + lane, block = block0 + wave;
    if (k < K && block < blocks) {
        const Raw* p = (const Raw*)x + (e * rows + block * kBlock) * (int64_t)K + k;
        Raw in[kBlock];
        uint32_t top = 0;
#pragma unroll
        for (int r = 0; r < kBlock; ++r) in[r] = p[(int64_t)r * K];
#pragma unroll
        for (int r = 0; r < kBlock; ++r) top = max(top, magnitude(RowType<DT>::value(in[r])));
        const uint32_t byte = scale_byte(top);
        const float inv = inverse_scale(byte);
        u32x4 c;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) v[r] = RowType<DT>::value(in[8 * q + r]);
            c[q] = byte == 255 ? 0u : encode8(v, inv);
        }
        staged[lane][wave] = c;
        staged_scale[lane][wave] = (uint8_t)byte;
    }
    __syncthreads();
    const int column = threadIdx.x / kColumnBlocks, part = threadIdx.x % kColumnBlocks;
    if (k0 + column < K && block0 + part < blocks) {
        const int64_t at = (e * K + k0 + column) * (int64_t)blocks + block0 + part;
        reinterpret_cast<u32x4*>(codes)[at] = staged[column][part];
        scales[at] = staged_scale[column][part];
    }
}

// Eight codes a thread.  value * 2^(byte - 127) is exact in float32 down to
// its subnormals; storing it to 16 bits rounds once.
template <int DT>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales,
                                                             int64_t eights, void* __restrict__ out)
{
    typedef typename RowType<DT>::Raw Raw;
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= eights) return;
    const uint32_t c = reinterpret_cast<const uint32_t*>(codes)[i];
    const uint32_t byte = scales[i >> 2];
    const float scale = byte == 255 ? __builtin_nanf("") : __builtin_bit_cast(float, byte == 0 ? 0x00400000u : byte << 23);
    const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3)};
    RowVec<Raw, 8> y;
#pragma unroll
    for (int q = 0; q < 8; ++q) y.v[q] = RowType<DT>::round(p[q >> 1][q & 1] * scale);
    store_vec<Raw, 8>((Raw*)out + i * 8, y);
}

unsigned blocks_for(int64_t n) { return (unsigned)((n + kThreads - 1) / kThreads); }

}  // namespace

hipError_t launch_mx_quantize(const void* x, int64_t row_stride, int64_t rows, int K, int dtype,
                              uint8_t* codes, uint8_t* scales, hipStream_t s)
{
    const int64_t eights = rows * (K / 8);
    auto go = [&](auto kernel) {
        launch(kernel, dim3(blocks_for(eights)), dim3(kThreads), s, x, row_stride, eights, K / 8,
               (int)(row_stride == K), codes, scales);
    };
    if (dtype == kF32) go(quantize_kernel<kF32>);
    else if (dtype == kBF16) go(quantize_kernel<kBF16>);
    else go(quantize_kernel<kF16>);
    return hipGetLastError();
}

hipError_t launch_mx_quantize_columns(const void* x, int E, int rows, int K, int dtype, uint8_t* codes,
                                      uint8_t* scales, hipStream_t s)
{
    const dim3 grid((unsigned)((K + kColumns - 1) / kColumns),
                    (unsigned)((rows / kBlock + kColumnBlocks - 1) / kColumnBlocks), (unsigned)E);
    auto go = [&](auto kernel) { launch(kernel, grid, dim3(64 * kColumnBlocks), s, x, rows, K, codes, scales); };
    if (dtype == kF32) go(quantize_columns_kernel<kF32>);
    else if (dtype == kBF16) go(quantize_columns_kernel<kBF16>);
    else go(quantize_columns_kernel<kF16>);
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t blocks, int dtype,
                                void* out, hipStream_t s)
{
    const int64_t eights = blocks * 4;
    auto go = [&](auto kernel) { launch(kernel, dim3(blocks_for(eights)), dim3(kThreads), s, codes, scales, eights, out); };
    if (dtype == kF32) go(dequantize_kernel<kF32>);
    else if (dtype == kBF16) go(dequantize_kernel<kBF16>);
    else go(dequantize_kernel<kF16>);
    return hipGetLastError();
}

}  // namespace qmoe
