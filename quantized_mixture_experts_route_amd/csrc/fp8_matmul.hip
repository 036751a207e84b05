// fp8_matmul.hip -- grouped product of rows in 8-bit floating point (e4m3) with
// expert weights in the same format, with a float32 scale for each block of 128:
//   out[r, n] = sum_b sa(r, b) sw(e, n/128, b) sum_{k in block b} a(r, k) w(e, n, k)
// for the rows offsets[e] <= r < offsets[e+1] of expert e, rounded once to the
// output's type; rows behind the last expert's are zero.
//
// v_mfma_f32_16x16x128 on e4m3 operands: lane l = 16 g + c supplies row c of
// either operand and 32 values of the block of 128; which of them does not
// matter, as long as both operands take the same.  Register i of the result is
// row 4 g + i of the first operand and row c of the second.
//
// What the instruction rounds (measured on it): of each eight neighbouring products
// of a lane what lies below 2^-13 of the largest is cut off; their sums, 16 of a
// block, and the addend meet in float32.  On normal values that leaves 2e-5 of the
// result (2-norm), a hundredth of the rounding to 16 bits; outputs in float32 would
// need the operands as f16 at half the rate, and are refused.
#include "expert_tiles.h"
#include "fp8_ops.h"
#include "qmoe_internal.h"

namespace qmoe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
constexpr int kE4M3 = 0;  // operand format code of the matrix instructions

__device__ inline i32x8 operand(u32x4 a, u32x4 b)
{
    return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// A block's product on its own: the scales are applied to it in float32.
__device__ inline f32x4 block_product(i32x8 w, i32x8 x)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{}, kE4M3, kE4M3, 0, 0, 0, 0);
}

constexpr int kThreads = 256;

// A wavefront computes 16 rows against 16 weight rows, operands straight from memory.
template <int DT>
__global__ __launch_bounds__(kThreads) void simple_kernel(Fp8MatmulArgs a)
{
    typedef typename RowType<DT>::Raw Raw;
    constexpr int BM = 16, BN = 64;
    __shared__ int first[kMaxExperts + 1], scratch[kMaxExperts + 1];
    build_tile_list<BM, kThreads>(first, scratch, a.offsets, a.E, a.rows);
    const int n_tiles = (a.N + BN - 1) / BN;
    const int total = mx_items(first[a.E], n_tiles, a.rows, BM, a.E);
    if (a.offsets) {  // rows behind the last expert's are zero
        const int64_t lo = (int64_t)scratch[a.E] * a.N, hi = (int64_t)a.rows * a.N;
        for (int64_t i = lo + blockIdx.x * (int64_t)kThreads + threadIdx.x; i < hi; i += (int64_t)gridDim.x * kThreads) {
            ((Raw*)a.out)[i] = 0;
        }
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    const int blocks = (a.K + kFp8Block - 1) / kFp8Block, n_blocks = (a.N + kFp8Block - 1) / kFp8Block;
    for (int item = blockIdx.x; item < total; item += gridDim.x) {
        const TileItem t = item_at<BM, BN>(first, [&](int e) { return scratch[e]; }, a.E, n_tiles, item, total);
        const int n0 = t.n0 + wave * 16;
        if (n0 >= a.N) continue;
        const int r = t.row0 + min(c, t.n - 1);
        int64_t source = r;
        bool there = true;
        if (a.sorted_routes) {
            const int route = a.sorted_routes[r];
            there = route >= 0 && route / a.top_k < a.a_rows;
            source = there ? route / a.top_k : 0;
        }
        const uint8_t* x = a.a_codes + source * a.K;
        const uint8_t* w = a.w_codes + ((int64_t)t.expert * a.N + min(n0 + c, a.N - 1)) * a.K;
        const float* sa = a.a_scales + source * blocks;
        const float* sw = a.w_scales + ((int64_t)t.expert * n_blocks + n0 / kFp8Block) * blocks;
        f32x4 acc = {};
        for (int b = 0; b < blocks; ++b) {
            u32x4 vx[2] = {}, vw[2] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = b * kFp8Block + g * 32 + h * 16;
                if (k < a.K) {
                    if (there) vx[h] = *reinterpret_cast<const u32x4*>(x + k);
                    vw[h] = *reinterpret_cast<const u32x4*>(w + k);
                }
            }
            const f32x4 p = block_product(operand(vw[0], vw[1]), operand(vx[0], vx[1]));
            const float f = there ? sa[b] * sw[b] : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = fmaf(f, p[i], acc[i]);
        }
        if (c < t.n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = n0 + 4 * g + i;
                if (n < a.N) ((Raw*)a.out)[(int64_t)(t.row0 + c) * a.N + n] = RowType<DT>::round(acc[i]);
            }
        }
    }
}

}  // namespace

hipError_t launch_fp8_matmul(const Fp8MatmulArgs& a, hipStream_t s)
{
    const dim3 grid(8 * kMxCUs);
    if (a.dtype == kBF16) launch(simple_kernel<kBF16>, grid, dim3(kThreads), s, a);
    else launch(simple_kernel<kF16>, grid, dim3(kThreads), s, a);
    return hipGetLastError();
}

}  // namespace qmoe
