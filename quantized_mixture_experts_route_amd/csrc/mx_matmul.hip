// mx_matmul.hip -- grouped product of MXFP4 rows with MXFP4 expert weights:
//   out[r, n] = sum_b 2^(sa(r,b) + sw(e,n,b) - 254) sum_{i in block b} a(r,i) w(e,n,i)
// for the rows offsets[e] <= r < offsets[e+1] of expert e, accumulated in
// float32 on the scaled matrix instruction and rounded once to the output's
// type; rows behind the last expert's are zero.
//
// v_mfma_scale_f32_32x32x64 with e2m1 operands: lane l = 32 h + c supplies
// row c of A and row c of W, each one block of 32 codes (16 bytes) with its
// scale byte; the lane half h is the block of the two that the step contracts.
// The result: register i of lane l is row 8 (i/4) + 4 h + i%4, column c.
#include "expert_ops.h"
#include "qmoe_internal.h"
#include "rowio.h"

namespace qmoe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr int kE2M1 = 4;  // operand format code of the scaled matrix instructions

__device__ inline i32x8 operand(u32x4 v)
{
    return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

// A row tile of one expert: rows [row0, row0 + n) of the product.
struct RowTile {
    int expert;  // E: the rows behind the last expert's
    int row0;
    int n;
};

// Tile `index` of the list that cuts every expert's rows, and then the rows
// behind them, into tiles of MT rows; n = 0 past the list's end.  Offsets are
// clamped to [0, rows], so no table content leads outside the output.
template <int MT>
__device__ RowTile find_tile(const int32_t* offsets, int E, int rows, int index)
{
    int left = index;
    if (offsets == nullptr) {
        const int row0 = left * MT;
        return RowTile{0, row0, row0 < rows ? min(MT, rows - row0) : 0};
    }
    int at = 0;
    for (int e = 0; e <= E; ++e) {
        const int lo = min(max(offsets[e], 0), rows);
        const int hi = e < E ? min(max(offsets[e + 1], lo), rows) : rows;
        const int tiles = (hi - lo + MT - 1) / MT;
        if (left < tiles) {
            at = lo + left * MT;
            return RowTile{e, at, min(MT, hi - at)};
        }
        left -= tiles;
    }
    return RowTile{E, 0, 0};
}

// One wavefront computes 32 rows x 32 columns with operands straight from
// global memory; four wavefronts take neighbouring column blocks.
template <int DT>
__global__ __launch_bounds__(256) void product_kernel(MxMatmulArgs a)
{
    typedef typename RowType<DT>::Raw Raw;
    const RowTile tile = find_tile<32>(a.offsets, a.E, a.rows, blockIdx.x);
    if (tile.n <= 0) return;
    const int lane = threadIdx.x & 63, c = lane & 31, half = lane >> 5;
    const int n0 = (blockIdx.y * 4 + (threadIdx.x >> 6)) * 32;
    if (n0 >= a.N) return;
    const int row = tile.row0 + min(c, tile.n - 1);
    const int col = min(n0 + c, a.N - 1);
    const int route = a.sorted_routes ? a.sorted_routes[row] : row;
    const int64_t src = a.sorted_routes ? route / a.top_k : route;
    const bool row_ok = route >= 0 && src < a.a_rows;
    const int blocks = a.K / 32;
    f32x16 acc = {};
    if (tile.expert < a.E) {
        const uint8_t* ac = a.a_codes + (row_ok ? src : 0) * (int64_t)(a.K / 2);
        const uint8_t* as = a.a_scales + (row_ok ? src : 0) * (int64_t)blocks;
        const int64_t wrow = (int64_t)tile.expert * a.N + col;
        const uint8_t* wc = a.w_codes + wrow * (a.K / 2);
        const uint8_t* ws = a.w_scales + wrow * blocks;
        for (int b = half; b < blocks + half; b += 2) {
            u32x4 x = {}, w = {};
            int sx = 0, sw = 0;
            if (b < blocks) {
                x = *reinterpret_cast<const u32x4*>(ac + b * 16);
                w = *reinterpret_cast<const u32x4*>(wc + b * 16);
                sx = as[b];
                sw = ws[b];
            }
            acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(x), operand(w), acc, kE2M1, kE2M1, 0, sx, 0, sw);
        }
    }
    const uint64_t ok = __ballot(row_ok);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = 8 * (i / 4) + 4 * half + i % 4;
        if (r < tile.n && n0 + c < a.N) {
            ((Raw*)a.out)[(int64_t)(tile.row0 + r) * a.N + n0 + c] =
                RowType<DT>::round((ok >> r) & 1 ? acc[i] : 0.0f);
        }
    }
}

}  // namespace

hipError_t launch_mx_matmul(const MxMatmulArgs& a, hipStream_t s)
{
    // one partial tile at most for every expert with rows and for the rows behind
    const int64_t groups = a.offsets ? (a.E + 1 < a.rows ? a.E + 1 : a.rows) : 1;
    const int64_t tiles = (a.rows + 31) / 32 + groups;
    const dim3 grid((unsigned)tiles, (unsigned)((a.N + 127) / 128));
    if (a.dtype == kF32) launch(product_kernel<kF32>, grid, dim3(256), s, a);
    else if (a.dtype == kBF16) launch(product_kernel<kBF16>, grid, dim3(256), s, a);
    else launch(product_kernel<kF16>, grid, dim3(256), s, a);
    return hipGetLastError();
}

}  // namespace qmoe
