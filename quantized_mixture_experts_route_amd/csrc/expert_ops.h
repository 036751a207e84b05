// expert_ops.h -- launch interface between expert_ops.cpp (the C ABI of the
// sort by expert and back and of the MXFP4 operators) and their kernels.
// Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmoe {

// Tokens sorted by expert (permute.hip).
struct PermuteArgs {
    const void* hidden;      // nullable (maps only): T rows of H elements, row_stride apart
    int64_t row_stride;      // elements
    int64_t T;
    int H;
    int elem;                // bytes per element (2 or 4)
    const int32_t* ids;      // [T * top_k]
    int top_k;
    int E;
    void* rows;              // nullable with hidden: [T * top_k, H]
    int32_t* offsets;        // [E + 1]
    int32_t* sorted_routes;  // [T * top_k]
    int32_t* route_rows;     // [T * top_k]
    int32_t* ws;             // permute_ws_ints() of them (unused where that is 0)
};

// int32 words of workspace launch_permute needs (0: one launch, no workspace).
int64_t permute_ws_ints(int64_t T, int top_k, int E);
hipError_t launch_permute(const PermuteArgs& a, hipStream_t s);

// Rows brought back to their tokens, and the gradient of that (permute.hip).
struct UnpermuteArgs {
    const void* rows;           // [T * top_k, H], row_stride apart
    int64_t row_stride;         // elements
    const int32_t* route_rows;  // [T, top_k]
    const float* weights;       // nullable (1): [T, top_k]
    int64_t T;
    int top_k;
    int H;
    int dtype;
    void* out;                  // forward: [T, H]
    const void* grad_out;       // backward: [T, H], grad_stride apart
    int64_t grad_stride;        // elements
    void* grad_rows;            // backward: [T * top_k, H]
    float* grad_weights;        // backward, nullable together with rows: [T, top_k]
};
hipError_t launch_unpermute(const UnpermuteArgs& a, hipStream_t s);
hipError_t launch_unpermute_backward(const UnpermuteArgs& a, hipStream_t s);

// MXFP4 conversion (mx_convert.hip).
hipError_t launch_mx_quantize(const void* x, int64_t row_stride, int64_t rows, int K, int dtype,
                              uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_mx_quantize_columns(const void* x, int E, int rows, int K, int dtype,
                                      uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t blocks,
                                int dtype, void* out, hipStream_t s);

// Grouped MXFP4 product (mx_matmul.hip).
struct MxMatmulArgs {
    const uint8_t* a_codes;        // [a_rows, K/2]
    const uint8_t* a_scales;       // [a_rows, K/32]
    int64_t a_rows;
    const uint8_t* w_codes;        // [E, N, K/2]
    const uint8_t* w_scales;       // [E, N, K/32]
    int E;
    int N;
    int K;
    const int32_t* offsets;        // nullable with E = 1: [E + 1]
    const int32_t* sorted_routes;  // nullable: [rows], a row = sorted_routes / top_k
    int top_k;
    int rows;
    int dtype;
    void* out;                     // [rows, N]
};
hipError_t launch_mx_matmul(const MxMatmulArgs& a, hipStream_t s);

// The calling thread's qmoe_last_error() becomes "" (qmoe_api.cpp).
void clear_error();

}  // namespace qmoe
