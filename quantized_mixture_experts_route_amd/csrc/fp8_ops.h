// fp8_ops.h -- launch interface between fp8_ops.cpp (the C ABI of routing by
// scores, 8-bit floating point in blocks of 128 and the gated activation) and
// their kernels.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmoe {

// Routing by scores and its gradient (route_scores.hip).
struct RouteScoresArgs {
    const void* logits;         // T rows of E elements, row_stride apart
    int64_t row_stride;         // elements
    int64_t T;
    int E;
    int dtype;
    const float* bias;          // nullable: [E]
    int top_k;
    int sigmoid;                // else softmax
    int n_groups;
    int top_groups;
    int group_top;
    int group_size;  // E / n_groups
    int normalize;
    float scale;
    int32_t* ids;               // [T, top_k]: written forward, read backward
    float* weights;             // forward: [T, top_k]
    const float* grad_weights;  // backward: [T, top_k]
    void* grad_logits;          // backward: [T, E]
};
hipError_t launch_route_scores(const RouteScoresArgs& a, hipStream_t s);
hipError_t launch_route_scores_backward(const RouteScoresArgs& a, hipStream_t s);

constexpr int kFp8Block = 128;

// Conversion to and from e4m3 in blocks of 128 (fp8_convert.hip).
hipError_t launch_fp8_quantize(const void* x, int64_t row_stride, int64_t rows, int K, int dtype, uint8_t* codes,
                               float* scales, hipStream_t s);
hipError_t launch_fp8_quantize_weights(const void* x, int E, int rows, int K, int dtype, bool transpose,
                                       uint8_t* codes, float* scales, hipStream_t s);
// block_rows: 1, or 128 with `rows` the rows of one of E matrices.
hipError_t launch_fp8_dequantize(const uint8_t* codes, const float* scales, int E, int64_t rows, int K,
                                 int block_rows, int dtype, void* out, hipStream_t s);

// Grouped product (fp8_matmul.hip).
struct Fp8MatmulArgs {
    const uint8_t* a_codes;        // [a_rows, K]
    const float* a_scales;         // [a_rows, ceil(K/128)]
    int64_t a_rows;
    const uint8_t* w_codes;        // [E, N, K]
    const float* w_scales;         // [E, ceil(N/128), ceil(K/128)]
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
hipError_t launch_fp8_matmul(const Fp8MatmulArgs& a, hipStream_t s);

// The gated activation and its gradient (activate.hip).
struct ActivateArgs {
    const void* y;        // rows of 2 * I elements, row_stride apart
    int64_t row_stride;   // elements
    int64_t rows;
    int I;
    int dtype;
    int geglu;            // else SwiGLU
    int halves;           // gate j, up I + j; else gate 2j, up 2j + 1
    float alpha;
    float beta;
    float limit;
    void* out;            // [rows, I], or NULL with codes
    uint8_t* codes;       // [rows, I]
    float* scales;        // [rows, ceil(I/128)]
    const void* grad;     // backward: [rows, I], grad_stride apart
    int64_t grad_stride;  // elements
    void* grad_y;         // backward: [rows, 2 * I]
};
hipError_t launch_activate(const ActivateArgs& a, hipStream_t s);
hipError_t launch_activate_backward(const ActivateArgs& a, hipStream_t s);

}  // namespace qmoe
