// fp8_ops.cpp -- the C ABI of routing by scores, 8-bit floating point in blocks
// of 128 with its grouped product, and the gated activation: argument checks
// and launches.  Every check runs before the first launch, so an error return
// leaves the stream and all outputs untouched.
#include <hip/hip_runtime.h>

#include <cmath>

#include "abi_checks.h"
#include "fp8_ops.h"
#include "mx_shape.h"
#include "qmoe.h"

namespace {

using namespace qmoe::abi;

constexpr int kMaxSlots = 64;   // a wavefront's lanes: top_k and n_groups of the choice by scores
constexpr int kMaxRowsEach = 1 << 24;

int check_fp8(const char* name, const uint8_t* codes, const float* scales)
{
    if (!codes || !scales) return set_error(QMOE_ERR_INVALID_ARG, "%s codes/scales is NULL", name);
    if (!aligned(codes, 16)) return set_error(QMOE_ERR_INVALID_ARG, "%s codes not 16-byte aligned", name);
    if (!aligned(scales, 4)) return set_error(QMOE_ERR_INVALID_ARG, "%s scales not 4-byte aligned", name);
    return QMOE_OK;
}

int check_sixteens(const char* name, int32_t n)
{
    if (n % 16) return set_error(QMOE_ERR_UNSUPPORTED, "%s=%d must be a multiple of 16", name, n);
    return QMOE_OK;
}

int check_values(int64_t rows, int32_t K)
{
    if (K > kMaxWidth) return set_error(QMOE_ERR_UNSUPPORTED, "K=%d must be at most 2^20", K);
    if (rows > kMaxValues / K) return set_error(QMOE_ERR_UNSUPPORTED, "rows*K must be at most 2^34");
    return QMOE_OK;
}

int check_scores(int64_t T, int32_t E, int32_t dtype, int32_t top_k, int32_t score, float scale)
{
    if (T < 0) return set_error(QMOE_ERR_INVALID_ARG, "T=%lld < 0", (long long)T);
    if (T > kMaxTokens) return set_error(QMOE_ERR_UNSUPPORTED, "T=%lld must be below 2^23", (long long)T);
    if (E < 1 || E > kMaxExperts) return set_error(QMOE_ERR_INVALID_ARG, "E=%d outside [1, %d]", E, kMaxExperts);
    QMOE_TRY(check_dtype(dtype));
    if (top_k < 1 || top_k > E) return set_error(QMOE_ERR_INVALID_ARG, "top_k=%d outside [1, E=%d]", top_k, E);
    if (top_k > kMaxSlots) return set_error(QMOE_ERR_UNSUPPORTED, "top_k=%d must be at most %d", top_k, kMaxSlots);
    if (score != QMOE_SCORE_SOFTMAX && score != QMOE_SCORE_SIGMOID) {
        return set_error(QMOE_ERR_INVALID_ARG, "score=%d is neither softmax (0) nor sigmoid (1)", score);
    }
    if (!std::isfinite(scale)) return set_error(QMOE_ERR_INVALID_ARG, "scale must be finite");
    return QMOE_OK;
}

int check_activation(int64_t rows, int32_t I, int32_t dtype, int32_t activation, int32_t fusion, float alpha,
                     float beta, float limit)
{
    if (rows < 0) return set_error(QMOE_ERR_INVALID_ARG, "rows=%lld < 0", (long long)rows);
    if (I < 1) return set_error(QMOE_ERR_INVALID_ARG, "I=%d must be >= 1", I);
    QMOE_TRY(check_dtype(dtype));
    if (activation != QMOE_ACT_SWIGLU && activation != QMOE_ACT_GEGLU) {
        return set_error(QMOE_ERR_INVALID_ARG, "activation=%d is neither SwiGLU (0) nor GeGLU (1)", activation);
    }
    if (fusion != QMOE_SWIGLU_INTERLEAVED && fusion != QMOE_SWIGLU_HALVES) {
        return set_error(QMOE_ERR_INVALID_ARG, "swiglu_fusion=%d is neither interleaved (1) nor halves (2)", fusion);
    }
    if (std::isnan(alpha) || std::isnan(beta) || !(limit > 0)) {
        return set_error(QMOE_ERR_INVALID_ARG, "activation_alpha or _beta is NaN, or swiglu_limit is not positive");
    }
    if (I > kMaxWidth / 2) return set_error(QMOE_ERR_UNSUPPORTED, "I=%d must be at most 2^19", I);
    if (rows > kMaxValues / I) return set_error(QMOE_ERR_UNSUPPORTED, "rows*I must be at most 2^34");
    return QMOE_OK;
}

qmoe::ActivateArgs activate_args(const void* y, int64_t row_stride, int64_t rows, int32_t I, int32_t dtype,
                                 int32_t activation, int32_t fusion, float alpha, float beta, float limit)
{
    qmoe::ActivateArgs a{};
    a.y = y;
    a.row_stride = row_stride;
    a.rows = rows;
    a.I = I;
    a.dtype = dtype;
    a.geglu = activation == QMOE_ACT_GEGLU;
    a.halves = fusion == QMOE_SWIGLU_HALVES;
    a.alpha = alpha;
    a.beta = beta;
    a.limit = limit;
    return a;
}

}  // namespace

extern "C" {

int qmoe_route_scores(const void* logits, int64_t row_stride, int64_t T, int32_t E, int32_t dtype, const float* bias,
                      int32_t top_k, int32_t score, int32_t n_groups, int32_t top_groups, int32_t group_top,
                      int32_t normalize, float scale, int32_t* ids, float* weights, void* stream)
{
    QMOE_TRY(check_scores(T, E, dtype, top_k, score, scale));
    if (n_groups < 1 || E % n_groups) {
        return set_error(QMOE_ERR_INVALID_ARG, "n_groups=%d does not divide E=%d", n_groups, E);
    }
    if (n_groups > kMaxSlots) {
        return set_error(QMOE_ERR_UNSUPPORTED, "n_groups=%d must be at most %d", n_groups, kMaxSlots);
    }
    if (top_groups < 1 || top_groups > n_groups) {
        return set_error(QMOE_ERR_INVALID_ARG, "top_groups=%d outside [1, n_groups=%d]", top_groups, n_groups);
    }
    if (group_top != 1 && group_top != 2) return set_error(QMOE_ERR_INVALID_ARG, "group_top=%d is neither 1 nor 2", group_top);
    if (top_k > E / n_groups * top_groups) {
        return set_error(QMOE_ERR_INVALID_ARG, "top_k=%d exceeds the %d experts of top_groups=%d groups", top_k,
                         E / n_groups * top_groups, top_groups);
    }
    if (T == 0) return finish(hipSuccess, "");
    QMOE_TRY(check_rows("logits", logits, T, row_stride, E, elem_bytes(dtype)));
    if (bias) QMOE_TRY(check_words("bias", bias));
    QMOE_TRY(check_words("ids", ids));
    QMOE_TRY(check_words("weights", weights));
    qmoe::RouteScoresArgs a{};
    a.logits = logits;
    a.row_stride = row_stride;
    a.T = T;
    a.E = E;
    a.dtype = dtype;
    a.bias = bias;
    a.top_k = top_k;
    a.sigmoid = score == QMOE_SCORE_SIGMOID;
    a.n_groups = n_groups;
    a.top_groups = top_groups;
    a.group_top = group_top;
    a.group_size = E / n_groups;
    a.normalize = normalize != 0;
    a.scale = scale;
    a.ids = ids;
    a.weights = weights;
    return finish(qmoe::launch_route_scores(a, (hipStream_t)stream), "route_scores launch");
}

int qmoe_route_scores_backward(const float* grad_weights, const void* logits, int64_t row_stride, const int32_t* ids,
                               int64_t T, int32_t E, int32_t dtype, int32_t top_k, int32_t score, int32_t normalize,
                               float scale, void* grad_logits, void* stream)
{
    QMOE_TRY(check_scores(T, E, dtype, top_k, score, scale));
    if (T == 0) return finish(hipSuccess, "");
    QMOE_TRY(check_words("grad_weights", grad_weights));
    QMOE_TRY(check_rows("logits", logits, T, row_stride, E, elem_bytes(dtype)));
    QMOE_TRY(check_words("ids", ids));
    QMOE_TRY(check_rows("grad_logits", grad_logits, T, E, E, elem_bytes(dtype)));
    qmoe::RouteScoresArgs a{};
    a.logits = logits;
    a.row_stride = row_stride;
    a.T = T;
    a.E = E;
    a.dtype = dtype;
    a.top_k = top_k;
    a.sigmoid = score == QMOE_SCORE_SIGMOID;
    a.normalize = normalize != 0;
    a.scale = scale;
    a.ids = const_cast<int32_t*>(ids);
    a.grad_weights = grad_weights;
    a.grad_logits = grad_logits;
    return finish(qmoe::launch_route_scores_backward(a, (hipStream_t)stream), "route_scores_backward launch");
}

int qmoe_blocks_quantize(const void* x, int64_t row_stride, int64_t rows, int32_t K, int32_t dtype, uint8_t* codes,
                      float* scales, void* stream)
{
    if (rows < 0 || K < 1) return set_error(QMOE_ERR_INVALID_ARG, "rows=%lld, K=%d", (long long)rows, K);
    QMOE_TRY(check_dtype(dtype));
    QMOE_TRY(check_sixteens("K", K));
    QMOE_TRY(check_values(rows, K));
    if (rows == 0) return finish(hipSuccess, "");
    QMOE_TRY(check_rows("x", x, rows, row_stride, K, elem_bytes(dtype)));
    QMOE_TRY(check_fp8("output", codes, scales));
    return finish(qmoe::launch_fp8_quantize(x, row_stride, rows, K, dtype, codes, scales, (hipStream_t)stream),
                  "fp8_quantize launch");
}

int qmoe_blocks_quantize_weights(const void* x, int32_t E, int32_t rows, int32_t K, int32_t dtype, int32_t transpose,
                              uint8_t* codes, float* scales, void* stream)
{
    if (E < 0 || rows < 1 || K < 1) return set_error(QMOE_ERR_INVALID_ARG, "E=%d, rows=%d, K=%d", E, rows, K);
    QMOE_TRY(check_dtype(dtype));
    QMOE_TRY(transpose ? check_sixteens("rows", rows) : check_sixteens("K", K));
    if (E > 65535 || rows > kMaxWidth || K > kMaxWidth || (int64_t)E * rows > kMaxValues / K) {
        return set_error(QMOE_ERR_UNSUPPORTED, "E must be below 2^16, rows and K at most 2^20, E*rows*K at most 2^34");
    }
    if (E == 0) return finish(hipSuccess, "");
    QMOE_TRY(check_rows("x", x, (int64_t)E * rows, K, K, elem_bytes(dtype)));
    QMOE_TRY(check_fp8("output", codes, scales));
    return finish(qmoe::launch_fp8_quantize_weights(x, E, rows, K, dtype, transpose != 0, codes, scales,
                                                    (hipStream_t)stream),
                  "fp8_quantize_weights launch");
}

int qmoe_blocks_dequantize(const uint8_t* codes, const float* scales, int64_t rows, int32_t K, int32_t dtype, void* out,
                        void* stream)
{
    if (rows < 0 || K < 1) return set_error(QMOE_ERR_INVALID_ARG, "rows=%lld, K=%d", (long long)rows, K);
    QMOE_TRY(check_dtype(dtype));
    QMOE_TRY(check_sixteens("K", K));
    QMOE_TRY(check_values(rows, K));
    if (rows == 0) return finish(hipSuccess, "");
    QMOE_TRY(check_fp8("input", codes, scales));
    QMOE_TRY(check_rows("out", out, rows, K, K, elem_bytes(dtype)));
    return finish(qmoe::launch_fp8_dequantize(codes, scales, 1, rows, K, 1, dtype, out, (hipStream_t)stream),
                  "fp8_dequantize launch");
}

int qmoe_blocks_dequantize_weights(const uint8_t* codes, const float* scales, int32_t E, int32_t rows, int32_t K,
                                int32_t dtype, void* out, void* stream)
{
    if (E < 0 || rows < 1 || K < 1) return set_error(QMOE_ERR_INVALID_ARG, "E=%d, rows=%d, K=%d", E, rows, K);
    QMOE_TRY(check_dtype(dtype));
    QMOE_TRY(check_sixteens("K", K));
    if (E > 65535 || rows > kMaxWidth || K > kMaxWidth || (int64_t)E * rows > kMaxValues / K) {
        return set_error(QMOE_ERR_UNSUPPORTED, "E must be below 2^16, rows and K at most 2^20, E*rows*K at most 2^34");
    }
    if (E == 0) return finish(hipSuccess, "");
    QMOE_TRY(check_fp8("input", codes, scales));
    QMOE_TRY(check_rows("out", out, (int64_t)E * rows, K, K, elem_bytes(dtype)));
    return finish(qmoe::launch_fp8_dequantize(codes, scales, E, rows, K, qmoe::kFp8Block, dtype, out,
                                              (hipStream_t)stream),
                  "fp8_dequantize_weights launch");
}

int qmoe_blocks_matmul(const uint8_t* a_codes, const float* a_scales, int64_t a_rows, const uint8_t* w_codes,
                    const float* w_scales, int32_t E, int32_t N, int32_t K, const int32_t* expert_offsets,
                    const int32_t* sorted_routes, int32_t top_k, int64_t rows, int32_t dtype, void* out, void* stream)
{
    if (E < 1 || E > kMaxExperts) return set_error(QMOE_ERR_INVALID_ARG, "E=%d outside [1, %d]", E, kMaxExperts);
    if (N < 1 || K < 1) return set_error(QMOE_ERR_INVALID_ARG, "N=%d and K=%d must be >= 1", N, K);
    if (rows < 0 || rows > INT32_MAX || a_rows < 0 || a_rows > INT32_MAX) {
        return set_error(QMOE_ERR_INVALID_ARG, "rows=%lld and a_rows=%lld must be in [0, 2^31)", (long long)rows,
                         (long long)a_rows);
    }
    QMOE_TRY(check_dtype(dtype));
    if (top_k < 1) return set_error(QMOE_ERR_INVALID_ARG, "top_k=%d must be >= 1", top_k);
    if (!expert_offsets && E != 1) {
        return set_error(QMOE_ERR_INVALID_ARG, "expert_offsets is NULL with E=%d experts", E);
    }
    if (!sorted_routes && a_rows < rows) {
        return set_error(QMOE_ERR_INVALID_ARG, "a_rows=%lld < rows=%lld", (long long)a_rows, (long long)rows);
    }
    if (dtype == QMOE_DTYPE_F32) return set_error(QMOE_ERR_UNSUPPORTED, "the product's dtype must be F16 or BF16");
    QMOE_TRY(check_sixteens("K", K));
    if (K > kMaxWidth || N > kMaxWidth) {
        return set_error(QMOE_ERR_UNSUPPORTED, "N=%d and K=%d must be at most 2^20", N, K);
    }
    if (rows >= kMaxRowsEach) return set_error(QMOE_ERR_UNSUPPORTED, "rows=%lld must be below 2^24", (long long)rows);
    if (rows * N > qmoe::kMxMaxOutputs) {
        return set_error(QMOE_ERR_UNSUPPORTED, "rows*N=%lld must be at most 2^40", (long long)(rows * N));
    }
    if (sorted_routes && a_rows > INT32_MAX / K) {
        return set_error(QMOE_ERR_UNSUPPORTED, "a_codes read through sorted_routes must be below 2^31 bytes");
    }
    if (rows == 0) return finish(hipSuccess, "");
    if (a_rows == 0) return set_error(QMOE_ERR_INVALID_ARG, "a_rows is 0");
    QMOE_TRY(check_fp8("a", a_codes, a_scales));
    QMOE_TRY(check_fp8("w", w_codes, w_scales));
    if (expert_offsets) QMOE_TRY(check_words("expert_offsets", expert_offsets));
    if (sorted_routes) QMOE_TRY(check_words("sorted_routes", sorted_routes));
    QMOE_TRY(check_rows("out", out, rows, N, N, elem_bytes(dtype)));
    qmoe::Fp8MatmulArgs a{};
    a.a_codes = a_codes;
    a.a_scales = a_scales;
    a.a_rows = a_rows;
    a.w_codes = w_codes;
    a.w_scales = w_scales;
    a.E = E;
    a.N = N;
    a.K = K;
    a.offsets = expert_offsets;
    a.sorted_routes = sorted_routes;
    a.top_k = top_k;
    a.rows = (int)rows;
    a.dtype = dtype;
    a.out = out;
    return finish(qmoe::launch_fp8_matmul(a, (hipStream_t)stream), "fp8_matmul launch");
}

int qmoe_activate(const void* y, int64_t row_stride, int64_t rows, int32_t I, int32_t dtype, int32_t activation,
                  int32_t swiglu_fusion, float activation_alpha, float activation_beta, float swiglu_limit, void* out,
                  void* stream)
{
    QMOE_TRY(check_activation(rows, I, dtype, activation, swiglu_fusion, activation_alpha, activation_beta, swiglu_limit));
    if (rows == 0) return finish(hipSuccess, "");
    QMOE_TRY(check_rows("y", y, rows, row_stride, 2 * (int64_t)I, elem_bytes(dtype)));
    QMOE_TRY(check_rows("out", out, rows, I, I, elem_bytes(dtype)));
    qmoe::ActivateArgs a = activate_args(y, row_stride, rows, I, dtype, activation, swiglu_fusion, activation_alpha,
                                         activation_beta, swiglu_limit);
    a.out = out;
    return finish(qmoe::launch_activate(a, (hipStream_t)stream), "activate launch");
}

int qmoe_activate_blocks(const void* y, int64_t row_stride, int64_t rows, int32_t I, int32_t dtype, int32_t activation,
                      int32_t swiglu_fusion, float activation_alpha, float activation_beta, float swiglu_limit,
                      uint8_t* codes, float* scales, void* stream)
{
    QMOE_TRY(check_activation(rows, I, dtype, activation, swiglu_fusion, activation_alpha, activation_beta, swiglu_limit));
    QMOE_TRY(check_sixteens("I", I));
    if (rows == 0) return finish(hipSuccess, "");
    QMOE_TRY(check_rows("y", y, rows, row_stride, 2 * (int64_t)I, elem_bytes(dtype)));
    QMOE_TRY(check_fp8("output", codes, scales));
    qmoe::ActivateArgs a = activate_args(y, row_stride, rows, I, dtype, activation, swiglu_fusion, activation_alpha,
                                         activation_beta, swiglu_limit);
    a.codes = codes;
    a.scales = scales;
    return finish(qmoe::launch_activate(a, (hipStream_t)stream), "activate_fp8 launch");
}

int qmoe_activate_backward(const void* grad, int64_t grad_stride, const void* y, int64_t row_stride, int64_t rows,
                           int32_t I, int32_t dtype, int32_t activation, int32_t swiglu_fusion,
                           float activation_alpha, float activation_beta, float swiglu_limit, void* grad_y,
                           void* stream)
{
    QMOE_TRY(check_activation(rows, I, dtype, activation, swiglu_fusion, activation_alpha, activation_beta, swiglu_limit));
    if (rows == 0) return finish(hipSuccess, "");
    QMOE_TRY(check_rows("grad", grad, rows, grad_stride, I, elem_bytes(dtype)));
    QMOE_TRY(check_rows("y", y, rows, row_stride, 2 * (int64_t)I, elem_bytes(dtype)));
    QMOE_TRY(check_rows("grad_y", grad_y, rows, 2 * (int64_t)I, 2 * (int64_t)I, elem_bytes(dtype)));
    qmoe::ActivateArgs a = activate_args(y, row_stride, rows, I, dtype, activation, swiglu_fusion, activation_alpha,
                                         activation_beta, swiglu_limit);
    a.grad = grad;
    a.grad_stride = grad_stride;
    a.grad_y = grad_y;
    return finish(qmoe::launch_activate_backward(a, (hipStream_t)stream), "activate_backward launch");
}

}  // extern "C"
