// expert_ops.cpp -- the C ABI of the sort by expert and back and of the MXFP4
// operators: argument checks and launches.  Every check runs before the first
// launch, so an error return leaves the stream and all outputs untouched.
#include <hip/hip_runtime.h>

#include "abi_checks.h"
#include "expert_ops.h"
#include "mx_shape.h"
#include "qmoe.h"

namespace {

using namespace qmoe::abi;

int check_mx(const char* name, const uint8_t* codes, const uint8_t* scales)
{
    if (!codes || !scales) return set_error(QMOE_ERR_INVALID_ARG, "%s codes/scales is NULL", name);
    if (!aligned(codes, 16)) return set_error(QMOE_ERR_INVALID_ARG, "%s codes not 16-byte aligned", name);
    return QMOE_OK;
}

}  // namespace

extern "C" {

size_t qmoe_permute_workspace_size(int64_t T, int32_t top_k, int32_t E)
{
    if (T < 0 || T > kMaxTokens || top_k < 1 || top_k > kMaxTopK || T * top_k > INT32_MAX || E < 1 ||
        E > kMaxExperts) {
        return 0;
    }
    return (size_t)qmoe::permute_ws_ints(T, top_k, E) * 4;
}

int qmoe_permute(const void* hidden, int64_t row_stride, int64_t T, int32_t H, int32_t dtype,
                 const int32_t* topk_ids, int32_t top_k, int32_t E, void* rows, int32_t* expert_offsets,
                 int32_t* sorted_routes, int32_t* route_rows, void* workspace, size_t workspace_bytes,
                 void* stream)
{
    QMOE_TRY(check_routes(T, top_k));
    if (E < 1 || E > kMaxExperts) {
        return set_error(QMOE_ERR_INVALID_ARG, "E=%d outside [1, %d]", E, kMaxExperts);
    }
    QMOE_TRY(check_words("expert_offsets", expert_offsets));
    if ((hidden == nullptr) != (rows == nullptr) && T > 0) {
        return set_error(QMOE_ERR_INVALID_ARG, "hidden and rows must both be given or both be NULL");
    }
    if (T > 0) {
        QMOE_TRY(check_words("topk_ids", topk_ids));
        QMOE_TRY(check_words("sorted_routes", sorted_routes));
        QMOE_TRY(check_words("route_rows", route_rows));
        if (hidden) {
            QMOE_TRY(check_dtype(dtype));
            QMOE_TRY(check_width(H));
            QMOE_TRY(check_rows("hidden", hidden, T, row_stride, H, elem_bytes(dtype)));
            QMOE_TRY(check_rows("rows", rows, T * top_k, H, H, elem_bytes(dtype)));
        }
        const size_t need = qmoe_permute_workspace_size(T, top_k, E);
        if (need > 0) {
            if (workspace_bytes < need) {
                return set_error(QMOE_ERR_WORKSPACE, "workspace_bytes=%zu < %zu", workspace_bytes, need);
            }
            QMOE_TRY(check_words("workspace", workspace));
        }
    }
    qmoe::PermuteArgs a;
    a.hidden = T > 0 ? hidden : nullptr;
    a.row_stride = row_stride;
    a.T = T;
    a.H = a.hidden ? H : 1;
    a.elem = elem_bytes(dtype);
    a.ids = topk_ids;
    a.top_k = top_k;
    a.E = E;
    a.rows = rows;
    a.offsets = expert_offsets;
    a.sorted_routes = sorted_routes;
    a.route_rows = route_rows;
    a.ws = static_cast<int32_t*>(workspace);
    return finish(qmoe::launch_permute(a, (hipStream_t)stream), "permute launch");
}

int qmoe_unpermute(const void* rows, int64_t row_stride, const int32_t* route_rows, const float* weights,
                   int64_t T, int32_t top_k, int32_t H, int32_t dtype, void* out, void* stream)
{
    QMOE_TRY(check_routes(T, top_k));
    QMOE_TRY(check_dtype(dtype));
    QMOE_TRY(check_width(H));
    if (T == 0) return finish(hipSuccess, "");
    QMOE_TRY(check_rows("rows", rows, T * top_k, row_stride, H, elem_bytes(dtype)));
    QMOE_TRY(check_words("route_rows", route_rows));
    if (weights) QMOE_TRY(check_words("weights", weights));
    QMOE_TRY(check_rows("out", out, T, H, H, elem_bytes(dtype)));
    qmoe::UnpermuteArgs a{};
    a.rows = rows;
    a.row_stride = row_stride;
    a.route_rows = route_rows;
    a.weights = weights;
    a.T = T;
    a.top_k = top_k;
    a.H = H;
    a.dtype = dtype;
    a.out = out;
    return finish(qmoe::launch_unpermute(a, (hipStream_t)stream), "unpermute launch");
}

int qmoe_unpermute_backward(const void* grad_out, int64_t grad_stride, const void* rows, int64_t row_stride,
                            const int32_t* route_rows, const float* weights, int64_t T, int32_t top_k,
                            int32_t H, int32_t dtype, void* grad_rows, float* grad_weights, void* stream)
{
    QMOE_TRY(check_routes(T, top_k));
    QMOE_TRY(check_dtype(dtype));
    QMOE_TRY(check_width(H));
    if (T == 0) return finish(hipSuccess, "");
    if ((rows == nullptr) != (grad_weights == nullptr)) {
        return set_error(QMOE_ERR_INVALID_ARG, "rows and grad_weights must both be given or both be NULL");
    }
    QMOE_TRY(check_rows("grad_out", grad_out, T, grad_stride, H, elem_bytes(dtype)));
    if (rows) {
        QMOE_TRY(check_rows("rows", rows, T * top_k, row_stride, H, elem_bytes(dtype)));
        QMOE_TRY(check_words("grad_weights", grad_weights));
    }
    QMOE_TRY(check_words("route_rows", route_rows));
    if (weights) QMOE_TRY(check_words("weights", weights));
    QMOE_TRY(check_rows("grad_rows", grad_rows, T * top_k, H, H, elem_bytes(dtype)));
    qmoe::UnpermuteArgs a{};
    a.rows = rows;
    a.row_stride = row_stride;
    a.route_rows = route_rows;
    a.weights = weights;
    a.T = T;
    a.top_k = top_k;
    a.H = H;
    a.dtype = dtype;
    a.grad_out = grad_out;
    a.grad_stride = grad_stride;
    a.grad_rows = grad_rows;
    a.grad_weights = grad_weights;
    return finish(qmoe::launch_unpermute_backward(a, (hipStream_t)stream), "unpermute backward launch");
}

int qmoe_mx_quantize(const void* x, int64_t row_stride, int64_t rows, int32_t K, int32_t dtype,
                     uint8_t* codes, uint8_t* scales, void* stream)
{
    if (rows < 0 || K < 1) return set_error(QMOE_ERR_INVALID_ARG, "rows=%lld, K=%d", (long long)rows, K);
    QMOE_TRY(check_dtype(dtype));
    if (K % 32) return set_error(QMOE_ERR_UNSUPPORTED, "K=%d must be a multiple of 32", K);
    if (rows > kMaxValues / K) return set_error(QMOE_ERR_UNSUPPORTED, "rows*K must be at most 2^34");
    if (rows == 0) return finish(hipSuccess, "");
    QMOE_TRY(check_rows("x", x, rows, row_stride, K, elem_bytes(dtype)));
    QMOE_TRY(check_mx("output", codes, scales));
    return finish(qmoe::launch_mx_quantize(x, row_stride, rows, K, dtype, codes, scales, (hipStream_t)stream),
                  "mx_quantize launch");
}

int qmoe_mx_quantize_columns(const void* x, int32_t E, int32_t rows, int32_t K, int32_t dtype,
                             uint8_t* codes, uint8_t* scales, void* stream)
{
    if (E < 0 || rows < 1 || K < 1) {
        return set_error(QMOE_ERR_INVALID_ARG, "E=%d, rows=%d, K=%d", E, rows, K);
    }
    QMOE_TRY(check_dtype(dtype));
    if (rows % 32) return set_error(QMOE_ERR_UNSUPPORTED, "rows=%d must be a multiple of 32", rows);
    if (E > 65535 || rows > kMaxWidth || K > kMaxWidth || (int64_t)E * rows > kMaxValues / K) {
        return set_error(QMOE_ERR_UNSUPPORTED,
                         "E must be below 2^16, rows and K at most 2^20, E*rows*K at most 2^34");
    }
    if (E == 0) return finish(hipSuccess, "");
    QMOE_TRY(check_rows("x", x, (int64_t)E * rows, K, K, elem_bytes(dtype)));
    QMOE_TRY(check_mx("output", codes, scales));
    return finish(qmoe::launch_mx_quantize_columns(x, E, rows, K, dtype, codes, scales, (hipStream_t)stream),
                  "mx_quantize_columns launch");
}

int qmoe_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t K, int32_t dtype,
                       void* out, void* stream)
{
    if (rows < 0 || K < 1) return set_error(QMOE_ERR_INVALID_ARG, "rows=%lld, K=%d", (long long)rows, K);
    QMOE_TRY(check_dtype(dtype));
    if (K % 32) return set_error(QMOE_ERR_UNSUPPORTED, "K=%d must be a multiple of 32", K);
    if (rows > kMaxValues / K) return set_error(QMOE_ERR_UNSUPPORTED, "rows*K must be at most 2^34");
    if (rows == 0) return finish(hipSuccess, "");
    QMOE_TRY(check_mx("input", codes, scales));
    QMOE_TRY(check_rows("out", out, rows, K, K, elem_bytes(dtype)));
    return finish(qmoe::launch_mx_dequantize(codes, scales, rows * (K / 32), dtype, out, (hipStream_t)stream),
                  "mx_dequantize launch");
}

int qmoe_mx_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int64_t a_rows, const uint8_t* w_codes,
                   const uint8_t* w_scales, int32_t E, int32_t N, int32_t K, const int32_t* expert_offsets,
                   const int32_t* sorted_routes, int32_t top_k, int64_t rows, int32_t dtype, void* out,
                   void* stream)
{
    if (E < 1 || E > kMaxExperts) {
        return set_error(QMOE_ERR_INVALID_ARG, "E=%d outside [1, %d]", E, kMaxExperts);
    }
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
    if (K % 32) return set_error(QMOE_ERR_UNSUPPORTED, "K=%d must be a multiple of 32", K);
    if (K > kMaxWidth || N > kMaxWidth) {
        return set_error(QMOE_ERR_UNSUPPORTED, "N=%d and K=%d must be at most 2^20", N, K);
    }
    if (rows >= (int64_t(1) << 24)) {
        return set_error(QMOE_ERR_UNSUPPORTED, "rows=%lld must be below 2^24", (long long)rows);
    }
    if (rows * N > qmoe::kMxMaxOutputs) {
        return set_error(QMOE_ERR_UNSUPPORTED, "rows*N=%lld must be at most 2^40", (long long)(rows * N));
    }
    if (sorted_routes && a_rows > INT32_MAX / (K / 2)) {
        return set_error(QMOE_ERR_UNSUPPORTED, "a_codes read through sorted_routes must be below 2^31 bytes");
    }
    if (rows == 0) return finish(hipSuccess, "");
    if (a_rows == 0) return set_error(QMOE_ERR_INVALID_ARG, "a_rows is 0");
    QMOE_TRY(check_mx("a", a_codes, a_scales));
    QMOE_TRY(check_mx("w", w_codes, w_scales));
    if (expert_offsets) QMOE_TRY(check_words("expert_offsets", expert_offsets));
    if (sorted_routes) QMOE_TRY(check_words("sorted_routes", sorted_routes));
    QMOE_TRY(check_rows("out", out, rows, N, N, elem_bytes(dtype)));
    qmoe::MxMatmulArgs a{};
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
    return finish(qmoe::launch_mx_matmul(a, (hipStream_t)stream), "mx_matmul launch");
}

}  // extern "C"
