// abi_checks.h -- argument checks shared by the C ABI of the operators beside
// the layer (expert_ops.cpp, fp8_ops.cpp).  Each sets qmoe_last_error() and
// returns its code.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_ops.h"
#include "qmoe.h"
#include "qmoe_internal.h"

namespace qmoe {

namespace abi {

using qmoe::set_error;

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 1024;
// Largest sizes the kernels' grids and 32-bit in-row arithmetic are laid out
// for: tokens (one launch thread group each), row width, and values of one
// conversion.
constexpr int64_t kMaxTokens = (int64_t(1) << 23) - 1;
constexpr int kMaxWidth = 1 << 20;
constexpr int64_t kMaxValues = int64_t(1) << 34;

inline int finish(hipError_t e, const char* what)
{
    if (e != hipSuccess) return set_error(QMOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
    qmoe::clear_error();
    return QMOE_OK;
}

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline int elem_bytes(int dtype) { return dtype == QMOE_DTYPE_F32 ? 4 : 2; }

inline int check_dtype(int dtype)
{
    if (dtype == QMOE_DTYPE_F16 || dtype == QMOE_DTYPE_BF16 || dtype == QMOE_DTYPE_F32) return QMOE_OK;
    return set_error(QMOE_ERR_INVALID_ARG, "dtype=%d is none of F16 (1), BF16 (2) and F32 (3)", dtype);
}

// Sizes shared by the sort and the way back.
inline int check_routes(int64_t T, int32_t top_k)
{
    if (T < 0) return set_error(QMOE_ERR_INVALID_ARG, "T=%lld < 0", (long long)T);
    if (top_k < 1 || top_k > kMaxTopK) {
        return set_error(QMOE_ERR_INVALID_ARG, "top_k=%d outside [1, %d]", top_k, kMaxTopK);
    }
    if (T > kMaxTokens) return set_error(QMOE_ERR_UNSUPPORTED, "T=%lld must be below 2^23", (long long)T);
    if (T * top_k > INT32_MAX) return set_error(QMOE_ERR_INVALID_ARG, "T*top_k must be < 2^31");
    return QMOE_OK;
}

inline int check_width(int32_t H)
{
    if (H < 1) return set_error(QMOE_ERR_INVALID_ARG, "H=%d must be >= 1", H);
    if (H > kMaxWidth) return set_error(QMOE_ERR_UNSUPPORTED, "H=%d must be at most 2^20", H);
    return QMOE_OK;
}

// Rows of `width` elements, `stride` elements apart.
inline int check_rows(const char* name, const void* p, int64_t n, int64_t stride, int64_t width, int elem)
{
    if (!p) return set_error(QMOE_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, elem)) return set_error(QMOE_ERR_INVALID_ARG, "%s is not aligned to its element", name);
    if (stride < width) {
        return set_error(QMOE_ERR_INVALID_ARG, "%s: row stride %lld below the row's %lld elements", name,
                         (long long)stride, (long long)width);
    }
    int64_t span;
    if (__builtin_mul_overflow(n, stride, &span) || span > INT64_MAX / 8) {
        return set_error(QMOE_ERR_INVALID_ARG, "%s: rows * row stride overflows", name);
    }
    return QMOE_OK;
}

inline int check_words(const char* name, const void* p)
{
    if (!p) return set_error(QMOE_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, 4)) return set_error(QMOE_ERR_INVALID_ARG, "%s is not 4-byte aligned", name);
    return QMOE_OK;
}

#define QMOE_TRY(call)        \
    do {                      \
        const int rc_ = call; \
        if (rc_) return rc_;  \
    } while (0)

}  // namespace abi
}  // namespace qmoe
