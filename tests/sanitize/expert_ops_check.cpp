// expert_ops_check.cpp -- drives every entry point of expert_ops.cpp through
// its host code with the kernel launchers replaced by the stand-ins below;
// built with AddressSanitizer and UndefinedBehaviorSanitizer.  Pointers stand
// for device memory and are never dereferenced.
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "expert_ops.h"
#include "qmoe.h"

namespace {

int g_checks = 0;
int g_launches = 0;
qmoe::PermuteArgs g_permute;
qmoe::MxMatmulArgs g_matmul;

#define EXPECT(cond)                                                                       \
    do {                                                                                   \
        ++g_checks;                                                                        \
        if (!(cond)) {                                                                     \
            std::fprintf(stderr, "%s:%d: %s (%s)\n", __FILE__, __LINE__, #cond, qmoe_last_error()); \
            std::abort();                                                                  \
        }                                                                                  \
    } while (0)

alignas(256) char g_mem[4096];
char* const kT = g_mem;
uint8_t* const kB = reinterpret_cast<uint8_t*>(g_mem);
int32_t* const kI = reinterpret_cast<int32_t*>(g_mem);
float* const kF = reinterpret_cast<float*>(g_mem);

}  // namespace

namespace qmoe {

int64_t permute_ws_ints(int64_t T, int top_k, int E) { return T * top_k > 1000 ? (T * top_k / 1000 + 2) * (E + 1) : 0; }
hipError_t launch_permute(const PermuteArgs& a, hipStream_t)
{
    ++g_launches;
    g_permute = a;
    return hipSuccess;
}
hipError_t launch_unpermute(const UnpermuteArgs&, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_unpermute_backward(const UnpermuteArgs&, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_mx_quantize(const void*, int64_t, int64_t, int, int, uint8_t*, uint8_t*, hipStream_t)
{
    return ++g_launches, hipSuccess;
}
hipError_t launch_mx_quantize_columns(const void*, int, int, int, int, uint8_t*, uint8_t*, hipStream_t)
{
    return ++g_launches, hipSuccess;
}
hipError_t launch_mx_dequantize(const uint8_t*, const uint8_t*, int64_t, int, void*, hipStream_t)
{
    return ++g_launches, hipSuccess;
}
hipError_t launch_mx_matmul(const MxMatmulArgs& a, hipStream_t)
{
    ++g_launches;
    g_matmul = a;
    return hipErrorLaunchFailure;  // a failing launch is reported, not swallowed
}

}  // namespace qmoe

namespace {

int permute(int64_t stride, int64_t T, int H, int dtype, int k, int E, size_t ws_bytes)
{
    return qmoe_permute(kT, stride, T, H, dtype, kI, k, E, kT, kI, kI, kI, kT, ws_bytes, nullptr);
}

void expect_error(int rc, int code)
{
    EXPECT(rc == code);
    EXPECT(std::strlen(qmoe_last_error()) > 6);
}

}  // namespace

int main()
{
    const int64_t big[] = {-1, INT64_MIN, INT64_MAX, int64_t(1) << 23, int64_t(1) << 40};
    const int32_t bad[] = {0, -1, INT_MIN, INT_MAX, 1025};
    EXPECT(permute(64, 4, 64, 1, 2, 8, 0) == QMOE_OK && g_launches == 1 && g_permute.elem == 2);
    EXPECT(permute(64, 4, 64, 3, 2, 8, 0) == QMOE_OK && g_permute.elem == 4);
    EXPECT(permute(64, 0, 64, 3, 2, 8, 0) == QMOE_OK && g_permute.hidden == nullptr);
    EXPECT(qmoe_last_error()[0] == 0);
    const int before = g_launches;
    for (int64_t T : big) {
        EXPECT(permute(64, T, 64, 1, 2, 8, SIZE_MAX) < 0);
        EXPECT(qmoe_unpermute(kT, 64, kI, kF, T, 2, 64, 1, kT, nullptr) < 0);
        EXPECT(qmoe_unpermute_backward(kT, 64, kT, 64, kI, kF, T, 2, 64, 1, kT, kF, nullptr) < 0);
        EXPECT(qmoe_permute_workspace_size(T, 2, 8) == 0);
        if (T < 0 || T > INT_MAX) {
            EXPECT(qmoe_mx_matmul(kB, kB, 8, kB, kB, 1, 8, 32, nullptr, nullptr, 1, T, 1, kT, nullptr) < 0);
            EXPECT(qmoe_mx_matmul(kB, kB, T, kB, kB, 1, 8, 32, nullptr, nullptr, 1, 8, 1, kT, nullptr) < 0);
            EXPECT(qmoe_mx_quantize(kT, 64, T, 64, 1, kB, kB, nullptr) < 0);
            EXPECT(qmoe_mx_dequantize(kB, kB, T, 64, 1, kT, nullptr) < 0);
        }
        EXPECT(permute(T, 4, T == (int64_t(1) << 23) || T == (int64_t(1) << 40) ? 0 : 64, 1, 2, 8, 0) < 0);
    }
    for (int32_t v : bad) {
        EXPECT(permute(64, 4, 64, 1, v, 8, 0) < 0);
        EXPECT(permute(64, 4, 64, 1, 2, v, 0) < 0);
        EXPECT(permute(64, 4, 64, v == 1025 ? 4 : v, 2, 8, 0) < 0);
        EXPECT(qmoe_permute_workspace_size(8, v, 8) == 0 && qmoe_permute_workspace_size(8, 2, v) == 0);
        EXPECT(qmoe_mx_matmul(kB, kB, 8, kB, kB, v, 8, 32, kI, nullptr, 1, 8, 1, kT, nullptr) < 0);
        if (v != 1025) {
            EXPECT(qmoe_mx_matmul(kB, kB, 8, kB, kB, 1, v, 32, nullptr, nullptr, 1, 8, 1, kT, nullptr) < 0);
            EXPECT(qmoe_mx_quantize_columns(kT, 1, 32, v, 1, kB, kB, nullptr) < 0);
        }
        EXPECT(qmoe_mx_matmul(kB, kB, 8, kB, kB, 1, 8, v, nullptr, nullptr, 1, 8, 1, kT, nullptr) < 0);
        EXPECT(qmoe_mx_quantize(kT, 1 << 30, 2, v, 1, kB, kB, nullptr) < 0);
        EXPECT(qmoe_mx_quantize_columns(kT, 1, v, 8, 1, kB, kB, nullptr) < 0);
        EXPECT(qmoe_mx_dequantize(kB, kB, 2, v, 1, kT, nullptr) < 0);
    }
    EXPECT(g_launches == before);
    expect_error(permute(64, 4000, 64, 1, 2, 8, 4), QMOE_ERR_WORKSPACE);
    EXPECT(permute(64, 4000, 64, 1, 2, 8, qmoe_permute_workspace_size(4000, 2, 8)) == QMOE_OK);
    EXPECT(qmoe_unpermute(kT, 64, kI, nullptr, 4, 2, 64, 3, kT, nullptr) == QMOE_OK);
    EXPECT(qmoe_unpermute_backward(kT, 64, nullptr, 0, kI, nullptr, 4, 2, 64, 3, kT, nullptr, nullptr) == QMOE_OK);
    EXPECT(qmoe_mx_quantize(kT, 64, 4, 64, 2, kB, kB, nullptr) == QMOE_OK);
    EXPECT(qmoe_mx_quantize_columns(kT, 3, 64, 5, 2, kB, kB, nullptr) == QMOE_OK);
    EXPECT(qmoe_mx_dequantize(kB, kB, 4, 64, 2, kT, nullptr) == QMOE_OK);
    expect_error(qmoe_mx_matmul(kB, kB, 8, kB, kB, 1, 8, 32, nullptr, kI, 3, 24, 1, kT, nullptr), QMOE_ERR_HIP);
    EXPECT(g_matmul.rows == 24 && g_matmul.a_rows == 8 && g_matmul.top_k == 3);
    std::printf("%d checks passed\n", g_checks);
    return 0;
}
