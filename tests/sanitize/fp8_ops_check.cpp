// fp8_ops_check.cpp -- drives every entry point of fp8_ops.cpp through its
// host code with the kernel launchers replaced by the stand-ins below; built
// with AddressSanitizer and UndefinedBehaviorSanitizer.  Pointers stand for
// device memory and are never dereferenced.
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "fp8_ops.h"
#include "qmoe.h"

namespace {

int g_checks = 0;
int g_launches = 0;
hipError_t g_result = hipSuccess;
qmoe::RouteScoresArgs g_route;
qmoe::Fp8MatmulArgs g_matmul;
qmoe::ActivateArgs g_activate;
int64_t g_rows = 0;
int g_block_rows = 0;

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

hipError_t launch_route_scores(const RouteScoresArgs& a, hipStream_t) { return ++g_launches, g_route = a, g_result; }
hipError_t launch_route_scores_backward(const RouteScoresArgs& a, hipStream_t) { return ++g_launches, g_route = a, g_result; }
hipError_t launch_fp8_quantize(const void*, int64_t, int64_t rows, int, int, uint8_t*, float*, hipStream_t)
{
    return ++g_launches, g_rows = rows, g_result;
}
hipError_t launch_fp8_quantize_weights(const void*, int, int rows, int, int, bool, uint8_t*, float*, hipStream_t)
{
    return ++g_launches, g_rows = rows, g_result;
}
hipError_t launch_fp8_dequantize(const uint8_t*, const float*, int, int64_t rows, int, int block_rows, int, void*, hipStream_t)
{
    return ++g_launches, g_rows = rows, g_block_rows = block_rows, g_result;
}
hipError_t launch_fp8_matmul(const Fp8MatmulArgs& a, hipStream_t) { return ++g_launches, g_matmul = a, g_result; }
hipError_t launch_activate(const ActivateArgs& a, hipStream_t) { return ++g_launches, g_activate = a, g_result; }
hipError_t launch_activate_backward(const ActivateArgs& a, hipStream_t) { return ++g_launches, g_activate = a, g_result; }

}  // namespace qmoe

namespace {

int route(int64_t T, int64_t stride, int32_t E, int32_t k, int32_t groups, int32_t kept, float scale)
{
    return qmoe_route_scores(kT, stride, T, E, 3, kF, k, 1, groups, kept, 2, 7, scale, kI, kF, nullptr);
}

int product(int64_t a_rows, int32_t E, int32_t N, int32_t K, const int32_t* routes, int32_t k, int64_t rows)
{
    return qmoe_blocks_matmul(kB, kF, a_rows, kB, kF, E, N, K, E > 0 ? kI : nullptr, routes, k, rows, 2, kT, nullptr);
}

int act(int64_t rows, int64_t stride, int32_t I, float limit)
{
    return qmoe_activate(kT, stride, rows, I, 1, 0, 1, 1.0f, 0.0f, limit, kT, nullptr);
}

}  // namespace

int main()
{
    const int64_t big[] = {-1, INT64_MIN, int64_t(1) << 23, int64_t(1) << 31, int64_t(1) << 62, INT64_MAX};
    const int32_t bad[] = {0, -1, INT_MIN, INT_MAX};
    EXPECT(route(4, 64, 64, 4, 8, 4, 1.0f) == QMOE_OK && g_route.normalize == 1 && g_route.sigmoid == 1 && g_route.top_groups == 4);
    EXPECT(route(0, 64, 64, 4, 8, 4, 1.0f) == QMOE_OK && g_launches == 1);
    EXPECT(product(8, 4, 32, 64, kI, 2, 16) == QMOE_OK && g_matmul.rows == 16 && g_matmul.top_k == 2);
    EXPECT(act(4, 128, 64, INFINITY) == QMOE_OK && g_activate.out == kT && !g_activate.codes);
    EXPECT(qmoe_activate_blocks(kT, 128, 4, 64, 1, 1, 2, 1.0f, 0.0f, 1.0f, kB, kF, nullptr) == QMOE_OK);
    EXPECT(g_activate.codes == kB && g_activate.halves && g_activate.geglu);
    EXPECT(qmoe_activate_backward(kT, 64, kT, 128, 4, 64, 2, 0, 1, 1.0f, 0.0f, 1.0f, kT, nullptr) == QMOE_OK && g_activate.grad == kT);
    EXPECT(qmoe_blocks_quantize(kT, 64, 4, 64, 3, kB, kF, nullptr) == QMOE_OK && g_rows == 4);
    EXPECT(qmoe_blocks_quantize_weights(kT, 2, 48, 5, 3, 1, kB, kF, nullptr) == QMOE_OK && g_rows == 48);
    EXPECT(qmoe_blocks_dequantize(kB, kF, 9, 64, 3, kT, nullptr) == QMOE_OK && g_block_rows == 1);
    EXPECT(qmoe_blocks_dequantize_weights(kB, kF, 2, 9, 64, 3, kT, nullptr) == QMOE_OK && g_block_rows == 128);
    EXPECT(qmoe_route_scores_backward(kF, kT, 64, kI, 4, 64, 1, 4, 0, 0, 1.0f, kT, nullptr) == QMOE_OK && g_route.sigmoid == 0);
    EXPECT(qmoe_last_error()[0] == 0);
    const int before = g_launches;
    for (int64_t n : big) {
        EXPECT(route(n, 64, 64, 4, 8, 4, 1.0f) < 0);
        EXPECT(qmoe_route_scores_backward(kF, kT, 64, kI, n, 64, 1, 4, 0, 0, 1.0f, kT, nullptr) < 0);
        if (n < 64 || n > int64_t(1) << 40) EXPECT(route(4, n, 64, 4, 8, 4, 1.0f) < 0);
        if (n < 0 || n > int64_t(1) << 34) {
            EXPECT(act(n, 128, 64, 1.0f) < 0);
            EXPECT(qmoe_blocks_quantize(kT, 64, n, 64, 3, kB, kF, nullptr) < 0);
            EXPECT(qmoe_blocks_dequantize(kB, kF, n, 64, 3, kT, nullptr) < 0);
            EXPECT(act(4, n, 64, 1.0f) < 0);
            EXPECT(qmoe_blocks_quantize(kT, n, 4, 64, 3, kB, kF, nullptr) < 0);
        }
        if (n < 0 || n > INT_MAX) {
            EXPECT(product(n, 4, 32, 64, nullptr, 1, 8) < 0);
            EXPECT(product(8, 4, 32, 64, nullptr, 1, n) < 0);
        }
    }
    for (int32_t v : bad) {
        EXPECT(route(4, INT_MAX, v, 4, 1, 1, 1.0f) < 0);
        EXPECT(route(4, 64, 64, v, 8, 4, 1.0f) < 0);
        EXPECT(route(4, 64, 64, 4, v, 1, 1.0f) < 0);
        EXPECT(route(4, 64, 64, 4, 8, v, 1.0f) < 0);
        EXPECT(qmoe_route_scores_backward(kF, kT, 64, kI, 4, 64, 1, v, 0, 0, 1.0f, kT, nullptr) < 0);
        EXPECT(product(8, v, 32, 64, nullptr, 1, 8) < 0);
        EXPECT(product(8, 4, v, 64, nullptr, 1, 8) < 0);
        EXPECT(product(8, 4, 32, v, nullptr, 1, 8) < 0);
        if (v != INT_MAX) EXPECT(product(8, 4, 32, 64, kI, v, 8) < 0);
        EXPECT(act(4, INT64_MAX / 64, v, 1.0f) < 0);
        EXPECT(qmoe_blocks_quantize(kT, INT_MAX, 4, v, 3, kB, kF, nullptr) < 0);
        EXPECT(qmoe_blocks_quantize_weights(kT, 2, v, 64, 3, 0, kB, kF, nullptr) < 0);
        EXPECT(qmoe_blocks_quantize_weights(kT, 2, 64, v, 3, 1, kB, kF, nullptr) < 0);
        EXPECT(qmoe_blocks_dequantize_weights(kB, kF, 2, v, 64, 3, kT, nullptr) < 0);
        if (v != 0) EXPECT(qmoe_blocks_quantize_weights(kT, v, 64, 64, 3, 0, kB, kF, nullptr) < 0);
    }
    const float wrong[] = {NAN, -1.0f, 0.0f, -INFINITY};
    for (float v : wrong) EXPECT(act(4, 128, 64, v) < 0);
    EXPECT(route(4, 64, 64, 4, 8, 4, INFINITY) < 0);
    EXPECT(g_launches == before);
    g_result = hipErrorInvalidValue;
    EXPECT(product(8, 4, 32, 64, nullptr, 1, 8) == QMOE_ERR_HIP && std::strstr(qmoe_last_error(), "launch"));
    EXPECT(act(4, 128, 64, 1.0f) == QMOE_ERR_HIP);
    EXPECT(route(4, 64, 64, 4, 8, 4, 1.0f) == QMOE_ERR_HIP);
    std::printf("%d checks passed\n", g_checks);
    return 0;
}
