// mx_shape_check.cpp -- the arithmetic that the grouped MXFP4 product shares
// with its launch (csrc/mx_shape.h), checked on the host under
// AddressSanitizer and UndefinedBehaviorSanitizer.
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "mx_shape.h"

namespace {

long g_checks = 0;

#define EXPECT(cond)                                                              \
    do {                                                                          \
        ++g_checks;                                                               \
        if (!(cond)) {                                                            \
            std::fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #cond);       \
            std::abort();                                                         \
        }                                                                         \
    } while (0)

// A lane that passes the comparison with what is left reads inside the buffer.
void check_bytes_left()
{
    const uint32_t sizes[] = {0, 1, 15, 16, 17, 48, 127, 128, 4096, 1u << 27, (1u << 31) - 16, (1u << 31) - 1};
    const uint32_t at[] = {0, 8, 16, 96, 127, 128, 129, 4080, 4096, 1u << 19, (1u << 20) + 896};
    for (uint32_t n : sizes) {
        for (uint32_t a : at) {
            const uint32_t left = qmoe::mx_bytes_left(n, a);
            EXPECT(left == 0 || (uint64_t)a + left == n);
            EXPECT(left == 0 ? a >= n : a < n);
            EXPECT(qmoe::kMxOutside >= left);
        }
    }
}

// The lanes' scale offsets of the product's steps, rows of `blocks` bytes read 32 at a time: what is
// used lies in its own row, and nothing that passes the comparison lies behind the last row.
void check_scale_rows()
{
    for (int rows = 1; rows <= 40; rows += 13) {
        for (int blocks = 16; blocks <= 176; blocks += 16) {
            const uint32_t bytes = (uint32_t)(rows * blocks);
            for (int at = 0; at < blocks + 64; at += 32) {  // groups of steps, and some of a tile that is over
                const uint32_t left = qmoe::mx_bytes_left(bytes, (uint32_t)at);
                for (int row = 0; row < rows; ++row) {
                    for (int chunk = 0; chunk < 32; chunk += 16) {
                        const uint32_t off = (uint32_t)(row * blocks + chunk);
                        if (off < left) EXPECT((uint64_t)at + off + 16 <= bytes);
                        if (at + chunk < blocks) EXPECT(off < left);
                    }
                }
            }
        }
    }
}

}  // namespace

int main()
{
    check_bytes_left();
    check_scale_rows();
    std::printf("%ld checks passed\n", g_checks);
    return 0;
}
