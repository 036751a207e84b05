// mx_shape_check.cpp -- the arithmetic that the grouped MXFP4 product shares
// with its launch (csrc/mx_shape.h), checked on the host under
// AddressSanitizer and UndefinedBehaviorSanitizer.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>

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

// Tables that do not decrease keep all their items; any table's items, and the products of a tile index
// with the column tiles that the search forms, count in 32 bits.
void check_items()
{
    const int tile[][2] = {{32, 64}, {64, 128}, {128, 128}, {256, 256}};
    uint32_t seed = 1;
    auto next = [&](uint32_t n) { return (seed = seed * 1664525u + 1013904223u) / 65536u % n; };
    for (auto& t : tile) {
        const int bm = t[0], bn = t[1];
        for (int rows : {1, 31, 32, 33, 4096, 65536, (1 << 24) - 1}) {
            for (int E : {1, 2, 7, 64, 1024}) {
                int64_t N = qmoe::kMxMaxOutputs / rows;
                if (N > 1 << 20) N = 1 << 20;
                const int n_tiles = (int)((N + bn - 1) / bn);
                int at = 0, tiles = 0;  // a random table that does not decrease
                for (int e = 0; e < E; ++e) {
                    const int to = e == E - 1 ? rows : at + (int)next((uint32_t)(rows - at) / 2 + 2);
                    const int end = to < rows ? to : rows;
                    tiles += (end - at + bm - 1) / bm;
                    at = end;
                }
                EXPECT(qmoe::mx_items(tiles, n_tiles, rows, bm, E) == tiles * n_tiles);
                EXPECT((int64_t)tiles * n_tiles <= INT32_MAX);
                // every second expert with all the rows, the table falling back in between
                const int64_t worst = (int64_t)(E + 1) / 2 * ((rows + bm - 1) / bm);
                const int got = qmoe::mx_items((int)worst, n_tiles, rows, bm, E);
                EXPECT(got >= 0 && (got == 0 || got == worst * n_tiles));
            }
        }
    }
}

// Lines "E N K rows": the tile, whether scales take the direct path (aligned), whether a half group ends it.
void answer_forms()
{
    static const char* const names[] = {"32x64s4", "64x128s4", "128x128s4", "64x128s2", "128x128s2", "256x256s2"};
    int E, N, K, rows;
    while (std::scanf("%d %d %d %d", &E, &N, &K, &rows) == 4) {
        const char* name = names[(int)qmoe::mx_tile(E, N, K, rows)];
        const int stages = name[std::strlen(name) - 1] - '0';
        std::printf("%s %s %s\n", name, qmoe::mx_whole(stages, K, nullptr, nullptr) ? "direct" : "registers",
                    qmoe::mx_half_group(stages, K) ? "half" : "full");
    }
}

}  // namespace

int main(int argc, char**)
{
    if (argc > 1) {
        answer_forms();
        return 0;
    }
    check_items();
    check_bytes_left();
    check_scale_rows();
    std::printf("%ld checks passed\n", g_checks);
    return 0;
}
