// fp8_shape.h -- which form of its kernel a grouped product of e4m3 rows takes,
// apart from the kernel, so that the choice can be checked on the host.  Not
// installed.
#pragma once

#include "mx_shape.h"

namespace qmoe {

// Tile rows x columns and LDS stages; kRows16 and kRows32: 16 x 16 and 16 x 32 with K shared by the
// wavefronts.
enum class Fp8Tile { kRows16, kRows32, k32x64s4, k64x128s3, k128x128s2, k256x256s2 };

// By the tiles that an even spread of the rows over the experts makes (the host knows the offsets' sizes only)
// for 256 CUs, and in the end by the rounds that they take.  The kernel's time in each form in us, whichever the
// rule takes (the starred), inputs out of cache:
//                                    16x16   16x32   32x64   64x128  128x128  256x256
//   E 8, N 4096, K 2048, rows 2        9.4     8.3*   11.4    13.0     16.0     21.9
//                        rows 8       18.9    19.2    13.8    14.0*    18.5     23.1
//                        rows 1024     215     178    46.6    32.1     32.8*    31.5
//   E 1, N 4096, K 4096, rows 16       9.8*   11.2    16.6    19.0     26.3     35.8
//                        rows 64      23.7    20.3    16.9*   22.4     27.6     36.7
//                        rows 256     84.6    66.5    19.2*   22.2     29.6     50.5
//                        rows 1024     315     250    60.0    34.9     31.6*    52.1
//                        rows 2048       -       -     116    62.6     50.4*    63.4
//                        rows 4096       -       -     224     119     94.4     69.9*
//   E 1, N 4096, K 14336, rows 1      16.7*   21.8    43.5    52.8     81.7      110
//                         rows 16     21.8*   29.0    43.6    53.5     82.3      112
//                         rows 32     36.8    29.4*   43.6    56.4     82.5      112
//                         rows 64     70.1    55.0    44.1*   71.0     82.7      115
//   E 1, N 8192, K 8192, rows 256      302     226    61.7    40.8*    54.0     97.4
//   E 8, N 4096, K 4096, rows 32      34.3    35.1    34.4    34.9*    36.8     44.2
//                        rows 256     94.9    81.8    40.5    35.4*    37.0     45.7
//                        rows 512      174     141    54.7    46.0     38.5*    46.9
//                        rows 1024     336     269    85.4    58.3     59.4*    55.4
//                        rows 2048       -       -     143    82.5     78.0     68.3*
//                        rows 4096       -       -     260     135      115*     113
//   E 8, N 8192, K 1040, rows 8192       -       -     449     199      152      126*
//   E 128, N 2048, K 768, rows 512     122     114    45.6    41.4*    45.6     50.0
//                         rows 4096      -       -    60.5    45.2*    47.9     54.0
//   E 512, N 1536, K 2048, rows 60    62.9    62.4    38.7    38.0*    44.7     49.8
// A round of 256 x 256 (one a CU) takes about 1.6 times as long as one of 128 x 128 (two a CU), for twice
// the work.
inline Fp8Tile fp8_tile(int E, int N, int rows)
{
    const int64_t experts = E < rows ? E : rows;
    const int64_t mean = rows / experts;
    auto tiles = [&](int bm, int bn) {  // of several experts, each one's last tile counts half
        const int64_t m = experts == 1 ? (rows + bm - 1) / bm : mean < bm ? experts : rows / bm + (experts + 1) / 2;
        return m * ((N + bn - 1) / bn);
    };
    if (tiles(16, 32) <= kMxCUs / 2) return Fp8Tile::kRows16;
    if (tiles(16, 32) <= kMxCUs) return Fp8Tile::kRows32;
    if (tiles(64, 128) <= kMxCUs / 2) return Fp8Tile::k32x64s4;
    if (mean <= 32 || tiles(64, 128) <= kMxCUs) return Fp8Tile::k64x128s3;
    const int64_t middle_rounds = (tiles(128, 128) + 2 * kMxCUs - 1) / (2 * kMxCUs);
    const int64_t large_rounds = (tiles(256, 256) + kMxCUs - 1) / kMxCUs;
    return 8 * large_rounds > 5 * middle_rounds ? Fp8Tile::k128x128s2 : Fp8Tile::k256x256s2;
}

}  // namespace qmoe
