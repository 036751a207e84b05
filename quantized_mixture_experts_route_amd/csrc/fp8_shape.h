// fp8_shape.h -- which form of its kernel a grouped product of e4m3 rows takes,
// apart from the kernel, so that the choice can be checked on the host.  Not
// installed.
#pragma once

#include "mx_shape.h"

namespace qmoe {

// Tile rows x columns and LDS stages; kRows16 and kRows32: 16 x 16 and 16 x 32 with K shared by the
// wavefronts.
enum class Fp8Tile { kRows16, kRows32, k32x64s4, k64x128s3, k128x128s2, k256x256s2 };

// By the tiles that an even spread of the rows over the experts makes (the host knows the offsets' sizes
// only) for 256 CUs, and in the end by the rounds that they take.  Measured in us, inputs out of cache, the
// call's 11 us of host time included:
//                                 rows   32x64   64x128   128x128   256x256
//   E 8, N 4096, K 2048, rows 2     11.7   13.5    14.3     16.5      22.2
//                        rows 8     16.6   13.5    14.6     16.7      22.2
//   E 1, N 4096, K 4096, rows 16    12.0   19.4    22.0     25.4      -
//                        rows 64    -      19.1    22.2     25.4      35.4
//                        rows 256   -      21.0    22.8     27.4      51.3
//                        rows 1024  -      67.0    30.6     29.8      52.0
//                        rows 2048  -      126     54.2     43.8      54.2
//                        rows 4096  -      241     103      79.0      65.3
//   E 1, N 4096, K 14336, rows 16   27.5   51.6    61.0     71.4      -
//   E 1, N 8192, K 8192, rows 256   -      63.6    39.5     47.5      91.9
//   E 8, N 4096, K 4096, rows 32    -      38.1    36.0     37.4      44.6
//                        rows 256   -      47.1    36.1     37.7      46.5
//                        rows 512   -      57.9    47.5     39.7      47.9
//                        rows 1024  -      86.9    59.5     58.9      55.0
//                        rows 2048  -      151     83.5     74.4      64.9
//                        rows 4096  -      273     138      110       111
//   E 128, N 2048, K 768, rows 512  -      47.7    42.1     46.2      50.1
//                         rows 4096 -      63.7    46.2     49.3      53.5
//   E 512, N 1536, K 2048, rows 60  61.3   39.3    36.8     44.2      49.4
// The rows are of kRows32; where its tiles leave half of the CUs without one, kRows16 takes 13.5 us for 18.8 (E 1, N
// 4096, K 14336, one row) and 20.1 for 26.3 (16 rows), and the same at K 2048.
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
