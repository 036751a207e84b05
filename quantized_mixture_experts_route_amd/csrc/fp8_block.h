// fp8_block.h -- one block of 128 values in 8-bit floating point (e4m3): the
// scale of its largest magnitude and the codes, shared by the conversions and
// by the activation that quantises what it computes.
//
// The scale is the least power of two s, at least 2^-126, with max |x| <= 448 s
// (448 is e4m3's largest value).  A power of two makes x / s an exact float32
// product (below 2^-126, where it may round, every code is 0 anyway), so a code
// is rounded once; e4m3 being a floating point format, a scale that is up to
// twice larger than max / 448 costs no precision but at the smallest values.
#pragma once

#include "fp8_ops.h"
#include "rowio.h"

namespace qmoe {

__device__ inline uint32_t magnitude_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

// The scale's float32 bits for a block whose largest magnitude has the bits `top` (NaN and infinities
// are the largest patterns): NaN for those.
__device__ inline uint32_t fp8_scale_bits(uint32_t top)
{
    // 448 = 1.75 * 2^8
    const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);
    return top >= 0x7f800000u ? 0x7fc00000u : (uint32_t)max(e, 1) << 23;
}

// 1 / scale of a finite block (its exponent is at most 120).
__device__ inline float fp8_inverse(uint32_t scale_bits)
{
    return __builtin_bit_cast(float, (254u << 23) - scale_bits);
}

// Four values over the scale to four codes, the first in the low byte.
__device__ inline uint32_t fp8_encode4(const float* v, float inv)
{
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, c, true);
    return (uint32_t)c;
}

// Maximum over the 16 lanes of a row; every lane of the row has to take part.
__device__ inline uint32_t row16_max(uint32_t v)
{
    v = max(v, dpp_u32<kDppXor1>(v));
    v = max(v, dpp_u32<kDppXor2>(v));
    v = max(v, dpp_u32<kDppHalfMirror>(v));
    return max(v, dpp_u32<kDppMirror>(v));
}

// 16 lanes with eight values each: a block.  Writes the lane's eight codes to `codes`, and lane 0 of
// the row the scale.  Lanes behind the row's end take part with zeros and `in` false.
__device__ inline void fp8_store_block(const float (&v)[8], bool in, uint8_t* codes, float* scale)
{
    uint32_t top = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) top = max(top, magnitude_bits(v[q]));
    const uint32_t bits = fp8_scale_bits(row16_max(top));
    if (!in) return;
    u32x2 c = {};
    if (bits != 0x7fc00000u) {
        const float inv = fp8_inverse(bits);
        c = u32x2{fp8_encode4(v, inv), fp8_encode4(v + 4, inv)};
    }
    *reinterpret_cast<u32x2*>(codes) = c;
    if ((threadIdx.x & 15) == 0) *scale = __builtin_bit_cast(float, bits);
}

}  // namespace qmoe
