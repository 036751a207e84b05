// mx_shape.h -- plain arithmetic of the grouped MXFP4 product that its kernel
// and its launch share with the checks on the host.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmoe {

// A byte offset behind every buffer (buffers are shorter than 2^31 bytes).
constexpr uint32_t kMxOutside = 0x80000000u;

// Bytes of a buffer of `bytes` that are left from byte `at` on.  A load's descriptor starts at its
// step's first byte and holds these, so the hardware compares a lane's whole remaining offset with
// what is left, and a step behind the buffer's end, or of no tile, reads nothing: with the step in the
// instruction's scalar offset this would hang on whether and how that offset enters the comparison.
// Both are below 2^31, so their difference has a sign, and the scalar units can do all of it.
__host__ __device__ inline uint32_t mx_bytes_left(uint32_t bytes, uint32_t at)
{
    const int32_t left = (int32_t)(bytes - at);
    return left > 0 ? (uint32_t)left : 0u;
}

}  // namespace qmoe
