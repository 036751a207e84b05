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

// Largest rows * N of a call: items (tiles of 32 x 64 or more) then count in 32 bits.
constexpr int64_t kMxMaxOutputs = int64_t(1) << 40;

// Items of `tiles` m-tiles of `bm` rows with n_tiles column tiles each.  Experts whose offsets do not
// decrease have at most one partial tile each; a table with more tiles than that decreases somewhere, and
// could count past 32 bits and lead the search for an item outside the output: it gets no items.
__host__ __device__ inline int mx_items(int tiles, int n_tiles, int rows, int bm, int E)
{
    return tiles <= rows / bm + (E < rows ? E : rows) ? tiles * n_tiles : 0;
}

}  // namespace qmoe
