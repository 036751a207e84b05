// rowio.h -- row access shared by the kernels that move or convert rows of
// any width: element types and vectors of V consecutive elements at element
// alignment (the target loads 16 bytes from any address).
#pragma once

#include "qmoe_device.h"

namespace qmoe {

enum : int { kF32 = 3 };  // beside kF16 and kBF16: rows in float32

// `Raw` is the element's bit pattern; value() and round() convert it.
template <int DT>
struct RowType {
    typedef uint16_t Raw;
    __device__ static inline float value(Raw x) { return Dt<DT>::to_float(x); }
    __device__ static inline Raw round(float x) { return Dt<DT>::from_float(x); }
};
template <>
struct RowType<kF32> {
    typedef float Raw;
    __device__ static inline float value(Raw x) { return x; }
    __device__ static inline Raw round(float x) { return x; }
};

// Rows of whole 16-byte vectors need no aligned start: a row of at least V
// elements is covered by vectors at 0, V, 2V, ... whose last one is moved
// back to end with the row (the elements two vectors share get the same value
// from both).  Rows shorter than V take V = 1.
template <class Raw, int V>
struct RowVec {
    Raw v[V];
};

template <class Raw, int V>
__device__ inline RowVec<Raw, V> load_vec(const Raw* p)
{
    RowVec<Raw, V> x;
    __builtin_memcpy(&x, p, sizeof x);
    return x;
}

template <class Raw, int V>
__device__ inline void store_vec(Raw* p, const RowVec<Raw, V>& x)
{
    __builtin_memcpy(p, &x, sizeof x);
}

template <int V>
__host__ __device__ inline int row_vecs(int H)
{
    return (H + V - 1) / V;
}

// First element of vector i of a row of H elements.
template <int V>
__device__ inline int vec_start(int i, int H)
{
    const int h = i * V;
    return V == 1 || h + V <= H ? h : H - V;
}

}  // namespace qmoe
