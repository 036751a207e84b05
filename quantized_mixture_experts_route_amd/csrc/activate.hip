// activate.hip -- the gated activation of a projection's outputs, and its
// gradient.  With g a gate and u its linear part,
//   SwiGLU: out = g' s(alpha g') (u' + beta), g' = min(g, limit), u' = u within
//           +-limit, s the logistic function
//   GeGLU:  out = g s(w) u with w = 2 sqrt(2/pi) (g + 0.044715 g^3), which is
//           tanh-GELU, since 0.5 (1 + tanh x) = s(2x)
// and with d the gradient of out
//   SwiGLU: to u: d g' s  (0 where the limit cut u)
//           to g: d (u' + beta) s (1 + z (1 - s)), z = alpha g'  (0 where it cut g)
//   GeGLU:  to u: d g s;  to g: d u s (1 + g w' (1 - s)), w' = dw/dg
// in float32, rounded once.  NaN passes through.
//
// Every value is read and written once, with some 20 to 40 operations for each
// output: bound by HBM (8192 rows of 2 x 14336 bf16: 138 us, 5.1 TB/s, what a copy
// reaches; straight to 8 bits 154, 3.8 TB/s, with codes for half of the bytes and
// the same operations; the gradient 205, 5.7 TB/s), small calls by the launch
// (3.2 us of the GPU).  Eight outputs a thread: 16 bytes a load and store, and 16
// threads are a block of 128, whose maximum stays within a row of lanes.
#include <algorithm>

#include "fp8_block.h"
#include "logistic.h"
#include "qmoe_internal.h"

namespace qmoe {
namespace {

constexpr int kThreads = 256;

struct Pair {
    float gate, up;
};

template <bool GEGLU>
struct Gate {
    float s, rest;   // s(z), 1 - s(z)
    float slope;     // z (1 - s) / (1 - s): alpha g', or g w'
    float g;         // g'
};

// z finite for every g that is not NaN, so that s (1 + z (1 - s)) has no 0 * inf.
template <bool GEGLU>
__device__ inline Gate<GEGLU> gate_of(float g, const ActivateArgs& a)
{
    Gate<GEGLU> r;
    if constexpr (GEGLU) {
        constexpr float c = 1.5957691216057308f;  // 2 sqrt(2/pi)
        // behind +-16 s is 0 or 1 to float32 and its slope 0
        const float h = g > 16.0f ? 16.0f : g < -16.0f ? -16.0f : g;
        const float h2 = h * h;
        const Logistic l = logistic(c * h * fmaf(0.044715f, h2, 1.0f));
        r.s = l.s;
        r.rest = l.rest;
        r.slope = c * h * fmaf(3.0f * 0.044715f, h2, 1.0f);
        r.g = g;
    } else {
        r.g = g > a.limit ? a.limit : g;
        float z = a.alpha * r.g;
        z = z > 200.0f ? 200.0f : z < -200.0f ? -200.0f : z;  // s is 0 or 1 there
        const Logistic l = logistic(z);
        r.s = l.s;
        r.rest = l.rest;
        r.slope = z;
    }
    return r;
}

template <bool GEGLU>
__device__ inline float linear_of(float u, const ActivateArgs& a)
{
    if constexpr (GEGLU) return u;
    return (u > a.limit ? a.limit : u < -a.limit ? -a.limit : u) + a.beta;
}

template <bool GEGLU>
__device__ inline float activated(float g, float u, const ActivateArgs& a)
{
    const auto t = gate_of<GEGLU>(g, a);
    return t.g * t.s * linear_of<GEGLU>(u, a);
}

template <bool GEGLU>
__device__ inline Pair gradient(float d, float g, float u, const ActivateArgs& a)
{
    const auto t = gate_of<GEGLU>(g, a);
    Pair r;
    r.up = d * (t.g * t.s);
    const float lin = linear_of<GEGLU>(u, a), slope = t.s * fmaf(t.slope, t.rest, 1.0f);
    // d lin may leave float32's range where the slope, at most 1.13 and often next to 0, brings it back
    const float to = d * lin;
    r.gate = fabsf(to) == INFINITY ? d * slope * lin : to * slope;
    if constexpr (!GEGLU) {
        if (u > a.limit || u < -a.limit) r.up = 0.0f;
        if (g > a.limit) r.gate = 0.0f;
    }
    return r;
}

// V gates and their linear parts from column j on.
template <int DT, bool HALVES, int V>
__device__ inline void load_pairs(const typename RowType<DT>::Raw* y, int I, int j, float (&g)[V], float (&u)[V])
{
    typedef typename RowType<DT>::Raw Raw;
    if constexpr (HALVES) {
        const auto a = load_vec<Raw, V>(y + j), b = load_vec<Raw, V>(y + I + j);
#pragma unroll
        for (int q = 0; q < V; ++q) {
            g[q] = RowType<DT>::value(a.v[q]);
            u[q] = RowType<DT>::value(b.v[q]);
        }
    } else {
        const auto a = load_vec<Raw, 2 * V>(y + 2 * (int64_t)j);
#pragma unroll
        for (int q = 0; q < V; ++q) {
            g[q] = RowType<DT>::value(a.v[2 * q]);
            u[q] = RowType<DT>::value(a.v[2 * q + 1]);
        }
    }
}

// V outputs a thread; a row's last vector ends with the row (rowio.h).
template <int DT, bool GEGLU, bool HALVES, int V>
__global__ __launch_bounds__(kThreads) void activate_kernel(ActivateArgs a, int64_t vecs)
{
    typedef typename RowType<DT>::Raw Raw;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < vecs; i += (int64_t)gridDim.x * kThreads) {
        const int per_row = row_vecs<V>(a.I);
        const int64_t row = i / per_row;
        const int j = vec_start<V>((int)(i - row * per_row), a.I);
        float g[V], u[V];
        load_pairs<DT, HALVES, V>((const Raw*)a.y + row * a.row_stride, a.I, j, g, u);
        RowVec<Raw, V> out;
#pragma unroll
        for (int q = 0; q < V; ++q) out.v[q] = RowType<DT>::round(activated<GEGLU>(g[q], u[q], a));
        store_vec<Raw, V>((Raw*)a.out + row * a.I + j, out);
    }
}

// Eight outputs a thread, 16 threads a block of 128.
template <int DT, bool GEGLU, bool HALVES>
__global__ __launch_bounds__(kThreads) void activate_fp8_kernel(ActivateArgs a, int64_t threads, int blocks)
{
    typedef typename RowType<DT>::Raw Raw;
    // a multiple of 16: a block's threads stay together
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < threads; i += (int64_t)gridDim.x * kThreads) {
        const int64_t block = i >> 4, row = block / blocks;
        const int j = (int)(block - row * blocks) * kFp8Block + (int)(i & 15) * 8;
        const bool in = j < a.I;
        float v[8] = {};
        if (in) {
            float g[8], u[8];
            load_pairs<DT, HALVES, 8>((const Raw*)a.y + row * a.row_stride, a.I, j, g, u);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = activated<GEGLU>(g[q], u[q], a);
        }
        fp8_store_block(v, in, a.codes + row * a.I + j, a.scales + block);
    }
}

template <int DT, bool GEGLU, bool HALVES, int V>
__global__ __launch_bounds__(kThreads) void activate_backward_kernel(ActivateArgs a, int64_t vecs)
{
    typedef typename RowType<DT>::Raw Raw;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < vecs; i += (int64_t)gridDim.x * kThreads) {
        const int per_row = row_vecs<V>(a.I);
        const int64_t row = i / per_row;
        const int j = vec_start<V>((int)(i - row * per_row), a.I);
        float g[V], u[V];
        load_pairs<DT, HALVES, V>((const Raw*)a.y + row * a.row_stride, a.I, j, g, u);
        const auto d = load_vec<Raw, V>((const Raw*)a.grad + row * a.grad_stride + j);
        Raw* to = (Raw*)a.grad_y + row * 2 * a.I;
        Raw gate[V], up[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
            const Pair p = gradient<GEGLU>(RowType<DT>::value(d.v[q]), g[q], u[q], a);
            gate[q] = RowType<DT>::round(p.gate);
            up[q] = RowType<DT>::round(p.up);
        }
        if constexpr (HALVES) {
            RowVec<Raw, V> x, z;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                x.v[q] = gate[q];
                z.v[q] = up[q];
            }
            store_vec<Raw, V>(to + j, x);
            store_vec<Raw, V>(to + a.I + j, z);
        } else {
            RowVec<Raw, 2 * V> x;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                x.v[2 * q] = gate[q];
                x.v[2 * q + 1] = up[q];
            }
            store_vec<Raw, 2 * V>(to + 2 * (int64_t)j, x);
        }
    }
}

// A launch has fewer than 2^32 threads; those of more run through several items.
unsigned blocks_for(int64_t n) { return (unsigned)std::min((n + kThreads - 1) / kThreads, int64_t(1) << 23); }

// go(dtype, geglu, halves) with each as a constant.
template <class Go>
void by_form(const ActivateArgs& a, Go go)
{
    auto layout = [&](auto dt, auto geglu) {
        if (a.halves) go(dt, geglu, std::true_type{});
        else go(dt, geglu, std::false_type{});
    };
    auto gate = [&](auto dt) {
        if (a.geglu) layout(dt, std::true_type{});
        else layout(dt, std::false_type{});
    };
    if (a.dtype == kF32) gate(std::integral_constant<int, kF32>{});
    else if (a.dtype == kBF16) gate(std::integral_constant<int, kBF16>{});
    else gate(std::integral_constant<int, kF16>{});
}

}  // namespace

hipError_t launch_activate(const ActivateArgs& a, hipStream_t s)
{
    by_form(a, [&](auto dt, auto geglu, auto halves) {
        constexpr int DT = decltype(dt)::value;
        constexpr bool G = decltype(geglu)::value, H = decltype(halves)::value;
        if (a.codes) {
            const int blocks = (a.I + kFp8Block - 1) / kFp8Block;
            const int64_t threads = a.rows * blocks * 16;
            launch(activate_fp8_kernel<DT, G, H>, dim3(blocks_for(threads)), dim3(kThreads), s, a, threads, blocks);
        } else if (a.I >= 8) {
            const int64_t vecs = a.rows * row_vecs<8>(a.I);
            launch(activate_kernel<DT, G, H, 8>, dim3(blocks_for(vecs)), dim3(kThreads), s, a, vecs);
        } else {
            const int64_t vecs = a.rows * a.I;
            launch(activate_kernel<DT, G, H, 1>, dim3(blocks_for(vecs)), dim3(kThreads), s, a, vecs);
        }
    });
    return hipGetLastError();
}

hipError_t launch_activate_backward(const ActivateArgs& a, hipStream_t s)
{
    by_form(a, [&](auto dt, auto geglu, auto halves) {
        constexpr int DT = decltype(dt)::value;
        constexpr bool G = decltype(geglu)::value, H = decltype(halves)::value;
        if (a.I >= 8) {
            const int64_t vecs = a.rows * row_vecs<8>(a.I);
            launch(activate_backward_kernel<DT, G, H, 8>, dim3(blocks_for(vecs)), dim3(kThreads), s, a, vecs);
        } else {
            const int64_t vecs = a.rows * a.I;
            launch(activate_backward_kernel<DT, G, H, 1>, dim3(blocks_for(vecs)), dim3(kThreads), s, a, vecs);
        }
    });
    return hipGetLastError();
}

}  // namespace qmoe
