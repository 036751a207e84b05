// route_scores.hip -- the experts of each token by softmax or sigmoid scores,
// with a bias that takes part in the choice alone and with groups of experts,
// and the gradient of the weights.
//
// With l a token's logits: s = softmax(l) or sigmoid(l), choice c = s + bias.  A
// group's rank is the sum of its best one or two choices; of the top_groups best
// groups the top_k largest choices are taken, ties to the lower index.  Weights
// are s at the chosen experts, divided by their sum (normalize), times scale.
//
// Choices are compared in float64: two experts whose choices differ by less than
// float32 tells apart would change places from one implementation to the next,
// and with them whole rows of the layer's output.
//
// Gradient, with G the gradient of the weights times scale and w the weights
// before scale:
//   sigmoid:               dl = G s (1 - s)
//   sigmoid, normalised:   dl = w (G - sum G w) (1 - s)
//   softmax:               dl = s (G - sum G s), every expert (G 0 where not chosen)
//   softmax, normalised:   dl = w (G - sum G w), the chosen experts
#include "fp8_ops.h"
#include "qmoe_internal.h"
#include "rowio.h"

namespace qmoe {
namespace {

constexpr int kWaves = 4;  // tokens a workgroup

// Doubles as integers of the same order: 0 for a masked expert (-inf), the largest for NaN; -0 as 0.
__device__ inline uint64_t key_of(double c)
{
    if (c != c) return ~0ull;
    if (c == -INFINITY) return 0;
    const uint64_t b = __builtin_bit_cast(uint64_t, c + 0.0);
    return b >> 63 ? ~b : b | 1ull << 63;
}

__device__ inline double value_of(uint64_t key)
{
    return __builtin_bit_cast(double, key >> 63 ? key & ~(1ull << 63) : ~key);
}

__device__ inline double wave_sum_f64(double v)
{
    auto plus = [](double x, uint64_t o) { return x + __builtin_bit_cast(double, o); };
    v = plus(v, dpp_u64<kDppXor1>(__builtin_bit_cast(uint64_t, v)));
    v = plus(v, dpp_u64<kDppXor2>(__builtin_bit_cast(uint64_t, v)));
    v = plus(v, dpp_u64<kDppHalfMirror>(__builtin_bit_cast(uint64_t, v)));
    v = plus(v, dpp_u64<kDppMirror>(__builtin_bit_cast(uint64_t, v)));
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return plus(__builtin_bit_cast(double, readlane_u64(b, 0)), readlane_u64(b, 16)) +
           plus(__builtin_bit_cast(double, readlane_u64(b, 32)), readlane_u64(b, 48));
}

// The largest two keys of two pairs.
struct Two {
    uint64_t first, second;
};

__device__ inline Two merge(Two a, Two b)
{
    const bool swap = b.first > a.first;
    return Two{swap ? b.first : a.first, max_u64(swap ? a.first : b.first, swap ? b.second : a.second)};
}

// A group's rank as a key: the sum of its best one or two choices; 0 where all are masked.
__device__ inline uint64_t rank_of(Two t, int group_top)
{
    if (group_top == 1 || t.second == 0 || t.first == ~0ull) return t.first;
    return key_of(value_of(t.first) + value_of(t.second));
}

// The lane that holds the wavefront's largest key, the lowest of several (all of its bits: the high words
// first, the low ones only where those tie); -1: no key is left.
__device__ inline int wave_best(uint64_t key)
{
    const uint32_t hi = (uint32_t)(key >> 32), top = wave_max_u32(hi);
    if (top == 0) return -1;  // only a masked choice's key has a high word of 0
    uint64_t holders = __ballot(hi == top);
    if (holders & (holders - 1)) {
        const uint32_t lo = hi == top ? (uint32_t)key : 0u, low = wave_max_u32(lo);
        holders = __ballot(hi == top && lo == low);
    }
    return __builtin_ctzll(holders);
}

// Sum over the chosen slots (lanes), in a fixed order.
__device__ inline float sum_slots(float v) { return wave_sum_f32(v); }

// exp(-|l|), and the logistic function and its rest from it.
__device__ inline float logistic_of(float l)
{
    const float e = expf(-fabsf(l));
    return (l >= 0.0f ? 1.0f : e) / (1.0f + e);
}

// A lane's chosen expert's score over the largest of the chosen (m their largest logit), from logits so
// far below 0 too that every score is 0 to float32: sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)).
__device__ inline float relative_score(bool sigmoid, float l, float m)
{
    if (!sigmoid) return expf(l - m);
    return expf(fminf(l, 0.0f) - fminf(m, 0.0f)) * ((1.0f + expf(-fabsf(m))) / (1.0f + expf(-fabsf(l))));
}

// One wavefront a token, EPL neighbouring experts a lane: EPL * lane + j, so that the lowest lane of several
// holds the lowest index.
//
// What bounds it: a chain of wavefront maxima, one for each slot, behind a float64 score for each expert.  TODO
template <int DT, int EPL>
__global__ __launch_bounds__(64 * kWaves) void route_scores_kernel(RouteScoresArgs a)
{
    typedef typename RowType<DT>::Raw Raw;
    __shared__ uint64_t choices[kWaves][EPL * kWave];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= a.T) return;  // the wavefronts of a workgroup do not meet
    const Raw* row = (const Raw*)a.logits + t * a.row_stride;
    const int e0 = lane * EPL;
    float l[EPL], bias[EPL] = {};
    if (e0 + EPL <= a.E) {
        const auto x = load_vec<Raw, EPL>(row + e0);
#pragma unroll
        for (int j = 0; j < EPL; ++j) l[j] = RowType<DT>::value(x.v[j]);
        if (a.bias) {
            const auto b = load_vec<float, EPL>(a.bias + e0);
#pragma unroll
            for (int j = 0; j < EPL; ++j) bias[j] = b.v[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            l[j] = e0 + j < a.E ? RowType<DT>::value(row[e0 + j]) : -INFINITY;
            if (a.bias && e0 + j < a.E) bias[j] = a.bias[e0 + j];
        }
    }
    float m = -INFINITY;
    double sum = 1.0;
    bool poisoned = false;
    double score[EPL];
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) score[j] = 1.0 / (1.0 + exp(-(double)l[j]));
    } else {
        bool nan = false;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            m = fmaxf(m, l[j]);
            nan |= l[j] != l[j];
        }
        m = wave_max_f32(m);
        poisoned = __any(nan) || m == INFINITY;
        double part = 0.0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            score[j] = l[j] == -INFINITY ? 0.0 : poisoned ? (double)NAN : exp((double)l[j] - (double)m);
            part += score[j];
        }
        sum = wave_sum_f64(part);
#pragma unroll
        for (int j = 0; j < EPL; ++j) score[j] /= sum;
    }
    uint64_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = l[j] == -INFINITY ? 0 : key_of(score[j] + (double)bias[j]);

    if (a.top_groups < a.n_groups) {
        const int size = a.E / a.n_groups, lanes = size / EPL;
        if (size % EPL == 0 && (lanes & (lanes - 1)) == 0) {
            // a group is `lanes` neighbouring lanes, a power of two of them
            Two best{key[0], 0};
#pragma unroll
            for (int j = 1; j < EPL; ++j) best = merge(best, Two{key[j], 0});
            if (lanes > 1) best = merge(best, Two{dpp_u64<kDppXor1>(best.first), dpp_u64<kDppXor1>(best.second)});
            if (lanes > 2) best = merge(best, Two{dpp_u64<kDppXor2>(best.first), dpp_u64<kDppXor2>(best.second)});
            if (lanes > 4) best = merge(best, Two{dpp_u64<kDppHalfMirror>(best.first), dpp_u64<kDppHalfMirror>(best.second)});
            if (lanes > 8) best = merge(best, Two{dpp_u64<kDppMirror>(best.first), dpp_u64<kDppMirror>(best.second)});
            for (int d = 16; d < lanes; d <<= 1) {
                best = merge(best, Two{(uint64_t)__shfl_xor((unsigned long long)best.first, d, kWave),
                                       (uint64_t)__shfl_xor((unsigned long long)best.second, d, kWave)});
            }
            const uint64_t rank = rank_of(best, a.group_top);
            int before = 0;  // groups ahead of the lane's
            for (int g = 0; g < a.n_groups; ++g) {
                const uint64_t other = readlane_u64(rank, g * lanes);
                before += other > rank || (other == rank && g * lanes < lane / lanes * lanes);
            }
            if (before >= a.top_groups || rank == 0) {
#pragma unroll
                for (int j = 0; j < EPL; ++j) key[j] = 0;
            }
        } else {
#pragma unroll
            for (int j = 0; j < EPL; ++j) choices[wave][e0 + j] = key[j];
            __builtin_amdgcn_wave_barrier();
            Two best{0, 0};  // lane g's group is g
            if (lane < a.n_groups) {
                for (int i = 0; i < size; ++i) best = merge(best, Two{choices[wave][lane * size + i], 0});
            }
            const uint64_t rank = rank_of(best, a.group_top);
            int before = 0;
            for (int g = 0; g < a.n_groups; ++g) {
                const uint64_t other = readlane_u64(rank, g);
                before += other > rank || (other == rank && g < lane);
            }
            const uint64_t open = __ballot(lane < a.n_groups && before < a.top_groups && rank != 0);
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                if (e0 + j < a.E && !(open >> ((e0 + j) / size) & 1)) key[j] = 0;
            }
        }
    }

    // slot s is lane s's
    int id = -1;
    float chosen = -INFINITY;  // its logit
    for (int s = 0; s < a.top_k; ++s) {
        uint64_t best = key[0];
        int at = 0;
        float logit = l[0];
#pragma unroll
        for (int j = 1; j < EPL; ++j) {
            if (key[j] > best) {
                best = key[j];
                at = j;
                logit = l[j];
            }
        }
        const int from = wave_best(best);
        if (from < 0) break;
        const int e = from * EPL + __builtin_amdgcn_readlane(at, from);
        const float v = readlane_f32(logit, from);
        if (lane == s) {
            id = e;
            chosen = v;
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            if (e0 + j == e) key[j] = 0;
        }
    }
    float w = 0.0f;
    if (a.normalize) {
        const float top = wave_max_f32(chosen);  // NaN compares false and is skipped
        const float r = id < 0 ? 0.0f : relative_score(a.sigmoid, chosen, top);
        const float total = sum_slots(r);
        if (id >= 0) w = r / total;
    } else if (id >= 0) {
        w = a.sigmoid ? logistic_of(chosen) : expf(chosen - m) / (float)sum;
    }
    if (poisoned && id >= 0) w = NAN;
    if (lane < a.top_k) {
        a.ids[t * a.top_k + lane] = id;
        a.weights[t * a.top_k + lane] = w * a.scale;
    }
}

template <int DT, int EPL>
__global__ __launch_bounds__(64 * kWaves) void route_scores_backward_kernel(RouteScoresArgs a)
{
    typedef typename RowType<DT>::Raw Raw;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= a.T) return;
    const Raw* row = (const Raw*)a.logits + t * a.row_stride;
    float l[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane + kWave * j;
        l[j] = e < a.E ? RowType<DT>::value(row[e]) : -INFINITY;
    }
    // slot s is lane s's: its expert, logit and gradient
    int id = -1;
    float g = 0.0f, chosen = -INFINITY;
    if (lane < a.top_k) {
        id = a.ids[t * a.top_k + lane];
        if ((uint32_t)id >= (uint32_t)a.E) id = -1;
        if (id >= 0) chosen = RowType<DT>::value(row[id]);
        if (chosen == -INFINITY) id = -1;
        if (id >= 0) g = a.grad_weights[t * a.top_k + lane] * a.scale;
    }
    float to_slot = g;      // the gradient that reaches the slot's logit
    float mean = 0.0f;      // softmax: sum G s
    float m = -INFINITY, total = 1.0f;
    if (a.normalize) {
        const float top = wave_max_f32(chosen);
        const float r = id < 0 ? 0.0f : relative_score(a.sigmoid, chosen, top);
        const float sum = sum_slots(r);
        const float w = id < 0 ? 0.0f : r / sum;
        const float centre = sum_slots(id < 0 ? 0.0f : g * w);
        to_slot = id < 0 ? 0.0f : w * (g - centre) * (a.sigmoid ? logistic_of(-chosen) : 1.0f);
    } else if (a.sigmoid) {
        to_slot = id < 0 ? 0.0f : g * (logistic_of(chosen) * logistic_of(-chosen));
    } else {
        bool nan = false;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            m = fmaxf(m, l[j]);
            nan |= l[j] != l[j];
        }
        m = __any(nan) ? NAN : wave_max_f32(m);
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) part += l[j] == -INFINITY ? 0.0f : expf(l[j] - m);
        total = wave_sum_f32(part);
        mean = sum_slots(id < 0 ? 0.0f : g * (expf(chosen - m) / total));
    }
    float out[EPL] = {};
    for (int s = 0; s < a.top_k; ++s) {
        const int e = __builtin_amdgcn_readlane(id, s);
        const float v = readlane_f32(to_slot, s);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            if (lane + kWave * j == e) out[j] += v;
        }
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane + kWave * j;
        if (e >= a.E) continue;
        if (!a.sigmoid && !a.normalize) out[j] = l[j] == -INFINITY ? 0.0f : expf(l[j] - m) / total * (out[j] - mean);
        ((Raw*)a.grad_logits)[t * a.E + e] = RowType<DT>::round(out[j]);
    }
}

// go(dtype, experts a lane) with each as a constant.
template <class Go>
void by_size(const RouteScoresArgs& a, Go go)
{
    auto size = [&](auto dt) {
        if (a.E <= 64) go(dt, std::integral_constant<int, 1>{});
        else if (a.E <= 128) go(dt, std::integral_constant<int, 2>{});
        else if (a.E <= 256) go(dt, std::integral_constant<int, 4>{});
        else if (a.E <= 512) go(dt, std::integral_constant<int, 8>{});
        else go(dt, std::integral_constant<int, 16>{});
    };
    if (a.dtype == kF32) size(std::integral_constant<int, kF32>{});
    else if (a.dtype == kBF16) size(std::integral_constant<int, kBF16>{});
    else size(std::integral_constant<int, kF16>{});
}

}  // namespace

hipError_t launch_route_scores(const RouteScoresArgs& a, hipStream_t s)
{
    by_size(a, [&](auto dt, auto epl) {
        launch(route_scores_kernel<decltype(dt)::value, decltype(epl)::value>, dim3((unsigned)((a.T + kWaves - 1) / kWaves)),
               dim3(64 * kWaves), s, a);
    });
    return hipGetLastError();
}

hipError_t launch_route_scores_backward(const RouteScoresArgs& a, hipStream_t s)
{
    by_size(a, [&](auto dt, auto epl) {
        launch(route_scores_backward_kernel<decltype(dt)::value, decltype(epl)::value>,
               dim3((unsigned)((a.T + kWaves - 1) / kWaves)), dim3(64 * kWaves), s, a);
    });
    return hipGetLastError();
}

}  // namespace qmoe
