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

__device__ inline uint64_t shfl_xor_u64(uint64_t v, int d)
{
    const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, d, kWave);
    const uint32_t hi = (uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), d, kWave);
    return (uint64_t)hi << 32 | lo;
}

struct Best {
    uint64_t key;
    int index;
};

// The wavefront's largest key, of equal ones the lowest index.
__device__ inline Best wave_best(Best b)
{
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const Best o{shfl_xor_u64(b.key, d), __shfl_xor(b.index, d, kWave)};
        if (o.key > b.key || (o.key == b.key && o.index < b.index)) b = o;
    }
    return b;
}

__device__ inline double wave_sum_f64(double v)
{
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v += __builtin_bit_cast(double, shfl_xor_u64(__builtin_bit_cast(uint64_t, v), d));
    return v;
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

// EPL experts a lane: expert lane + 64 j.
template <int DT, int EPL>
__global__ __launch_bounds__(64 * kWaves) void route_scores_kernel(RouteScoresArgs a)
{
    typedef typename RowType<DT>::Raw Raw;
    __shared__ uint64_t choices[kWaves][EPL * kWave];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= a.T) return;  // the wavefronts of a workgroup do not meet
    const Raw* row = (const Raw*)a.logits + t * a.row_stride;
    float l[EPL];
    float m = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane + kWave * j;
        l[j] = e < a.E ? RowType<DT>::value(row[e]) : -INFINITY;
        m = fmaxf(m, l[j]);
        nan |= l[j] != l[j];
    }
    m = wave_max_f32(m);
    const bool poisoned = !a.sigmoid && (__any(nan) || m == INFINITY);

    double sum = 0.0;
    double score[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        if (a.sigmoid) {
            score[j] = 1.0 / (1.0 + exp(-(double)l[j]));
        } else {
            score[j] = l[j] == -INFINITY ? 0.0 : poisoned ? (double)NAN : exp((double)l[j] - (double)m);
            sum += score[j];
        }
    }
    if (!a.sigmoid) sum = wave_sum_f64(sum);
    uint64_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane + kWave * j;
        if (!a.sigmoid) score[j] /= sum;
        const double c = a.bias && e < a.E ? score[j] + (double)a.bias[e] : score[j];
        key[j] = l[j] == -INFINITY ? 0 : key_of(c);
    }

    if (a.top_groups < a.n_groups) {
        const int size = a.E / a.n_groups;
        for (int j = 0; j < EPL; ++j) choices[wave][lane + kWave * j] = key[j];
        __builtin_amdgcn_wave_barrier();
        // lane g ranks group g
        uint64_t rank = 0;
        if (lane < a.n_groups) {
            uint64_t first = 0, second = 0;
            for (int i = 0; i < size; ++i) {
                const uint64_t k = choices[wave][lane * size + i];
                second = max(second, min(first, k));
                first = max(first, k);
            }
            rank = first;
            if (a.group_top == 2 && second != 0 && first != ~0ull) {
                auto value = [](uint64_t k) { return __builtin_bit_cast(double, k >> 63 ? k & ~(1ull << 63) : ~k); };
                rank = key_of(value(first) + value(second));
            }
        }
        uint64_t open = 0;
        for (int i = 0; i < a.top_groups; ++i) {
            const Best b = wave_best(Best{open >> lane & 1 ? 0 : rank, lane});
            if (b.key == 0) break;
            open |= 1ull << b.index;
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane + kWave * j;
            if (e < a.E && !(open >> (e / size) & 1)) key[j] = 0;
        }
    }

    // slot s is lane s's
    int id = -1;
    float chosen = -INFINITY;  // its logit
    for (int s = 0; s < a.top_k; ++s) {
        Best b{0, a.E};
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            if (key[j] > b.key) b = Best{key[j], lane + kWave * j};
        }
        b = wave_best(b);
        if (b.key == 0) break;
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            if (lane + kWave * j == b.index) {
                key[j] = 0;
                v = l[j];
            }
        }
        v = __shfl(v, b.index % kWave, kWave);
        if (lane == s) {
            id = b.index;
            chosen = v;
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
