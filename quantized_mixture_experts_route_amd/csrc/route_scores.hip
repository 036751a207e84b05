// route_scores.hip -- the experts of each token by softmax or sigmoid scores,
// with a bias that takes part in the choice alone and with groups of experts,
// and the gradient of the weights.
//
// With l a token's logits: s = softmax(l) or sigmoid(l), choice c = s + bias.  A
// group's rank is the sum of its best one or two choices; of the top_groups best
// groups the top_k largest choices are taken, ties to the lower index.  Weights
// are s at the chosen experts, divided by their sum (normalize), times scale.
//
// Choices are ordered as in float64 (in float32 first, again in float64 where that
// is too near to tell): two experts whose choices differ by less than float32 tells
// apart would change places from one implementation to the next, and with them
// whole rows of the layer's output.
//
// Gradient, with G the gradient of the weights times scale and w the weights
// before scale:
//   sigmoid:               dl = G s (1 - s)
//   sigmoid, normalised:   dl = w (G - sum G w) (1 - s)
//   softmax:               dl = s (G - sum G s), every expert (G 0 where not chosen)
//   softmax, normalised:   dl = w (G - sum G w), the chosen experts
#include "fp8_ops.h"
#include "logistic.h"
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

// The same for floats, -inf and all (no NaN); -0 as 0.
__device__ inline uint32_t ordered(float c)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, c + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ inline float float_of(uint32_t key)
{
    return __builtin_bit_cast(float, key ^ ((int32_t)key < 0 ? 0x80000000u : ~0u));
}

// Maximum of a wavefront's floats without NaN: as integers it takes a DPP operation a step, where one of floats
// that keeps -0 and NaN in their places takes four.
__device__ inline float wave_largest(float v) { return float_of(wave_max_u32(ordered(v))); }

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

// A lane's chosen expert's score over the largest of the chosen (m their largest logit), from logits so
// far below 0 too that every score is 0 to float32: sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)).
__device__ inline float relative_score(bool sigmoid, float l, float m)
{
    if (!sigmoid) return exp_of(l - m);
    return exp_of(fminf(l, 0.0f) - fminf(m, 0.0f)) * ((1.0f + exp_minus(fabsf(m))) / (1.0f + exp_minus(fabsf(l))));
}

// ---------------------------------------------------------------- the choice
// One wavefront a token, EPL neighbouring experts a lane: EPL * lane + j, so that the lowest lane of several
// holds the lowest index.  Both forms leave slot s's expert in lane s (-1: none is left).

// Choices in float32, and float64 where they come too near one another.  A word holds a choice's bits in their
// order, the last log2(EPL) of them replaced by the expert's place in its lane, so that a lane sorts its words by
// minima and maxima alone.  In units u of 2^-24: a score in float32 is off by 8 u of it (sigmoid) or 30 u of 1
// (softmax: the sum's rounding, and that of l - m, which keeps the order and whose mean over the scores is below
// log E), its sum with a bias by one u of that, and the place by up to 30 u, downwards.  So two choices differ in
// float64 as they do here if they are further apart than 60 u + 32 u (|c| + |d|), without a bias 46 u |c|; kNear
// is 64 u.  Choices in a chain of near ones, which may reach past the last slot, are put in order by their float64
// values, one a lane, equal ones by their index.  False where that does not do: groups that near one another at
// the last place or whose ranks leave float32's range, near choices by softmax with a bias (their sum over all
// experts counts), groups of other sizes.
constexpr float kNear = 0x1p-18f;

template <int EPL>
__device__ inline float value32(uint32_t key)
{
    return float_of(key & ~(uint32_t)(EPL - 1));
}

struct Two32 {
    uint32_t first, second;
};

__device__ inline Two32 merge(Two32 a, Two32 b)
{
    return Two32{max(a.first, b.first), max(min(a.first, b.first), max(a.second, b.second))};
}

template <int CTRL>
__device__ inline Two32 merge_dpp(Two32 a)
{
    return merge(a, Two32{dpp_u32<CTRL>(a.first), dpp_u32<CTRL>(a.second)});
}

// Largest first: Batcher's odd-even merge sort.
template <int N>
__device__ inline void sort_down(uint32_t (&v)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2) {
#pragma unroll
        for (int k = p; k >= 1; k /= 2) {
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k) {
#pragma unroll
                for (int i = 0; i < k; ++i) {
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t hi = max(v[i + j], v[i + j + k]);
                        v[i + j + k] = min(v[i + j], v[i + j + k]);
                        v[i + j] = hi;
                    }
                }
            }
        }
    }
}

// Whether a group is a whole power of two of lanes.
__device__ inline bool groups_fit(int size, int epl)
{
    const int lanes = size / epl;
    return size % epl == 0 && (lanes & (lanes - 1)) == 0;
}

template <int DT, int EPL>
__device__ inline bool choose_fast(const RouteScoresArgs& a, const typename RowType<DT>::Raw* row, int lane,
                                   const float (&score)[EPL], const float (&bias)[EPL], const float (&l)[EPL], float m,
                                   int& id)
{
    uint32_t key[EPL];  // masked: 0, which no other word is
    const float base = a.bias ? 1.0f : 0.0f;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const float c = score[j] + bias[j];
        nan |= c != c && l[j] != -INFINITY;
        key[j] = l[j] == -INFINITY || c == -INFINITY ? 0u : (ordered(c) & ~(uint32_t)(EPL - 1)) | j;
    }
    if (__any(nan)) return false;
    sort_down(key);
    if (a.top_groups < a.n_groups) {
        const int lanes = a.group_size / EPL;
        if (!groups_fit(a.group_size, EPL)) return false;
        Two32 best{key[0], EPL > 1 ? key[EPL > 1] : 0};
        if (lanes > 1) best = merge_dpp<kDppXor1>(best);
        if (lanes > 2) best = merge_dpp<kDppXor2>(best);
        if (lanes > 4) best = merge_dpp<kDppHalfMirror>(best);
        if (lanes > 8) best = merge_dpp<kDppMirror>(best);
        for (int d = 16; d < lanes; d <<= 1) {
            best = merge(best, Two32{(uint32_t)__shfl_xor((int)best.first, d, kWave),
                                     (uint32_t)__shfl_xor((int)best.second, d, kWave)});
        }
        float rank = best.first ? value32<EPL>(best.first) : -INFINITY, size_of = best.first ? fabsf(rank) : 0.0f;
        if (a.group_top == 2 && best.second) {
            const float second = value32<EPL>(best.second);
            rank += second;
            size_of += fabsf(second);
        }
        // two finite choices may add up to less than float32 holds, where -inf stands for a group without experts
        if (__any(best.first && rank == -INFINITY)) return false;
        const int mine = lane / lanes;
        int before = 0;  // groups ahead of the lane's; equal ones are kept or dropped together
        for (int g = 0; g < a.n_groups; ++g) before += readlane_f32(rank, g * lanes) > rank;
        const bool in = mine < a.n_groups, kept = before < a.top_groups;
        const float least = -wave_largest(in && kept ? -rank : -INFINITY);
        const float most = wave_largest(in && !kept ? rank : -INFINITY);
        // A rank's error goes with what it is the sum of, which with a bias may be far larger than the rank; without
        // one, a score's relative error also has the rounding of l - m, up to 64 u.  Without an expert left in the
        // best of the others nothing hangs on it.
        const float scale = a.bias ? 2.0f + wave_largest(size_of) : 4.0f * least;
        if (__popcll(__ballot(in && kept && rank > -INFINITY)) > a.top_groups * lanes) return false;
        if (most > -INFINITY && !(least - most > kNear * scale + 0x1p-120f)) return false;
        if (!kept) {
#pragma unroll
            for (int j = 0; j < EPL; ++j) key[j] = 0;
        }
    }
    auto near = [&](float before, float c) { return !(before - c > kNear * (base + fabsf(c))); };  // inf and inf too
    uint32_t own = 0, last = 0;
    int n = 0;  // candidates, in lanes 0 .. n - 1
    for (;; ++n) {
        const uint32_t top = wave_max_u32(key[0]);
        if (top == 0) break;
        if (n >= a.top_k) {
            if (!near(value32<EPL>(last), value32<EPL>(top))) break;
            if (n == kWave) return false;
        }
        last = top;
        const int from = __builtin_ctzll(__ballot(key[0] == top));
        if (lane == n) {
            own = top;
            id = from * EPL + (int)(top & (EPL - 1));
        }
        const bool taken = lane == from;
#pragma unroll
        for (int j = 0; j < EPL; ++j) key[j] = taken ? (j + 1 < EPL ? key[j + 1 < EPL ? j + 1 : j] : 0u) : key[j];
    }
    const uint32_t before = (uint32_t)__shfl_up((int)own, 1, kWave);
    if (__any(lane > 0 && lane < n && near(value32<EPL>(before), value32<EPL>(own)))) {
        if (!a.sigmoid && a.bias) return false;
        const double logit = id < 0 ? 0.0 : (double)RowType<DT>::value(row[id]);
        // softmax without a bias: exp(l - m) orders as the scores do
        const double score64 = a.sigmoid ? 1.0 / (1.0 + exp(-logit)) : exp(logit - (double)m);
        const uint64_t exact = id < 0 ? 0 : key_of(score64 + (a.bias ? (double)a.bias[id] : 0.0));
        int ahead = 0;
        for (int i = 0; i < n; ++i) {
            const uint64_t other = readlane_u64(exact, i);
            ahead += other > exact || (other == exact && __builtin_amdgcn_readlane(id, i) < id);
        }
        id = __builtin_amdgcn_ds_permute((lane < n ? ahead : lane) * 4, id);
    }
    if (lane >= a.top_k) id = -1;
    return true;
}

// The same in float64, whatever the margins.  choices: EPL * 64 words of LDS.
template <int EPL>
__device__ inline int choose_exactly(const RouteScoresArgs& a, int lane, const float (&l)[EPL], const float (&bias)[EPL],
                                     float m, bool poisoned, uint64_t* choices)
{
    const int e0 = lane * EPL;
    double score[EPL];
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) score[j] = 1.0 / (1.0 + exp(-(double)l[j]));
    } else {
        double part = 0.0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            score[j] = l[j] == -INFINITY ? 0.0 : poisoned ? (double)NAN : exp((double)l[j] - (double)m);
            part += score[j];
        }
        const double sum = wave_sum_f64(part);
#pragma unroll
        for (int j = 0; j < EPL; ++j) score[j] /= sum;
    }
    uint64_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = l[j] == -INFINITY ? 0 : key_of(score[j] + (double)bias[j]);

    if (a.top_groups < a.n_groups) {
        const int size = a.group_size, lanes = size / EPL;
        if (groups_fit(size, EPL)) {
            Two best{key[0], 0};
#pragma unroll
            for (int j = 1; j < EPL; ++j) best = merge(best, Two{key[j], 0});
            if (lanes > 1) best = merge(best, Two{dpp_u64<kDppXor1>(best.first), dpp_u64<kDppXor1>(best.second)});
            if (lanes > 2) best = merge(best, Two{dpp_u64<kDppXor2>(best.first), dpp_u64<kDppXor2>(best.second)});
            if (lanes > 4) {
                best = merge(best, Two{dpp_u64<kDppHalfMirror>(best.first), dpp_u64<kDppHalfMirror>(best.second)});
            }
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
            for (int j = 0; j < EPL; ++j) choices[e0 + j] = key[j];
            __builtin_amdgcn_wave_barrier();
            Two best{0, 0};  // lane g's group is g
            if (lane < a.n_groups) {
                for (int i = 0; i < size; ++i) best = merge(best, Two{choices[lane * size + i], 0});
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

    int id = -1;
    for (int s = 0; s < a.top_k; ++s) {
        uint64_t best = key[0];
        int at = 0;
#pragma unroll
        for (int j = 1; j < EPL; ++j) {
            if (key[j] > best) {
                best = key[j];
                at = j;
            }
        }
        const int from = wave_best(best);
        if (from < 0) break;
        const int e = from * EPL + __builtin_amdgcn_readlane(at, from);
        if (lane == s) id = e;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            if (e0 + j == e) key[j] = 0;
        }
    }
    return id;
}

// What bounds it: few tokens, the launch and the chain of wavefront maxima, one for each slot; many, the
// instructions of a token, about 650 (65536 tokens, 256 experts in 8 groups, top-8: 71 us for 72 MB; with every
// choice in float64 102; 4096 tokens of 1024 experts, top-16: 17 us against 33; without the sort within a lane
// 84 and 24; tokens in turn in a launch of 2048 workgroups: 90).  A lane holds neighbouring experts
// so that a group is a few lanes and its best two come by DPP; a wavefront a token, since a token's maxima are
// then one reduction each and nothing waits at a barrier.
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
    float m = -INFINITY, sum = 1.0f;
    bool poisoned = false;
    float score[EPL];
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) score[j] = logistic(l[j]).s;
    } else {
        bool nan = false;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            m = fmaxf(m, l[j]);
            nan |= l[j] != l[j];
        }
        m = wave_largest(m);
        poisoned = __any(nan) || m == INFINITY;
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            score[j] = l[j] == -INFINITY ? 0.0f : exp_of(l[j] - m);
            part += score[j];
        }
        sum = wave_sum_f32(part);
        float inverse = __builtin_amdgcn_rcpf(sum);  // of a sum within [1, 1024]
        inverse = fmaf(fmaf(-sum, inverse, 1.0f), inverse, inverse);
#pragma unroll
        for (int j = 0; j < EPL; ++j) score[j] *= inverse;
    }
    int id = -1;
    if (poisoned || !choose_fast<DT, EPL>(a, row, lane, score, bias, l, m, id)) {
        id = choose_exactly<EPL>(a, lane, l, bias, m, poisoned, choices[wave]);
    }
    const float chosen = id >= 0 ? RowType<DT>::value(row[id]) : -INFINITY;
    float w = 0.0f;
    if (a.normalize) {
        const float top = wave_largest(chosen == chosen ? chosen : -INFINITY);
        const float r = id < 0 ? 0.0f : relative_score(a.sigmoid, chosen, top);
        const float total = sum_slots(r);
        if (id >= 0) w = r / total;
    } else if (id >= 0) {
        w = a.sigmoid ? logistic(chosen).s : exp_of(chosen - m) / sum;
    }
    if (poisoned && id >= 0) w = NAN;
    if (lane < a.top_k) {
        a.ids[t * a.top_k + lane] = id;
        a.weights[t * a.top_k + lane] = w * a.scale;
    }
}

// A row is read and written once and its slots' logits once more; sums of a token by DPP.  Bound by HBM where there
// are many tokens (65536 tokens of 256 experts, top-8, sigmoid: 40 us for 138 MB, 3.5 TB/s), else by the launch.
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
        const float top = wave_largest(chosen == chosen ? chosen : -INFINITY);
        const float r = id < 0 ? 0.0f : relative_score(a.sigmoid, chosen, top);
        const float sum = sum_slots(r);
        const float w = id < 0 ? 0.0f : r / sum;
        const float centre = sum_slots(id < 0 ? 0.0f : g * w);
        to_slot = id < 0 ? 0.0f : w * (g - centre) * (a.sigmoid ? logistic(chosen).rest : 1.0f);
    } else if (a.sigmoid) {
        const Logistic s = logistic(chosen);
        to_slot = id < 0 ? 0.0f : g * (s.s * s.rest);
    } else {
        bool nan = false;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            m = fmaxf(m, l[j]);
            nan |= l[j] != l[j];
        }
        m = __any(nan) ? NAN : wave_largest(m);
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) part += l[j] == -INFINITY ? 0.0f : exp_of(l[j] - m);
        total = wave_sum_f32(part);
        mean = sum_slots(id < 0 ? 0.0f : g * (exp_of(chosen - m) / total));
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
        if (!a.sigmoid && !a.normalize) out[j] = l[j] == -INFINITY ? 0.0f : exp_of(l[j] - m) / total * (out[j] - mean);
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
