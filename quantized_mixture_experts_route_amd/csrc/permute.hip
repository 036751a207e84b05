// permute.hip -- tokens sorted by expert, and their rows brought back with the
// routing weights, with the gradients of both.
//
// Sort.  Route r = t * top_k + s has key(r) = its expert, or E where the id is
// outside [0, E) (a dropped route).  Its row is
//   row(r) = |{q : key(q) < key(r)}| + |{q < r : key(q) = key(r)}|,
// a stable counting sort: the first term is an exclusive scan of the expert
// counts, the second the count among earlier routes.  Every workgroup owns a
// run of consecutive tokens, counts the routes before its own (per expert),
// ranks its own with ballots, and copies its tokens' rows: a token's row is
// read once and written top_k times.  No atomic decides an order, so the
// result is unique and deterministic.
//
// Counting.  Up to kOneLaunchRoutes routes every workgroup counts all of them
// itself (ids come from L2), so the whole operator is one launch; above it,
// count_kernel counts spans of about kSpanRoutes routes first, and a workgroup
// adds up the spans before its own and counts the part of its span before its
// tokens.  From more than kSummedSpans spans on, scan_kernel adds them up for
// everybody.
//
// Back.  out[t] = sum over slots, in slot order, of w[t, s] * rows[row(t, s)]
// in float32, rounded once; the gradient of the sort is the same sum without
// weights.  The gradient of the weighted sum is w * grad_out at the route's
// row and, for the weight, the dot product of grad_out with that row.  All of
// them move each row once and do a few operations an element, so they are
// bound by HBM: 4096 tokens of 4096 bf16 columns, top-2, take 30 us to sort
// (100 MB, 3.4 TB/s), 21 us to bring back (4.9 TB/s) and 34 us for the
// gradient (168 MB, 4.9 TB/s) with inputs out of cache; 23, 17 and 31 us with
// the inputs of the pass before.
#include "expert_ops.h"
#include "qmoe_internal.h"
#include "rowio.h"

namespace qmoe {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 1024;
constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int64_t kOneLaunchRoutes = 8192;
constexpr int kSummedSpans = 32;
constexpr int kSpanRoutes = 4096;  // (a span is at most that or one workgroup's tokens)

__device__ inline int route_key(int id, int E) { return id >= 0 && id < E ? id : E; }

// Lanes of the wavefront that hold the same key as this one, of those in `valid`.
__device__ inline uint64_t same_key(int key, uint64_t valid, int bits)
{
    uint64_t peers = valid;
    for (int i = 0; i < bits; ++i) {
        const bool bit = (key >> i) & 1;
        const uint64_t set = __ballot(bit);
        peers &= bit ? set : ~set;
    }
    return peers;
}

// Adds the keys of routes lo .. hi (at most kMaxCounted of them) to a table in
// LDS.  Many keys: each lane adds its own.  With up to 16 keys the lanes of a
// wavefront would queue at a handful of words (worst where neighbouring routes
// go to one expert), so each thread counts in bytes of two 64-bit registers,
// and a wavefront sums those with cross-lane adds before one lane adds them.
constexpr int kFewKeys = 16;
constexpr int64_t kMaxCounted = 255 * kSortThreads;  // a thread's count of a key fits a byte
static_assert(kOneLaunchRoutes <= kMaxCounted && kSpanRoutes <= kMaxCounted && kMaxTopK <= kMaxCounted, "counts");
__device__ void count_routes(const int32_t* ids, int64_t lo, int64_t hi, int E, int* table)
{
    if (E >= kFewKeys) {
        for (int64_t r = lo + threadIdx.x; r < hi; r += kSortThreads) atomicAdd(&table[route_key(ids[r], E)], 1);
        return;
    }
    if (lo + (threadIdx.x & ~63) >= hi) return;  // nothing for this wavefront
    uint64_t low = 0, high = 0;  // keys 0..7 and 8..15
    for (int64_t r = lo + threadIdx.x; r < hi; r += kSortThreads) {
        const int key = route_key(ids[r], E);
        const uint64_t one = 1ull << (8 * (key & 7));
        if (key < 8) low += one; else high += one;
    }
    // pairs of 16-bit counts: a wavefront's stay below 64 * 255
    uint32_t pair[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t word = (uint32_t)((i < 2 ? low : high) >> (32 * (i & 1)));
        pair[2 * i] = word & 0x00ff00ffu;             // keys 4i and 4i + 2
        pair[2 * i + 1] = (word >> 8) & 0x00ff00ffu;  // keys 4i + 1 and 4i + 3
    }
    const int lane = threadIdx.x & 63;
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t v = pair[i];
        v += dpp_u32<kDppXor1>(v);
        v += dpp_u32<kDppXor2>(v);
        v += dpp_u32<kDppHalfMirror>(v);
        v += dpp_u32<kDppMirror>(v);
        v = (uint32_t)__builtin_amdgcn_readlane((int)v, 0) + (uint32_t)__builtin_amdgcn_readlane((int)v, 16) +
            (uint32_t)__builtin_amdgcn_readlane((int)v, 32) + (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
        // lane = key takes its half: pair i holds keys 4 (i/2) + i%2 and 2 more
        const int key = 4 * (i >> 1) + (i & 1);
        if (lane == key) mine = v & 0xffffu;
        if (lane == key + 2) mine = v >> 16;
    }
    if (lane <= E && mine) atomicAdd(&table[lane], (int)mine);
}

// Exclusive scan of v[0..n), n <= kMaxExperts + 1, by the whole workgroup.
__device__ void scan_counts(int* v, int n, int* wave_sums)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (n + kSortThreads - 1) / kSortThreads;  // consecutive entries per thread
    const int lo = tid * per;
    int sum = 0;
    for (int i = 0; i < per; ++i) {
        if (lo + i < n) sum += v[lo + i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int y = __shfl_up(incl, d, kWave);
        if (lane >= d) incl += y;
    }
    if (lane == kWave - 1) wave_sums[wave] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < wave; ++w) run += wave_sums[w];
    for (int i = 0; i < per; ++i) {
        if (lo + i < n) {
            const int c = v[lo + i];
            v[lo + i] = run;
            run += c;
        }
    }
    __syncthreads();
}

// The tokens of workgroup b are [b * tokens_per_wg, ...); spans are whole
// multiples of that.
struct SortShape {
    int tokens_per_wg;
    int wgs_per_span;  // 0: no spans, every workgroup counts all routes
};

template <int EB, int V>
__global__ __launch_bounds__(kSortThreads) void permute_kernel(
    const void* __restrict__ hidden, int64_t row_stride, int64_t T, int H,
    const int32_t* __restrict__ ids, int top_k, int E, void* __restrict__ rows,
    int32_t* __restrict__ offsets, int32_t* __restrict__ sorted, int32_t* __restrict__ route_rows,
    const int32_t* __restrict__ counts, int summed, const int32_t* __restrict__ totals, SortShape sh)
{
    typedef typename std::conditional<EB == 2, uint16_t, uint32_t>::type Raw;
    __shared__ int before[kMaxExperts + 1];  // routes of the key before this workgroup's, then its next row
    __shared__ int base[kMaxExperts + 1];    // routes of the key anywhere, then the key's first row
    __shared__ int row_of[kMaxTopK > 64 ? kMaxTopK : 64];  // ~row for a dropped route
    __shared__ int wave_sums[kSortWaves];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int64_t t0 = (int64_t)blockIdx.x * sh.tokens_per_wg;
    const int tokens = (int)(T - t0 < sh.tokens_per_wg ? T - t0 : sh.tokens_per_wg);
    const int64_t r0 = t0 * top_k;
    const int routes = tokens * top_k;
    const bool spans = sh.wgs_per_span > 0;
    const int64_t span = spans ? blockIdx.x / sh.wgs_per_span : 0;

    // the first vectors of the tokens' rows are on their way while the routes are counted
    constexpr int AHEAD = V > 1 ? 4 : 1;
    const int nvec = row_vecs<V>(H);
    const int vecs = hidden ? tokens * nvec : 0;
    auto load = [&](int i) {
        const int t = i / nvec;
        return load_vec<Raw, V>((const Raw*)hidden + (t0 + t) * row_stride + vec_start<V>(i - t * nvec, H));
    };
    RowVec<Raw, V> x[AHEAD];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
        if (tid + q * kSortThreads < vecs) x[q] = load(tid + q * kSortThreads);
    }

    for (int e = tid; e <= E; e += kSortThreads) {
        int b = 0, all = 0;
        if (spans && totals) {  // counts[span] was made the count in earlier spans
            b = counts[span * (E + 1) + e];
            all = totals[e];
        } else if (spans) {
            for (int c = 0; c < summed; ++c) {
                const int n = counts[c * (E + 1) + e];
                if (c < span) b += n;
                all += n;
            }
        }
        before[e] = b;
        base[e] = all;
    }
    __syncthreads();
    {
        const int64_t lo = spans ? span * sh.wgs_per_span * (int64_t)sh.tokens_per_wg * top_k : 0;
        const int64_t hi = spans ? r0 : T * top_k;
        count_routes(ids, lo, r0, E, before);
        count_routes(ids, r0, hi, E, base);
    }
    __syncthreads();
    if (!spans) {
        for (int e = tid; e <= E; e += kSortThreads) base[e] += before[e];
        __syncthreads();
    }
    scan_counts(base, E + 1, wave_sums);
    for (int e = tid; e <= E; e += kSortThreads) {
        before[e] += base[e];
        if (blockIdx.x == 0) offsets[e] = base[e];
    }
    __syncthreads();

    // rows of this workgroup's routes, 64 at a time and in order: lanes of one
    // key find each other with ballots over the key's bits, the rank is the
    // count of lower peers, and the highest peer moves the key's next row on
    if (tid < kWave) {
        const int bits = 32 - __builtin_clz((unsigned)E);
        for (int b = 0; b < routes; b += kWave) {
            const bool valid = b + lane < routes;
            const int key = valid ? route_key(ids[r0 + b + lane], E) : -1;
            const uint64_t peers = same_key(key, __ballot(valid), bits);
            if (valid) {
                const int row = before[key] + __popcll(peers & ((1ull << lane) - 1ull));
                row_of[b + lane] = key < E ? row : ~row;
                sorted[row] = (int32_t)(r0 + b + lane);
                route_rows[r0 + b + lane] = key < E ? row : ~row;
            }
            __builtin_amdgcn_wave_barrier();
            if (valid && (peers >> lane) == 1ull) before[key] += __popcll(peers);
            __builtin_amdgcn_wave_barrier();
        }
    }
    if (hidden == nullptr) return;
    __syncthreads();

    for (int i = tid; i < vecs; i += AHEAD * kSortThreads) {
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
            const int j = i + q * kSortThreads;
            if (j >= vecs) break;
            const int t = j / nvec, h = vec_start<V>(j - t * nvec, H);
            for (int s = 0; s < top_k; ++s) {
                const int row = row_of[t * top_k + s];
                Raw* dst = (Raw*)rows + (int64_t)(row < 0 ? ~row : row) * H + h;
                store_vec<Raw, V>(dst, row < 0 ? RowVec<Raw, V>{} : x[q]);
            }
            if (j + AHEAD * kSortThreads < vecs) x[q] = load(j + AHEAD * kSortThreads);
        }
    }
}

// Routes of each key in span blockIdx.x: counts[span][E + 1].
__global__ __launch_bounds__(kSortThreads) void count_kernel(const int32_t* __restrict__ ids,
                                                             int64_t R, int E, int span_routes,
                                                             int32_t* __restrict__ counts)
{
    __shared__ int cnt[kMaxExperts + 1];
    for (int e = threadIdx.x; e <= E; e += kSortThreads) cnt[e] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * span_routes;
    const int64_t hi = lo + span_routes < R ? lo + span_routes : R;
    count_routes(ids, lo, hi, E, cnt);
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kSortThreads) counts[blockIdx.x * (int64_t)(E + 1) + e] = cnt[e];
}

// counts[span][key] becomes the number of routes of the key in earlier spans,
// totals[key] the number in all: 64 keys a workgroup, the spans in 16 parts.
constexpr int kScanParts = 16;
__global__ __launch_bounds__(64 * kScanParts) void scan_kernel(int32_t* __restrict__ counts, int spans,
                                                              int n, int32_t* __restrict__ totals)
{
    __shared__ int sums[kScanParts][64];
    const int lane = threadIdx.x & 63, part = threadIdx.x >> 6;
    const int key = blockIdx.x * 64 + lane;
    const int per = (spans + kScanParts - 1) / kScanParts;
    const int lo = part * per < spans ? part * per : spans;
    const int hi = lo + per < spans ? lo + per : spans;
    int sum = 0;
    if (key < n) {
        for (int c = lo; c < hi; ++c) sum += counts[c * (int64_t)n + key];
    }
    sums[part][lane] = sum;
    __syncthreads();
    int run = 0;
    for (int p = 0; p < part; ++p) run += sums[p][lane];
    if (key < n) {
        for (int c = lo; c < hi; ++c) {
            const int x = counts[c * (int64_t)n + key];
            counts[c * (int64_t)n + key] = run;
            run += x;
        }
        if (part == kScanParts - 1) totals[key] = run;
    }
}

// Threads that share one token: a power of two, so that a workgroup of 256
// holds whole tokens and no division splits its index.
constexpr int kBackThreads = 256;
constexpr unsigned kBackCUs = 256;
template <int V>
int threads_per_token(int H)
{
    int n = 8;
    while (n < kBackThreads && n < row_vecs<V>(H)) n *= 2;
    return n;
}

// Two slots at a time, their vectors requested together (4096 tokens of 2048
// bf16 columns, top-8: 31.2 us, 4.8 TB/s; all eight at a time 40.7).
template <int DT, int V>
__global__ __launch_bounds__(kBackThreads) void unpermute_kernel(
    const void* __restrict__ rows, int64_t row_stride, const int32_t* __restrict__ route_rows,
    const float* __restrict__ weights, int64_t T, int top_k, int H, int tpt_log2,
    void* __restrict__ out)
{
    typedef typename RowType<DT>::Raw Raw;
    constexpr int G = 2;
    const int64_t R = T * top_k;
    const int64_t t = ((int64_t)blockIdx.x * kBackThreads + threadIdx.x) >> tpt_log2;
    if (t >= T) return;
    const int nvec = row_vecs<V>(H);
    for (int i = threadIdx.x & ((1 << tpt_log2) - 1); i < nvec; i += 1 << tpt_log2) {
        const int h = vec_start<V>(i, H);
        const Raw* in = (const Raw*)rows + h;
        float sum[V] = {};
        for (int s0 = 0; s0 < top_k; s0 += G) {
            RowVec<Raw, V> x[G];
            bool on[G];
            float w[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                on[g] = s0 + g < top_k;
                const int64_t j = on[g] ? route_rows[t * top_k + s0 + g] : -1;
                on[g] = j >= 0 && j < R;
                w[g] = on[g] && weights ? weights[t * top_k + s0 + g] : 1.0f;
                if (on[g]) x[g] = load_vec<Raw, V>(in + j * row_stride);
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (!on[g]) continue;
#pragma unroll
                for (int q = 0; q < V; ++q) sum[q] = __builtin_fmaf(w[g], RowType<DT>::value(x[g].v[q]), sum[q]);
            }
        }
        RowVec<Raw, V> y;
#pragma unroll
        for (int q = 0; q < V; ++q) y.v[q] = RowType<DT>::round(sum[q]);
        store_vec<Raw, V>((Raw*)out + t * H + h, y);
    }
}

// G slots of a token at a time: grad_out's vector is read once for the G rows
// it goes to, and G dot products run along.  The dot products are summed in a
// fixed order: inside a wavefront cross-lane, then the token's wavefronts (1 to
// 4) in order, through LDS and behind the one barrier at the end.
template <int DT, int V, int G>
__global__ __launch_bounds__(kBackThreads) void unpermute_backward_kernel(
    const void* __restrict__ grad_out, int64_t grad_stride, const void* __restrict__ rows,
    int64_t row_stride, const int32_t* __restrict__ route_rows, const float* __restrict__ weights,
    int64_t T, int top_k, int H, int tpt_log2, void* __restrict__ grad_rows,
    float* __restrict__ grad_weights)
{
    typedef typename RowType<DT>::Raw Raw;
    constexpr int WAVES = kBackThreads / kWave;
    __shared__ float wave_dot[WAVES][kMaxTopK];
    const int64_t R = T * top_k;
    const int tpt = 1 << tpt_log2;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int sub = threadIdx.x & (tpt - 1);
    const int64_t t = ((int64_t)blockIdx.x * kBackThreads + threadIdx.x) >> tpt_log2;
    const bool live = t < T;
    const int nvec = row_vecs<V>(H);
    for (int s0 = 0; s0 < top_k; s0 += G) {
        int64_t j[G];   // the row, or -1
        bool kept[G];
        float w[G], dot[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const bool on = live && s0 + g < top_k;
            const int64_t v = on ? route_rows[t * top_k + s0 + g] : R;
            kept[g] = v >= 0 && v < R;
            const int64_t at = v < 0 ? -1 - v : v;
            j[g] = on && at < R ? at : -1;
            w[g] = !kept[g] ? 0.0f : weights ? weights[t * top_k + s0 + g] : 1.0f;
            dot[g] = 0.0f;
        }
        for (int i = live ? sub : nvec; i < nvec; i += tpt) {
            const int h = vec_start<V>(i, H);
            const int skip = i * V - h;  // leading elements that the vector before counted already
            const auto d = load_vec<Raw, V>((const Raw*)grad_out + t * grad_stride + h);
            RowVec<Raw, V> x[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (kept[g] && rows) x[g] = load_vec<Raw, V>((const Raw*)rows + j[g] * row_stride + h);
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (j[g] < 0) continue;
                RowVec<Raw, V> y = {};
                if (kept[g]) {
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        const float dv = RowType<DT>::value(d.v[q]);
                        y.v[q] = RowType<DT>::round(w[g] * dv);
                        if (rows && q >= skip) dot[g] = __builtin_fmaf(dv, RowType<DT>::value(x[g].v[q]), dot[g]);
                    }
                }
                store_vec<Raw, V>((Raw*)grad_rows + j[g] * H + h, y);
            }
        }
        if (!grad_weights) continue;
        if (tpt >= kWave) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float sum = wave_sum_f32(dot[g]);
                if (lane == 0 && s0 + g < top_k) wave_dot[wave][s0 + g] = sum;
            }
        } else {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                for (int d = tpt / 2; d > 0; d >>= 1) dot[g] += __shfl_xor(dot[g], d, kWave);
                if (live && sub == 0 && s0 + g < top_k) grad_weights[t * top_k + s0 + g] = dot[g];
            }
        }
    }
    if (grad_weights && tpt >= kWave) {
        __syncthreads();
        for (int s = sub; live && s < top_k; s += tpt) {
            float sum = 0.0f;
            for (int q = 0; q < tpt / kWave; ++q) sum += wave_dot[(threadIdx.x - sub) / kWave + q][s];
            grad_weights[t * top_k + s] = sum;
        }
    }
}

int log2_of(int x) { return 31 - __builtin_clz((unsigned)x); }

SortShape sort_shape(int64_t T, int top_k)
{
    const int64_t R = T * top_k;
    SortShape sh;
    // about 64 routes a workgroup, fewer while that leaves CUs without one, more
    // where workgroups come in many rounds
    int64_t routes = R / 1024;
    routes = routes < 64 ? 64 : routes > 256 ? 256 : routes;
    int64_t per = routes / top_k;
    const int64_t spread = T / 512;
    if (spread < per) per = spread;
    sh.tokens_per_wg = per < 1 ? 1 : (int)per;
    sh.wgs_per_span = 0;
    if (R > kOneLaunchRoutes) {
        const int w = kSpanRoutes / (sh.tokens_per_wg * top_k);
        sh.wgs_per_span = w < 1 ? 1 : w;
    }
    return sh;
}

int64_t span_count(int64_t T, const SortShape& sh)
{
    const int64_t tokens = (int64_t)sh.tokens_per_wg * sh.wgs_per_span;
    return (T + tokens - 1) / tokens;
}

}  // namespace

int64_t permute_ws_ints(int64_t T, int top_k, int E)
{
    const SortShape sh = sort_shape(T, top_k);
    if (!sh.wgs_per_span) return 0;
    return (span_count(T, sh) + 1) * (E + 1);
}

hipError_t launch_permute(const PermuteArgs& a, hipStream_t s)
{
    const SortShape sh = sort_shape(a.T, a.top_k);
    const int32_t* totals = nullptr;
    const int64_t spans = sh.wgs_per_span ? span_count(a.T, sh) : 0;
    if (spans > 0) {
        launch(count_kernel, dim3((unsigned)spans), dim3(kSortThreads), s, a.ids, a.T * a.top_k, a.E,
               sh.tokens_per_wg * sh.wgs_per_span * a.top_k, a.ws);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (spans > kSummedSpans) {
        int32_t* tot = a.ws + spans * (a.E + 1);
        launch(scan_kernel, dim3((unsigned)((a.E + 1 + 63) / 64)), dim3(64 * kScanParts), s, a.ws, (int)spans,
               a.E + 1, tot);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        totals = tot;
    }
    // T = 0 still launches one workgroup, which writes the offsets
    const int64_t wgs = a.T > 0 ? (a.T + sh.tokens_per_wg - 1) / sh.tokens_per_wg : 1;
    auto go = [&](auto kernel) {
        launch(kernel, dim3((unsigned)wgs), dim3(kSortThreads), s, a.hidden, a.row_stride, a.T, a.H, a.ids,
               a.top_k, a.E, a.rows, a.offsets, a.sorted_routes, a.route_rows, (const int32_t*)a.ws, (int)spans, totals, sh);
    };
    if (a.elem == 2) {
        if (a.H >= 8) go(permute_kernel<2, 8>);
        else go(permute_kernel<2, 1>);
    } else {
        if (a.H >= 4) go(permute_kernel<4, 4>);
        else go(permute_kernel<4, 1>);
    }
    return hipGetLastError();
}

namespace {

template <int DT, int V>
hipError_t unpermute_as(const UnpermuteArgs& a, hipStream_t s)
{
    const int tpt = threads_per_token<V>(a.H);
    const dim3 grid((unsigned)((a.T * tpt + kBackThreads - 1) / kBackThreads));
    launch(unpermute_kernel<DT, V>, grid, dim3(kBackThreads), s, a.rows, a.row_stride, a.route_rows, a.weights,
           a.T, a.top_k, a.H, log2_of(tpt), a.out);
    return hipGetLastError();
}

template <int DT, int V>
hipError_t unpermute_backward_as(const UnpermuteArgs& a, hipStream_t s)
{
    const int tpt = threads_per_token<V>(a.H);
    const dim3 grid((unsigned)((a.T * tpt + kBackThreads - 1) / kBackThreads));
    auto go = [&](auto kernel) {
        launch(kernel, grid, dim3(kBackThreads), s, a.grad_out, a.grad_stride, a.rows, a.row_stride,
               a.route_rows, a.weights, a.T, a.top_k, a.H, log2_of(tpt), a.grad_rows, a.grad_weights);
    };
    // Two slots at a time, so that their loads overlap.  The bfloat16 form holds 76 registers a lane for
    // that, six workgroups a CU: where more are launched than fit the chip at once, one slot at a time (56
    // registers, all eight) is faster.  us, one against two, out of cache:
    //   bf16, H 2048, top-6: 1024 tokens 20.9, 18.8;  1536 24.0, 22.2;  1792 25.5, 30.9;  4096 50.8, 55.6
    //         H 4096, top-2: 1024 13.5, 12.6;  1536 15.9, 15.0;  1792 17.6, 20.5;  4096 36.5, 38.2
    //         H 1001, top-6 (two tokens a workgroup): 2816 26.2, 22.9;  3584 28.6, 32.6
    //   f16, H 2048, top-4: 1024 14.3, 12.2;  4096 34.8, 32.5
    //   f32, H 2048, top-4: 512 17.3, 13.0;  2048 34.8, 30.0;  8192 131.8, 129.9
    // Inputs that are still in cache like two slots better between 3500 and 6100 tokens of H 4096 (top-2
    // 4096 tokens: 36.0, 33.7); there the rule goes by what a training step meets.  A bound of 64 registers
    // on the bfloat16 form spills and loses everywhere.
    if constexpr (DT == kBF16 && V > 1) {
        if (grid.x > 6 * kBackCUs) {
            go(unpermute_backward_kernel<DT, V, 1>);
            return hipGetLastError();
        }
    }
    go(unpermute_backward_kernel<DT, V, 2>);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_unpermute(const UnpermuteArgs& a, hipStream_t s)
{
    if (a.dtype == kF32) return a.H >= 4 ? unpermute_as<kF32, 4>(a, s) : unpermute_as<kF32, 1>(a, s);
    if (a.dtype == kBF16) return a.H >= 8 ? unpermute_as<kBF16, 8>(a, s) : unpermute_as<kBF16, 1>(a, s);
    return a.H >= 8 ? unpermute_as<kF16, 8>(a, s) : unpermute_as<kF16, 1>(a, s);
}

hipError_t launch_unpermute_backward(const UnpermuteArgs& a, hipStream_t s)
{
    if (a.dtype == kF32) return a.H >= 4 ? unpermute_backward_as<kF32, 4>(a, s) : unpermute_backward_as<kF32, 1>(a, s);
    if (a.dtype == kBF16) return a.H >= 8 ? unpermute_backward_as<kBF16, 8>(a, s) : unpermute_backward_as<kBF16, 1>(a, s);
    return a.H >= 8 ? unpermute_backward_as<kF16, 8>(a, s) : unpermute_backward_as<kF16, 1>(a, s);
}

}  // namespace qmoe
