// fp8_matmul.hip -- grouped product of rows in 8-bit floating point (e4m3) with
// expert weights in the same format, with a float32 scale for each block of 128:
//   out[r, n] = sum_b sa(r, b) sw(e, n/128, b) sum_{k in block b} a(r, k) w(e, n, k)
// for the rows offsets[e] <= r < offsets[e+1] of expert e, rounded once to the
// output's type; rows behind the last expert's are zero.
//
// v_mfma_f32_16x16x128 on e4m3 operands: lane l = 16 g + c supplies row c of
// either operand and 32 values of the block of 128; which of them does not
// matter, as long as both operands take the same.  Register i of the result is
// row 4 g + i of the first operand and row c of the second.
//
// What the instruction rounds (measured on it): of each eight neighbouring products
// of a lane what lies below 2^-13 of the largest is cut off; their sums, 16 of a
// block, and the addend meet in float32.  In the 2-norm of the result that leaves
// 1.5e-5 on normal rows, 3.5e-5 on gated activations, 5.6e-5 with outliers of 30
// times the rest, whatever K: a thirtieth and less of the rounding to bf16 (1.66e-3),
// about a quarter and less of f16's (2.1e-4).  Outputs in float32 would need the operands
// as f16 at half the rate, and are refused.
//
// What bounds it: large products the cycles of a step, times a clock that the power
// limit holds down (8192 x 28672 x 4096 over 8 experts 900 to 930 us, 2.1 PFLOP/s;
// the unscaled library product of the same sizes 738; 8192^3 450 to 500).  A step of
// the largest tile, 2048 cycles of products a SIMD, takes 3380, so the matrix units
// are busy in 55% of 1.73 M cycles.  Without the products, the loads or the
// multiply-adds the kernel takes 1.75, 1.69 and 1.64 M: none of them alone is the
// bound, but the operands' reads from LDS between two barriers, which all of these
// keep (a bare loop of a step's products and multiply-adds takes 2080 cycles, with
// the reads 2840, with the loads too 3030, with one barrier 3200).  The clock is 1.8
// GHz, without the products 2.3.  14336 inputs, 4096 outputs, 8192 rows over 8
// experts (535 to 550 us): 590 tiles are three rounds on 256 CUs, where 2.3 would do.
// Products of few rows: HBM (60 rows over 512 experts, 2048 inputs, 1536 outputs: 39
// us, 4.6 TB/s out of the cache), and the smallest the chain of table, routes, rows
// and sum (2 rows over 8 experts: 7.7 us).
#include "expert_tiles.h"
#include "fp8_ops.h"
#include "fp8_shape.h"
#include "qmoe_internal.h"

namespace qmoe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
constexpr int kE4M3 = 0;  // operand format code of the matrix instructions

__device__ inline i32x8 operand(u32x4 a, u32x4 b)
{
    return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// f(0), ..., each with its number as a constant.
template <int FROM, int TO, class F>
__device__ inline void static_for(F f)
{
    if constexpr (FROM < TO) {
        f(std::integral_constant<int, FROM>{});
        static_for<FROM + 1, TO>(f);
    }
}

// A block's product on its own: the scales are applied to it in float32.
__device__ inline f32x4 block_product(i32x8 w, i32x8 x)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{}, kE4M3, kE4M3, 0, 0, 0, 0);
}

// A workgroup of WM x WN wavefronts computes BM = 16 MT WM rows against BN = 16 NT WN weight rows; a
// wavefront MT x NT blocks of 16 x 16.  W is the instruction's first operand, so a lane's registers run
// along n, and the row scale is the lane's own while the weight scale is the wavefront's: one factor for
// each 16 rows and block of 128, and one multiply-add for each result and block.
//
// K runs in steps of one block of 128: 128 bytes of codes a row, a whole cache line, written to LDS by the
// load itself (buffer_load ... lds) into one of STAGES stages, with the rows' scales of the block.  The one
// barrier of a step stands before its last group of products: then every operand of the step is in registers,
// its stage takes the loads of the step STAGES ahead, and the next step has landed.  Loads run on over the end
// of a tile into the workgroup's next one, so only its first tile waits for memory.
//
// LDS rows are 128 bytes (32 banks); the 16-byte chunk of row r sits in slot chunk ^ (r / 2 % 8), so that 16
// rows read at one chunk cover all 64 banks.
//
// WHOLE: K is a multiple of 128 with a step for each stage.  Otherwise codes and scales behind the row's end
// are read out of the buffer's bounds, which gives 0.
constexpr int kStepBytes = kFp8Block;  // codes of one row and step
constexpr int kSlots = kWave;          // scales a wavefront loads in a step

// Bytes that a tile reads of codes or scales; its descriptor from byte `at` on.
struct Span {
    const uint8_t* base;
    uint32_t size;
    __device__ inline __amdgpu_buffer_rsrc_t from(uint32_t at) const
    {
        const uint32_t bytes = __builtin_amdgcn_readfirstlane(size);
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base + at), 0, mx_bytes_left(bytes, at), 0x00020000);
    }
};

// A span in scalar registers.  It is uniform, which the compiler does not see of what came out of LDS or through
// a product on the vector units; each load would run in a loop over its lanes' descriptors.
__device__ inline Span uniform_span(const void* base, uint32_t bytes)
{
    const uint64_t p = (uint64_t)base;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)p);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
    return Span{(const uint8_t*)((uint64_t)hi << 32 | lo), (uint32_t)__builtin_amdgcn_readfirstlane(bytes)};
}

// The lane, worked out where it stands.  What is made from it needs no register over the K loop; what the
// compiler keeps there is spilled, and a reload waits for every load and store before it.
__device__ inline int lane_now()
{
    int zero = 0;
    asm volatile("" : "+s"(zero));
    return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, zero));
}

// BYTES a lane from the buffer to LDS at `to` + BYTES * lane (to is uniform); zeros where the lane's offset is
// not in the buffer.
template <int BYTES>
__device__ inline void load_to_lds(__amdgpu_buffer_rsrc_t r, uint32_t lane_offset, void* to)
{
    auto* const lds = (__attribute__((address_space(3))) void*)to;
    if constexpr (BYTES == 16) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds, 16, lane_offset, 0, 0, 0);
    else __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds, 4, lane_offset, 0, 0, 0);
}

// Rows behind the last expert's are zero; `end` is the last offset.
template <int THREADS>
__device__ inline void clear_behind(const Fp8MatmulArgs& a, int end)
{
    if (!a.offsets) return;
    uint16_t* const out = (uint16_t*)a.out;
    const int64_t lo = (int64_t)min(max(end, 0), a.rows) * a.N, hi = (int64_t)a.rows * a.N;
    for (int64_t i = lo + (blockIdx.x * (int64_t)THREADS + threadIdx.x) * 8; i < hi; i += (int64_t)gridDim.x * THREADS * 8) {
        if (i + 8 <= hi) {
            store_vec<uint16_t, 8>(out + i, RowVec<uint16_t, 8>{});
        } else {
            for (int64_t q = i; q < hi; ++q) out[q] = 0;
        }
    }
}

// Stores two neighbouring blocks of 16 x 16 results: lane 16 g + c holds row c, columns 4 g + i of either in
// register i.  `out` is the first row and column; rows and cols say how many of them exist (WHOLE: all).
template <int DT, bool WHOLE>
__device__ inline void store_blocks(uint16_t* out, int N, int rows, int cols, const f32x4& left, const f32x4& right,
                                    int lane)
{
    // lane groups trade columns, so that each lane holds eight neighbours (store_sixteen's order)
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto t = __builtin_amdgcn_permlane16_swap(pack_pair<DT>(left[2 * i], left[2 * i + 1]),
                                                        pack_pair<DT>(right[2 * i], right[2 * i + 1]), false, false);
        v[i] = t[0];
        v[2 + i] = t[1];
    }
    store_sixteen<WHOLE>(out, N, rows, cols, v, lane);
}

template <int DT, int MT, int NT, int WM, int WN, int STAGES, bool WHOLE>
__global__ __launch_bounds__(64 * WM * WN) void tiled_kernel(Fp8MatmulArgs a)
{
    constexpr int BM = 16 * MT * WM, BN = 16 * NT * WN, ROWS = BM + BN;
    constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
    constexpr int LOADS_A = BM / 8 / WAVES, LOADS_W = BN / 8 / WAVES;  // code loads of a wavefront and step: 8 rows each
    constexpr int LOADS = LOADS_A + LOADS_W + 1;                       // and one of scales
    constexpr int FIRST = LOADS_A + LOADS_W / 2 + 1;                   // those that the first half of a step issues
    constexpr int A_SLOTS = (BM + kSlots - 1) / kSlots;                // wavefronts that load rows' scales; the next: weights'
    constexpr int N_BLOCKS = (BN + kFp8Block - 1) / kFp8Block;
    static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0 && WAVES % 2 == 0, "load split");
    static_assert(A_SLOTS < WAVES && NT % 2 == 0 && NT * 16 <= kFp8Block, "a wavefront's columns share their scale");

    // one array for all of it: between arrays of their own the compiler tells apart what a load to
    // LDS writes and waits for every such load before it reads LDS
    constexpr int SCALES = ROWS * kStepBytes, STAGE = SCALES + WAVES * kSlots * 4;
    constexpr int LIST = STAGES * STAGE, SOURCE = LIST + (kMaxExperts + 1) * 4;
    static_assert(STAGE >= (kMaxExperts + 1) * 4, "the offsets' place");
    __shared__ __align__(16) uint8_t lds[SOURCE + 2 * BM * 4];
    int* const first = reinterpret_cast<int*>(lds + LIST);
    int* const source = reinterpret_cast<int*>(lds + SOURCE);

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int K = a.K, blocks = (K + kFp8Block - 1) / kFp8Block, n_blocks = (a.N + kFp8Block - 1) / kFp8Block;
    const int steps = max(blocks, STAGES);  // the loading side is STAGES ahead and stays within one tile

    // the last stage's space, not loaded before the first barrier, holds the offsets for the first item
    int* const scratch = reinterpret_cast<int*>(lds + (STAGES - 1) * STAGE);
    build_tile_list<BM, THREADS>(first, scratch, a.offsets, a.E, a.rows);
    const int n_tiles = (a.N + BN - 1) / BN;
    const int total = __builtin_amdgcn_readfirstlane(mx_items(first[a.E], n_tiles, a.rows, BM, a.E));
    // workgroups go to the 8 dies in turn: each die takes one run of items, so
    // that the workgroups of a die share rows and weights in its L2
    const int per_die = gridDim.x / 8;
    const int die = blockIdx.x % 8;
    const int end = (int)((int64_t)total * (die + 1) / 8);
    int next_item = (int)((int64_t)total * die / 8) + blockIdx.x / 8;

    clear_behind<THREADS>(a, a.offsets ? a.offsets[a.E] : 0);

    // ---- the loading side: an item and a step, up to STAGES steps ahead
    TileItem load_tile;
    int load_step = 0;
    auto load_chunk = [&](int lane) { return (uint32_t)((lane & 7) ^ ((wave & 1) * 4 + (lane >> 4))) * 16; };
    uint32_t code_at[LOADS_A];  // byte offset of the lane's chunk at step 0
    // rows behind N: out of bounds
    const uint32_t w_row = (wave * 8 + (lane_now() >> 3)) * (uint32_t)K + load_chunk(lane_now());
    uint32_t scale_at;          // byte offset of the lane's scale at step 0
    Span a_span, w_span, scale_span;
    // The next item, found between two tiles, where registers are free; and in LDS its rows' source rows in a
    // (from the tile's first row where there are no routes; -1: outside; rows behind the tile's repeat its last).
    TileItem next_tile;
    int found = 0;  // tables of source rows take turns
    auto find_tile = [&](auto offset) {
        next_tile = item_at<BM, BN>(first, offset, a.E, n_tiles, next_item, end);
        next_item += per_die;
        found ^= BM;
        for (int r = wave * kWave + lane_now(); r < BM && next_tile.n > 0; r += THREADS) {
            int row = min(r, next_tile.n - 1);
            if (a.sorted_routes) {
                const int route = a.sorted_routes[next_tile.row0 + row];
                row = route < 0 || route / a.top_k >= a.a_rows ? -1 : route / a.top_k;
            }
            source[found + r] = row;
        }
    };
    auto offset_of = [&](int e) { return a.offsets ? min(max(constant(a.offsets)[e], 0), a.rows) : e * a.rows; };
    auto start_tile = [&]() {  // all but what goes by the source rows
        load_tile = next_tile;
        load_step = 0;
        const TileItem& t = load_tile;
        const bool on = t.n > 0;
        const int w_rows = on ? min(BN, a.N - t.n0) : 0;
        const int64_t w0 = on ? (int64_t)t.expert * a.N + t.n0 : 0;
        w_span = uniform_span(a.w_codes + w0 * K, (uint32_t)(w_rows * K));
        const int64_t a0 = a.sorted_routes ? 0 : t.row0;
        const int64_t a_rows = !on ? 0 : a.sorted_routes ? a.a_rows : t.n;
        a_span = uniform_span(a.a_codes + a0 * K, (uint32_t)(a_rows * K));
        if (wave < A_SLOTS) {
            scale_span = uniform_span(a.a_scales + a0 * blocks, (uint32_t)(a_rows * blocks * 4));
        } else {
            const int64_t s0 = on ? (int64_t)t.expert * n_blocks + t.n0 / kFp8Block : 0;
            const int rows = on && wave == A_SLOTS ? min(N_BLOCKS, n_blocks - t.n0 / kFp8Block) : 0;
            scale_span = uniform_span(a.w_scales + s0 * blocks, (uint32_t)(rows * blocks * 4));
            const int lane = lane_now();
            scale_at = lane < rows ? lane * (uint32_t)blocks * 4 : kMxOutside;
        }
    };
    auto start_rows = [&]() {
        const int lane = lane_now();
#pragma unroll
        for (int j = 0; j < LOADS_A; ++j) {
            const int row = source[found + (j * WAVES + wave) * 8 + (lane >> 3)];
            code_at[j] = row < 0 ? kMxOutside : row * (uint32_t)K + load_chunk(lane);
        }
        if (wave < A_SLOTS) {
            // a lane's MT rows' scales lie side by side
            const int at = wave * kSlots + lane, block = at / (16 * MT), in = at % (16 * MT);
            const int row = source[found + min(block * 16 * MT + in % MT * 16 + in / MT, BM - 1)];
            scale_at = row < 0 ? kMxOutside : row * (uint32_t)blocks * 4;
        }
    };
    // The weights' halves: rows that a wavefront's first and last NT / 2 blocks read, 8 WAVES rows in turn.
    static_assert(NT * 8 == 8 * WAVES, "a load of all wavefronts covers half of one's columns");
    // The loads of a step, one by one: scales, rows, the first halves of the weights (FIRST of them), the second halves.
    auto load = [&](int stage, int q) {
        const uint32_t at = (uint32_t)load_step * kStepBytes;
        uint8_t* const to = lds + stage * STAGE;
        if (q == 0) {
            load_to_lds<4>(scale_span.from(load_step * 4), WHOLE || load_step < blocks ? scale_at : kMxOutside,
                           to + SCALES + wave * kSlots * 4);
            return;
        }
        const int lane = lane_now();
        const bool in = WHOLE || at + load_chunk(lane) < (uint32_t)K;
        if (q <= LOADS_A) {
            const int j = q - 1;
            load_to_lds<16>(a_span.from(at), in ? code_at[j] : kMxOutside, to + (j * WAVES + wave) * 8 * kStepBytes);
        } else {
            const int j = q < FIRST ? 2 * (q - 1 - LOADS_A) : 2 * (q - FIRST) + 1;
            load_to_lds<16>(w_span.from(at), in ? opaque(w_row) + (uint32_t)(j * WAVES * 8) * K : kMxOutside,
                            to + (BM + (j * WAVES + wave) * 8) * kStepBytes);
        }
    };
    auto load_all = [&](int stage, auto from, auto to) {
        static_for<decltype(from)::value, decltype(to)::value>([&](auto q) { load(stage, q); });
    };
    constexpr std::integral_constant<int, 0> kNone;
    constexpr std::integral_constant<int, 1 + LOADS_A> kWeights;
    constexpr std::integral_constant<int, LOADS> kAll;
    find_tile([&](int e) { return __builtin_amdgcn_readfirstlane(scratch[e]); });
    start_tile();
    load_all(0, kWeights, kAll);  // weights do not wait for the table of rows
    __syncthreads();
    start_rows();
    load_all(0, kNone, kWeights);
    ++load_step;
#pragma unroll
    for (int i = 1; i < STAGES - 1; ++i) {
        load_all(i, kNone, kAll);
        ++load_step;
    }
    find_tile(offset_of);

    // ---- the computing side: chunks g and g + 4 of row c are lane 16 g + c's
    const int c = lane_now() & 15, g = lane_now() >> 4;
    const uint32_t read_lo = c * (uint32_t)kStepBytes + (uint32_t)(g ^ (c >> 1)) * 16, read_hi = read_lo ^ 64;
    constexpr int W_BUFFERS = NT < 4 ? NT : 4;  // two blocks ahead
    i32x8 x[MT], w[W_BUFFERS];
    typedef float RowScales __attribute__((ext_vector_type(MT)));
    RowScales sa;
    float sw;
    const uint32_t x_base = wm * MT * 16 * kStepBytes, w_base = (BM + wn * NT * 16) * kStepBytes;
    auto read_operand = [&](uint32_t at) {
        return operand(*reinterpret_cast<const u32x4*>(lds + at + read_lo),
                       *reinterpret_cast<const u32x4*>(lds + at + read_hi));
    };
    auto read_scales = [&](int stage) {
        const uint8_t* from = lds + stage * STAGE + SCALES;
        sa = *reinterpret_cast<const RowScales*>(from + (wm * 16 + c) * MT * 4);
        sw = *reinterpret_cast<const float*>(from + (A_SLOTS * kSlots + wn * NT * 16 / kFp8Block) * 4);
    };
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((STAGES - 2) * LOADS) : "memory");
    load_all(STAGES - 1, kNone, kAll);
    ++load_step;
    read_scales(0);
#pragma unroll
    for (int j = 0; j < MT; ++j) x[j] = read_operand(x_base + j * 16 * kStepBytes);
    w[0] = read_operand(w_base);
    w[1] = read_operand(w_base + 16 * kStepBytes);
    int stage = 0;
    while (load_tile.n > 0) {
        const TileItem tile = load_tile;
        // wavefronts whose rows lie behind the tile's leave their products out
        const bool active = wm * MT * 16 < tile.n;
        f32x4 acc[NT][MT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{};
        }
        for (int s = 0; s < steps; ++s) {
            const int next = stage + 1 == STAGES ? 0 : stage + 1;
            float f[MT];
            // A product's multiply-adds run behind the product LAG further on.  Products are counted in the order of
            // their issue: block by block, the last two blocks row by row.
            constexpr int LAG = 2, COUNT = NT * MT;
            f32x4 p[LAG + 1];
            auto add = [&](auto t) {
                constexpr int n = decltype(t)::value, tail = n - (NT - 2) * MT;
                constexpr int i = tail < 0 ? n / MT : NT - 2 + tail % 2, j = tail < 0 ? n % MT : tail / 2;
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][j][q] = fmaf(f[j], p[n % (LAG + 1)][q], acc[i][j][q]);
                asm volatile("" : "+v"(acc[i][j]));
            };
            auto product = [&](auto t, auto i, auto j) {
                constexpr int n = decltype(t)::value;
                p[n % (LAG + 1)] = block_product(w[decltype(i)::value % W_BUFFERS], x[decltype(j)::value]);
                asm volatile("" : "+v"(p[n % (LAG + 1)]));
                __builtin_amdgcn_sched_barrier(0);  // the product first, or its issue waits for the one that is added
                if constexpr (n == LAG) {
#pragma unroll
                    for (int q = 0; q < MT; ++q) f[q] = sa[q] * sw;
                }
                if constexpr (n >= LAG) add(std::integral_constant<int, n - LAG>{});
                __builtin_amdgcn_sched_barrier(0);
            };
            auto read_row = [&](auto j) { x[j] = read_operand(next * STAGE + x_base + j * 16 * kStepBytes); };
            // The rows and the first halves of the weights are in registers: their places take the loads of the
            // step STAGES ahead.
            auto first_half = [&]() {
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                if (load_step == steps) {
                    start_tile();
                    start_rows();
                }
            };
            // The rest is read, and the next step has landed once no more than the loads behind it are left.
            auto second_half = [&]() {
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"((STAGES - 2) * LOADS + FIRST) : "memory");
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            };
            if (active) {
                auto read_weight = [&](auto i, int from, int n) {
                    w[decltype(i)::value % W_BUFFERS] = read_operand(from * STAGE + w_base + n * 16 * kStepBytes);
                };
                // Loads are spread over the products (all at once they hold up the wavefront: 14336 inputs, 4096
                // outputs, 8192 rows over 8 experts: 672 -> 557 us).
                constexpr int MID = NT / 2 - 2, PLACES = (NT - 2 - MID) * MT;
                static_for<0, NT - 2>([&](auto row) {
                    constexpr int i = decltype(row)::value;
                    if constexpr (i == MID) first_half();
                    read_weight(std::integral_constant<int, i + 2>{}, stage, i + 2);
                    __builtin_amdgcn_sched_barrier(0);
                    static_for<0, MT>([&](auto column) {
                        constexpr int j = decltype(column)::value, place = (i - MID) * MT + j;
                        product(std::integral_constant<int, i * MT + j>{}, row, column);
                        if constexpr (place >= 0) {
                            static_for<0, FIRST>([&](auto q) {
                                if constexpr (decltype(q)::value * PLACES / FIRST == place) load(stage, q);
                            });
                        }
                    });
                });
                if constexpr (NT == 2) {
                    first_half();
                    static_for<0, FIRST>([&](auto q) { load(stage, q); });
                }
                second_half();
                // The last two blocks' products by rows, so that a row's operand is read for the next step as early
                // as can be: the wavefronts' reads come all at once here.
                if constexpr (NT > 2) read_weight(std::integral_constant<int, NT>{}, next, 0);
                __builtin_amdgcn_sched_barrier(0);
                static_for<0, MT>([&](auto column) {
                    constexpr int j = decltype(column)::value, n = (NT - 2) * MT + 2 * j;
                    product(std::integral_constant<int, n>{}, std::integral_constant<int, NT - 2>{}, column);
                    product(std::integral_constant<int, n + 1>{}, std::integral_constant<int, NT - 1>{}, column);
                    read_row(column);
                    static_for<FIRST, LOADS>([&](auto q) {
                        if constexpr ((decltype(q)::value - FIRST) * MT / (LOADS - FIRST) == j) load(stage, q);
                    });
                });
                if constexpr (NT == 2) read_weight(std::integral_constant<int, NT>{}, next, 0);
                read_weight(std::integral_constant<int, NT + 1>{}, next, 1);
                __builtin_amdgcn_sched_barrier(0);
                static_for<COUNT - LAG, COUNT>([&](auto t) { add(t); });
                read_scales(next);  // behind the last use of this step's
            } else {
                first_half();
                static_for<0, FIRST>([&](auto q) { load(stage, q); });
                second_half();
                static_for<FIRST, LOADS>([&](auto q) { load(stage, q); });
                read_scales(next);
                w[0] = read_operand(next * STAGE + w_base);
                w[1] = read_operand(next * STAGE + w_base + 16 * kStepBytes);
                static_for<0, MT>(read_row);
            }
            ++load_step;
            stage = next;
        }
        find_tile(offset_of);
        const int lane = lane_now();
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int m0 = (wm * MT + j) * 16;
#pragma unroll
            for (int i = 0; i < NT; i += 2) {
                const int n = tile.n0 + (wn * NT + i) * 16;
                uint16_t* out = (uint16_t*)a.out + (int64_t)(tile.row0 + m0) * a.N + n;
                if (tile.n - m0 >= 16 && a.N - n >= 32) {
                    store_blocks<DT, true>(out, a.N, 16, 32, acc[i][j], acc[i + 1][j], lane);
                } else {
                    store_blocks<DT, false>(out, a.N, tile.n - m0, a.N - n, acc[i][j], acc[i + 1][j], lane);
                }
            }
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may reach LDS behind the workgroup's end
}

// ---------------------------------------------------------------- few rows
// Up to 16 rows against COLUMNS (16 or 32) weight rows; the eight wavefronts share K block by block, operands
// straight from memory, every load of four blocks a wavefront under way at once (a ring that loads a block's place
// again behind its products was slower: one row, 14336 inputs, 20.4 us against 18.7).  Their sums meet in LDS, in
// the order of the wavefronts.  For products of few tiles, which are a chain of latencies: the tiled kernel walks K
// step by step.
constexpr int kRowsWaves = 8, kRowsTile = 16, kRowsAhead = 4;

template <int DT, int COLUMNS>
__global__ __launch_bounds__(64 * kRowsWaves) void rows_kernel(Fp8MatmulArgs a)
{
    constexpr int THREADS = 64 * kRowsWaves, NT = COLUMNS / 16, PITCH = COLUMNS + 4;
    __shared__ int first[kMaxExperts + 1], scratch[kMaxExperts + 1];
    __shared__ __align__(16) float sums[kRowsWaves][kRowsTile][PITCH];
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int K = a.K, blocks = (K + kFp8Block - 1) / kFp8Block, n_blocks = (a.N + kFp8Block - 1) / kFp8Block;
    build_tile_list<kRowsTile, THREADS>(first, scratch, a.offsets, a.E, a.rows);
    const int n_tiles = (a.N + COLUMNS - 1) / COLUMNS;
    const int total = __builtin_amdgcn_readfirstlane(mx_items(first[a.E], n_tiles, a.rows, kRowsTile, a.E));
    clear_behind<THREADS>(a, scratch[a.E]);
    for (int item = blockIdx.x; item < total; item += gridDim.x) {
        const TileItem t = item_at<kRowsTile, COLUMNS>(
            first, [&](int e) { return __builtin_amdgcn_readfirstlane(scratch[e]); }, a.E, n_tiles, item, total);
        int source = min(c, t.n - 1);  // from the tile's first row where there are no routes
        if (a.sorted_routes) {
            const int route = a.sorted_routes[t.row0 + source];
            source = route < 0 || route / a.top_k >= a.a_rows ? -1 : route / a.top_k;
        }
        const int64_t a0 = a.sorted_routes ? 0 : t.row0, a_rows = a.sorted_routes ? a.a_rows : t.n;
        const int64_t w0 = (int64_t)t.expert * a.N + t.n0;
        const int w_rows = min(COLUMNS, a.N - t.n0);
        const Span x_span{a.a_codes + a0 * K, (uint32_t)(a_rows * K)}, w_span{a.w_codes + w0 * K, (uint32_t)(w_rows * K)};
        const Span sx_span{(const uint8_t*)(a.a_scales + a0 * blocks), (uint32_t)(a_rows * blocks * 4)};
        const float* const sw_row = a.w_scales + ((int64_t)t.expert * n_blocks + t.n0 / kFp8Block) * blocks;
        const uint32_t x_at = source < 0 ? kMxOutside : source * (uint32_t)K;
        const uint32_t sx_at = source < 0 ? kMxOutside : source * (uint32_t)blocks * 4;
        const uint32_t w_at = c * (uint32_t)K;  // rows behind N: out of bounds
        f32x4 acc[NT] = {};
        for (int b0 = wave; b0 < blocks; b0 += kRowsWaves * kRowsAhead) {
            u32x4 x[kRowsAhead][2], w[kRowsAhead][NT][2];
            float sx[kRowsAhead], sw[kRowsAhead];
#pragma unroll
            for (int q = 0; q < kRowsAhead; ++q) {
                const int b = b0 + q * kRowsWaves;
                const bool there = b < blocks;
                const uint32_t at = there ? (uint32_t)b * kStepBytes : 0;
                const auto xr = x_span.from(at), wr = w_span.from(at);
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // chunks g and g + 4, as in the tiled kernel
                    const uint32_t k = (g + 4 * h) * 16;
                    const bool in = there && at + k < (uint32_t)K;
                    x[q][h] = __builtin_amdgcn_raw_buffer_load_b128(xr, in && source >= 0 ? x_at + k : kMxOutside, 0, 0);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        w[q][n][h] = __builtin_amdgcn_raw_buffer_load_b128(
                            wr, in ? w_at + (uint32_t)(n * 16) * K + k : kMxOutside, 0, 0);
                    }
                }
                sx[q] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                      sx_span.from(there ? b * 4 : 0), there ? sx_at : kMxOutside, 0, 0));
                sw[q] = there ? sw_row[b] : 0.0f;
            }
#pragma unroll
            for (int q = 0; q < kRowsAhead; ++q) {
                const float f = sx[q] * sw[q];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const f32x4 p = block_product(operand(w[q][n][0], w[q][n][1]), operand(x[q][0], x[q][1]));
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][i] = fmaf(f, p[i], acc[n][i]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4*>(&sums[wave][c][n * 16 + g * 4]) = acc[n];
        __syncthreads();
        const int row = threadIdx.x / COLUMNS, column = threadIdx.x % COLUMNS;
        if (row < t.n && t.n0 + column < a.N) {  // t.n <= kRowsTile
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kRowsWaves; ++i) sum += sums[i][row][column];
            ((uint16_t*)a.out)[(int64_t)(t.row0 + row) * a.N + t.n0 + column] = Dt<DT>::from_float(sum);
        }
        __syncthreads();
    }
}

// At most one partial tile for every expert with rows.
int64_t most_items(const Fp8MatmulArgs& a, int bm, int bn)
{
    const int64_t experts = a.E < a.rows ? a.E : a.rows;
    return (experts + (a.rows - experts) / bm) * ((a.N + bn - 1) / bn);
}

template <int DT, int COLUMNS>
hipError_t launch_rows(const Fp8MatmulArgs& a, hipStream_t s)
{
    const int64_t items = most_items(a, kRowsTile, COLUMNS);
    launch(rows_kernel<DT, COLUMNS>, dim3((unsigned)(items < 2 * kMxCUs ? items : 2 * kMxCUs)), dim3(64 * kRowsWaves), s, a);
    return hipGetLastError();
}

// wgs_per_cu: as many as fit by LDS and registers.
template <int DT, int MT, int NT, int WM, int WN, int STAGES>
hipError_t launch_tiled(const Fp8MatmulArgs& a, int wgs_per_cu, hipStream_t s)
{
    constexpr int BM = 16 * MT * WM, BN = 16 * NT * WN;
    int64_t grid = (most_items(a, BM, BN) + 7) / 8 * 8;
    if (grid > kMxCUs * wgs_per_cu) grid = kMxCUs * wgs_per_cu;
    const dim3 threads(64 * WM * WN);
    if (a.K % kFp8Block == 0 && a.K / kFp8Block >= STAGES) {
        launch(tiled_kernel<DT, MT, NT, WM, WN, STAGES, true>, dim3((unsigned)grid), threads, s, a);
    } else {
        launch(tiled_kernel<DT, MT, NT, WM, WN, STAGES, false>, dim3((unsigned)grid), threads, s, a);
    }
    return hipGetLastError();
}

template <int DT>
hipError_t launch_by_shape(const Fp8MatmulArgs& a, hipStream_t s)
{
    switch (fp8_tile(a.E, a.N, a.rows)) {
    case Fp8Tile::kRows16: return launch_rows<DT, 16>(a, s);
    case Fp8Tile::kRows32: return launch_rows<DT, 32>(a, s);
    case Fp8Tile::k32x64s4: return launch_tiled<DT, 2, 2, 1, 2, 4>(a, 2, s);
    case Fp8Tile::k64x128s3: return launch_tiled<DT, 2, 4, 2, 2, 3>(a, 2, s);
    case Fp8Tile::k128x128s2: return launch_tiled<DT, 4, 4, 2, 2, 2>(a, 2, s);
    case Fp8Tile::k256x256s2: break;
    }
    return launch_tiled<DT, 4, 8, 4, 2, 2>(a, 1, s);
}

}  // namespace

hipError_t launch_fp8_matmul(const Fp8MatmulArgs& a, hipStream_t s)
{
    return a.dtype == kBF16 ? launch_by_shape<kBF16>(a, s) : launch_by_shape<kF16>(a, s);
}

}  // namespace qmoe
