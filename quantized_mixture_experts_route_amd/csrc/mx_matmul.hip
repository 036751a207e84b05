// mx_matmul.hip -- grouped product of MXFP4 rows with MXFP4 expert weights:
//   out[r, n] = sum_b 2^(sa(r,b) + sw(e,n,b) - 254) sum_{i in block b} a(r,i) w(e,n,i)
// for the rows offsets[e] <= r < offsets[e+1] of expert e, accumulated in
// float32 on the scaled matrix instruction and rounded once to the output's
// type; rows behind the last expert's are zero.
//
// v_mfma_scale_f32_32x32x64 with e2m1 operands: lane l = 32 h + c supplies
// row c of A and row c of W, each one block of 32 codes (16 bytes) with its
// scale byte; the lane half h is the block of the two that the step contracts.
// The result: register i of lane l is row 8 (i/4) + 4 h + i%4, column c.
#include "expert_ops.h"
#include "mx_shape.h"
#include "qmoe_internal.h"
#include "rowio.h"

namespace qmoe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr int kMaxExperts = 1024;
constexpr int kE2M1 = 4;  // operand format code of the scaled matrix instructions

__device__ inline i32x8 operand(u32x4 v)
{
    return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

// ---------------------------------------------------------------- tiled kernel
// A workgroup of WM x WN wavefronts computes BM = 32 MT WM rows against
// BN = 32 NT WN weight rows; a wavefront MT x NT blocks of 32 x 32.  W is the
// instruction's first operand, so a lane's registers run along n and its
// results leave as 16-byte stores.
//
// K runs in steps of 256 values: 128 bytes of codes a row, a whole cache line
// (64-byte pieces read every line twice from L2), written to LDS by the load
// itself (buffer_load ... lds) into one of STAGES stages.  A step is four
// quarters of 64 values; a quarter's operands are read while the matrix
// instructions of the quarter before run.  The one barrier of a step stands
// before its last quarter: then every operand of the step is in registers, its
// stage takes the loads of the step STAGES ahead, and the next step has landed.
// Loads run on over the end of a tile into the workgroup's next one, so only
// its first tile waits for memory.  Two stages where tiles are large (LDS);
// four where few rows leave latency as the bound.
//
// A group of four steps needs 32 bytes of scales a row.  With two stages there
// is one buffer: its last read is behind the group's second barrier, the next
// group's load is issued behind the third and has landed at the fourth.  With
// four stages there are two, loaded a group ahead.  A lane reads 8 bytes a step
// and picks its byte by shift and operand select.  With two stages a tile may end
// behind half a group (8192 x 8192 x 1536 over 8 experts: 108 -> 99 us).
//
// LDS rows are 128 bytes (32 banks); the 16-byte chunk of row r sits in slot
// chunk ^ (r / 2 % 8), so that 16 rows read at one chunk cover all 64 banks.
// Scale rows of 32 bytes swap their halves where r / 8 is odd.
//
// WHOLE: K fills its steps (a multiple of 1024, with two stages of 512 from 1024
// on) and the scale rows are 16-byte aligned, so scales take the direct path to
// LDS too and no step has a tail.  Otherwise scales go through registers, and
// codes behind the row's end are read out of the buffer's bounds, which gives 0.
//
// What bounds it.  8192 x 28672 x 4096 over 8 skewed experts: 572 to 583 us on
// its own (3.3 PFLOP/s), 610 us on average over longer runs, where the card's
// clock moves a launch between 570 and 757 us.  1.15 million cycles, the matrix
// units busy in 41% of them, at about 2.0 GHz; an earlier step that took out a
// sixth of the cycles gained 4% of the time, so power has a part in it.  So has
// memory: 991 MB are read where the operands hold 508, with 472 MB written 290 us
// of traffic.  Why the second half is read has not been found.  8192^3, one
// expert: 266 us, 4.1 PFLOP/s.  Rows that do not start on lines cost more: K =
// 4064 at N 16384, 8192 rows 370 to 380 us, K = 4096 303.  Short K leaves the
// stores uncovered: 8192 x 8192 x 1536 over 8 experts 95 us, 2.5 times the floor.
// Few rows: HBM; 60 rows over 512 experts 22 us for 97 MB (4.4 TB/s).
constexpr int kStepBytes = 128;  // codes of one row and step
constexpr int kGroupSteps = 4;   // steps whose scales are loaded together
constexpr int kScaleBytes = 32;  // ... and their bytes a row

// Bytes of codes or scales that a tile reads; its descriptor from byte `at` on.
struct Span {
    const uint8_t* base;
    uint32_t bytes;
    __device__ inline __amdgpu_buffer_rsrc_t from(uint32_t at) const
    {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base + at), 0, mx_bytes_left(bytes, at), 0x00020000);
    }
};

// The lane, worked out where it stands.  Addresses made from it there need no register over the
// K loop and the stores; those that the compiler keeps are spilled, and a reload waits for every
// load and store before it.
__device__ inline int lane_now()
{
    int zero = 0;
    asm volatile("" : "+s"(zero));
    return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, zero));
}

// 16 bytes a lane from the buffer to LDS at `to` + 16 * lane (to is uniform); zeros where the lane's
// offset is not in the buffer.
__device__ inline void load_to_lds(__amdgpu_buffer_rsrc_t r, uint32_t lane_offset, void* to)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 16, lane_offset, 0, 0, 0);
}

template <int DT>
__device__ inline uint32_t pack_pair(float lo, float hi)
{
    if constexpr (DT == kBF16) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
    } else {
        return pack2(Dt<kF16>::from_float(lo), Dt<kF16>::from_float(hi));
    }
}

// Stores one block of 32 x 32 results: lane (c, half) holds row c, columns
// 8 q + 4 half + i in register 4 q + i.  `out` is the block's first row and
// column; rows and cols say how many of them exist (WHOLE: all 32).
template <int DT, bool WHOLE>
__device__ inline void store_block(typename RowType<DT>::Raw* out, int N, int rows, int cols, const f32x16& acc, int lane)
{
    typedef typename RowType<DT>::Raw Raw;
    constexpr int V = 16 / sizeof(Raw);
    const int c = lane & 31, half = lane >> 5;
    auto store = [&](int row, int col, const u32x4& v) {
        if (!WHOLE && row >= rows) return;
        RowVec<Raw, V> y;
        __builtin_memcpy(&y, &v, 16);
        Raw* p = out + (int64_t)row * N + col;
        if (WHOLE || col + V <= cols) {
            store_vec<Raw, V>(p, y);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (col + i < cols) p[i] = y.v[i];
            }
        }
    };
    if constexpr (DT == kF32) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            u32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __builtin_bit_cast(uint32_t, (float)acc[4 * q + i]);
            store(c, 8 * q + 4 * half, v);
        }
    } else {
        // the halves trade four columns, so that each lane holds eight neighbours: v[0] columns
        // 8 half .. 8 half + 7, v[1] the same 16 further on
        u32x4 v[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const auto t = __builtin_amdgcn_permlane32_swap(
                    pack_pair<DT>(acc[8 * q + 2 * i], acc[8 * q + 2 * i + 1]),
                    pack_pair<DT>(acc[8 * q + 4 + 2 * i], acc[8 * q + 5 + 2 * i]), false, false);
                v[q][i] = t[0];
                v[q][2 + i] = t[1];
            }
        }
        // then rows 16..31 trade with rows 0..15: a store writes 16 rows of 64 neighbouring bytes
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const auto t = __builtin_amdgcn_permlane16_swap(v[0][i], v[1][i], false, false);
            v[0][i] = t[0];
            v[1][i] = t[1];
        }
        const int col = 8 * half + 16 * ((lane >> 4) & 1);
        if (WHOLE && (((uintptr_t)out | (uintptr_t)N << 1) & 2)) {
            // rows that start between two words: they are stored one column on, in whole words, with
            // the first column of the neighbour's eight at the end; columns 0 and 31 on their own
            // (18498 rows of 2175 columns: 90 us, with 16-byte stores that split words 105)
            const int neighbour = lane < 32 ? lane + 32 : lane - 16;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                Raw* p = out + (int64_t)(16 * q + (lane & 15)) * N + col;
                const uint32_t next = (uint32_t)__shfl((int)v[q][0], neighbour, kWave);
                const bool odd = (uintptr_t)p & 2;
                if (odd) {
                    if (col == 0) p[0] = (Raw)v[q][0];
                    if (col == 24) p[7] = (Raw)(v[q][3] >> 16);
                    v[q] = u32x4{v[q][0] >> 16 | v[q][1] << 16, v[q][1] >> 16 | v[q][2] << 16,
                                 v[q][2] >> 16 | v[q][3] << 16, v[q][3] >> 16 | next << 16};
                }
                __builtin_memcpy(p + odd, &v[q], 12);
                if (!odd || col < 24) __builtin_memcpy(p + odd + 6, (const char*)&v[q] + 12, 4);
            }
            return;
        }
        store(lane & 15, col, v[0]);
        store(16 + (lane & 15), col, v[1]);
    }
}

// The 16 scale bytes at p, `chunk` bytes into a row that has `left` more from
// there: 0 behind the row's end, and nothing read outside the row.
__device__ inline u32x4 load_scale_chunk(const uint8_t* p, int chunk, int left)
{
    uint64_t lo = 0, hi = 0;
    if (left >= 16) {
        __builtin_memcpy(&lo, p, 8);
        __builtin_memcpy(&hi, p + 8, 8);
    } else if (left > 0 && chunk > 0) {  // the row's last 16 bytes, shifted down
        __builtin_memcpy(&lo, p + left - 16, 8);
        __builtin_memcpy(&hi, p + left - 8, 8);
        const int shift = 8 * (16 - left);
        lo = shift < 64 ? lo >> shift | hi << (64 - shift) : hi >> (shift - 64);
        hi = shift < 64 ? hi >> shift : 0;
    } else if (left > 0) {  // a row of fewer than 16: one load for each bit of its length
        uint64_t v8 = 0;
        uint32_t v4 = 0;
        uint16_t v2 = 0;
        uint8_t v1 = 0;
        if (left & 8) __builtin_memcpy(&v8, p, 8);
        if (left & 4) __builtin_memcpy(&v4, p + (left & 8), 4);
        if (left & 2) __builtin_memcpy(&v2, p + (left & 12), 2);
        if (left & 1) v1 = p[left - 1];
        const uint64_t rest = (uint64_t)v4 | (uint64_t)v2 << (8 * (left & 4)) | (uint64_t)v1 << (8 * (left & 6));
        lo = left & 8 ? v8 : rest;
        hi = left & 8 ? rest : 0;
    }
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// m-tiles of each expert in LDS: first[e] .. first[e + 1] of the tile list.
// Offsets are clamped to [0, rows] and mx_items() bounds the count, so no table
// content leads outside the output.  scratch: E + 1 words of LDS.
template <int BM, int THREADS>
__device__ void build_tile_list(int* first, int* scratch, const int32_t* offsets, int E, int rows)
{
    for (int e = threadIdx.x; e <= E; e += THREADS) {
        scratch[e] = offsets ? min(max(offsets[e], 0), rows) : e * rows;
    }
    __syncthreads();
    if (threadIdx.x < kWave) {
        const int lane = threadIdx.x, per = (E + kWave - 1) / kWave;  // consecutive experts a lane
        auto tiles = [&](int e) { return e < E ? (max(scratch[e + 1] - scratch[e], 0) + BM - 1) / BM : 0; };
        int sum = 0;
        for (int i = 0; i < per; ++i) sum += tiles(lane * per + i);
        int incl = sum;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int y = __shfl_up(incl, d, kWave);
            if (lane >= d) incl += y;
        }
        int run = incl - sum;
        for (int i = 0; i < per; ++i) {
            const int e = lane * per + i;
            if (e < E) first[e] = run;
            run += tiles(e);
        }
        if (lane == kWave - 1) first[E] = run;
    }
    __syncthreads();
}

// Reads through it are scalar and wait for no vector memory; what it points to does not change
// while the kernel runs.
__device__ inline const __attribute__((address_space(4))) int32_t* constant(const int32_t* p)
{
    return (const __attribute__((address_space(4))) int32_t*)p;
}

// The workgroups that run on a die at a time (32 of the largest tile) share rows and weights in its
// L2: bands of 8 m-tiles make that about 8 row blocks and 4 weight blocks, in place of one column of
// 32 (8192^3: 281 -> 246 us; bands of 4 and of 12 were slower).
constexpr int kBand = 8;

struct TileItem {
    int expert;
    int row0;
    int n;   // rows; 0: no item
    int n0;  // first column
};

// offset(e) gives expert e's clamped offset.
template <int BM, int BN, class Offset>
__device__ TileItem item_at(const int* first, Offset offset, int E, int n_tiles, int item, int end)
{
    if (item >= end) return TileItem{0, 0, 0, 0};
    int lo = 0, hi = E - 1;  // the last expert whose first item is <= item
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] * n_tiles <= item) lo = mid; else hi = mid - 1;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    const int base = __builtin_amdgcn_readfirstlane(first[lo]);
    const int m_tiles = __builtin_amdgcn_readfirstlane(first[lo + 1]) - base;
    // bands of up to kBand m-tiles, in a band neighbouring items share the weights
    int local = item - base * n_tiles;
    int m0 = 0, band = m_tiles;
    if (m_tiles > kBand) {
        const int bands = (m_tiles + kBand - 1) / kBand;
        band = (m_tiles + bands - 1) / bands;
        m0 = local / (band * n_tiles) * band;
        local -= m0 * n_tiles;
        band = min(band, m_tiles - m0);
    }
    const int nt = local / band;
    const int r_lo = offset(lo), r_hi = offset(lo + 1);
    const int row0 = r_lo + (m0 + local - nt * band) * BM;
    return TileItem{lo, row0, min(BM, r_hi - row0), nt * BN};
}

template <int DT, int MT, int NT, int WM, int WN, int STAGES, bool WHOLE>
__global__ __launch_bounds__(64 * WM * WN) void tiled_kernel(MxMatmulArgs a)
{
    typedef typename RowType<DT>::Raw Raw;
    constexpr int BM = 32 * MT * WM, BN = 32 * NT * WN, ROWS = BM + BN;
    constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
    constexpr int LOADS = ROWS / 8 / WAVES;     // code loads of a wavefront and step: 8 rows each
    constexpr int LOADS_A = BM / 8 / WAVES;
    constexpr int SCALE_LOADS = (ROWS / 32 + WAVES - 1) / WAVES;  // scale loads: 32 rows each
    // The tile that fills the registers: addresses by lane_now, the next item found in a tile's last
    // steps, and a tile's first barrier does not wait for the stores of the tile before it (8192 x
    // 28672 x 4096 over 8 experts: 583 -> 567 us).  With scales through registers it gained nothing.
    constexpr bool FULL = WHOLE && MT * NT >= 8;
    static_assert(!FULL || (STAGES == 2 && BM <= THREADS), "one route a thread, taken behind start_tile");
    static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0 && WAVES % 2 == 0, "load split");

    // one array for all of it: between arrays of their own the compiler tells apart what a load to
    // LDS writes and waits for every such load before it reads LDS
    constexpr int SCALE_BUFFERS = STAGES / 2;
    constexpr int STAGE = ROWS * kStepBytes, SCALES = STAGES * STAGE;
    constexpr int LIST = SCALES + SCALE_BUFFERS * ROWS * kScaleBytes, SOURCE = LIST + (kMaxExperts + 1) * 4;
    __shared__ __align__(16) uint8_t lds[SOURCE + 2 * BM * 4];
    uint8_t* const scales = lds + SCALES;
    int* const first = reinterpret_cast<int*>(lds + LIST);
    int* const source = reinterpret_cast<int*>(lds + SOURCE);

    const int lane = threadIdx.x & 63;
    auto lane_here = [&]() { return FULL ? lane_now() : lane; };
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int K2 = a.K / 2, blocks = a.K / 32;
    // whole groups of steps; with two stages the last may be half a group, but not the only one: the
    // loading side is two steps ahead and would be at its end before the tile begins
    const bool half_group = mx_half_group(STAGES, a.K);
    const int steps = (a.K + 256 * kGroupSteps - 1) / (256 * kGroupSteps) * kGroupSteps - (half_group ? 2 : 0);

    // the last stage's space, not loaded before the first barrier, holds the offsets for the first item
    int* const scratch = reinterpret_cast<int*>(lds + (STAGES - 1) * STAGE);
    build_tile_list<BM, THREADS>(first, scratch, a.offsets, a.E, a.rows);
    const int n_tiles = (a.N + BN - 1) / BN;
    const int total = mx_items(first[a.E], n_tiles, a.rows, BM, a.E);
    // workgroups go to the 8 dies in turn: each die takes one run of items, so
    // that the workgroups of a die share rows and weights in its L2
    const int per_die = gridDim.x / 8;
    const int die = blockIdx.x % 8;
    const int end = (int)((int64_t)total * (die + 1) / 8);
    int next_item = (int)((int64_t)total * die / 8) + blockIdx.x / 8;

    // rows behind the last expert's are zero
    if (a.offsets) {
        const int64_t lo = (int64_t)min(max(a.offsets[a.E], 0), a.rows) * a.N, hi = (int64_t)a.rows * a.N;
        constexpr int V = 16 / sizeof(Raw);
        for (int64_t i = lo + (blockIdx.x * (int64_t)THREADS + threadIdx.x) * V; i < hi; i += (int64_t)gridDim.x * THREADS * V) {
            if (i + V <= hi) {
                store_vec<Raw, V>((Raw*)a.out + i, RowVec<Raw, V>{});
            } else {
                for (int64_t q = i; q < hi; ++q) ((Raw*)a.out)[q] = 0;
            }
        }
    }

    // ---- the loading side: an item and a step, up to STAGES steps ahead
    TileItem load_tile;
    int load_step = 0;
    auto load_chunk = [&](int id) { return (uint32_t)((id & 7) ^ ((wave & 1) * 4 + (id >> 4))) * 16; };
    auto scale_chunk = [](int id) { return (uint32_t)((id & 1) ^ ((id >> 4) & 1)) * 16; };
    uint32_t code_at[LOADS_A];      // byte offset of the lane's chunk at step 0
    const uint32_t w_at = (wave * 8 + (lane >> 3)) * (uint32_t)K2 + load_chunk(lane);  // rows behind N: out of bounds
    uint32_t scale_at[SCALE_LOADS]; // byte offset of the lane's half of a scale row's group
    Span a_span, w_span, as_span, ws_span;  // codes and scales of the loading side's tile

    // The next item, and in LDS its rows' source rows in a (from the tile's first row where there
    // are no routes; -1: outside; rows behind the tile's repeat its last).  Found between two tiles,
    // where registers are free; FULL: in the tile's last steps, so that the routes are there by then.
    TileItem next_tile;
    int found = 0;  // tables of source rows take turns
    auto find_tile = [&](auto offset) {
        next_tile = item_at<BM, BN>(first, offset, a.E, n_tiles, next_item, end);
        next_item += per_die;
        found ^= BM;
    };
    auto offset_of = [&](int e) { return a.offsets ? min(max(constant(a.offsets)[e], 0), a.rows) : e * a.rows; };
    auto route_of = [&](int r) {
        r = min(r, next_tile.n - 1);
        return a.sorted_routes ? a.sorted_routes[next_tile.row0 + r] : r;
    };
    auto set_source = [&](int r, int route) {
        if (a.sorted_routes) route = route < 0 || route / a.top_k >= a.a_rows ? -1 : route / a.top_k;
        source[found + r] = route;
    };
    auto find_rows = [&]() {
        for (int r = wave * kWave + lane_here(); r < BM && next_tile.n > 0; r += THREADS) set_source(r, route_of(r));
    };
    int route = 0;  // FULL: on its way from the tile's last steps on
    auto start_tile = [&]() {  // all but what goes by the source rows
        load_tile = next_tile;
        load_step = 0;
        const TileItem& t = load_tile;
        const bool on = t.n > 0;
        const int w_rows = on ? min(BN, a.N - t.n0) : 0;
        const int64_t w0 = on ? (int64_t)t.expert * a.N + t.n0 : 0;
        w_span = Span{a.w_codes + w0 * K2, (uint32_t)(w_rows * K2)};
        ws_span = Span{a.w_scales + w0 * blocks, (uint32_t)(w_rows * blocks)};
        const int64_t a0 = a.sorted_routes ? 0 : t.row0;
        const int64_t a_rows = !on ? 0 : a.sorted_routes ? a.a_rows : t.n;
        a_span = Span{a.a_codes + a0 * K2, (uint32_t)(a_rows * K2)};
        as_span = Span{a.a_scales + a0 * blocks, (uint32_t)(a_rows * blocks)};
    };
    auto start_rows = [&]() {
        const int id = lane_here();
        const int w_rows = min(BN, a.N - load_tile.n0);
#pragma unroll
        for (int j = 0; j < LOADS_A; ++j) {
            const int row = source[found + (j * WAVES + wave) * 8 + (id >> 3)];
            code_at[j] = row < 0 ? kMxOutside : row * (uint32_t)K2 + load_chunk(id);
        }
#pragma unroll
        for (int j = 0; j < SCALE_LOADS; ++j) {
            const int r0 = (j * WAVES + wave) * 32;
            const int row = r0 < BM ? source[found + r0 + (id >> 1)] : min(r0 - BM + (id >> 1), w_rows - 1);
            scale_at[j] = row < 0 ? kMxOutside : row * (uint32_t)blocks + scale_chunk(id);
        }
    };
    // codes of the loading side's step into stage `stage`; loads [from, to) of the wavefront
    auto load_part = [&](int stage, auto from, auto to) {
        const uint32_t at = (uint32_t)load_step * kStepBytes;
        const __amdgpu_buffer_rsrc_t a_buf = a_span.from(at), w_buf = w_span.from(at);
#pragma unroll
        for (int j = decltype(from)::value; j < decltype(to)::value; ++j) {
            uint32_t off = j < LOADS_A ? code_at[j < LOADS_A ? j : 0] : w_at + (uint32_t)((j - LOADS_A) * WAVES * 8) * K2;
            if constexpr (!WHOLE) {
                if (at + load_chunk(lane) >= (uint32_t)K2) off = kMxOutside;
            }
            load_to_lds(j < LOADS_A ? a_buf : w_buf, off, lds + stage * STAGE + (j * WAVES + wave) * 8 * kStepBytes);
        }
    };
    constexpr std::integral_constant<int, 0> kFirst;
    constexpr std::integral_constant<int, LOADS_A> kWeights;
    constexpr std::integral_constant<int, LOADS> kEnd;
    auto load_codes = [&](int stage) { load_part(stage, kFirst, kEnd); };
    u32x4 scale_regs[WHOLE ? 1 : SCALE_LOADS];
    auto load_scales = [&](int buffer) {  // of the group that starts at the loading side's step
        const int at = load_step * 8;
        const __amdgpu_buffer_rsrc_t as_buf = as_span.from(at), ws_buf = ws_span.from(at);
#pragma unroll
        for (int j = 0; j < SCALE_LOADS; ++j) {
            const int r0 = (j * WAVES + wave) * 32;
            if (r0 >= ROWS) continue;
            if constexpr (WHOLE) {
                load_to_lds(r0 < BM ? as_buf : ws_buf, scale_at[j], scales + (buffer * ROWS + r0) * kScaleBytes);
            } else {
                u32x4 v = {};
                if (load_tile.n > 0 && scale_at[j] != kMxOutside) {
                    const int chunk = at + scale_chunk(lane);
                    v = load_scale_chunk((r0 < BM ? as_span.base : ws_span.base) + scale_at[j] + at, chunk, blocks - chunk);
                }
                scale_regs[j] = v;
            }
        }
    };
    auto store_scales = [&](int buffer) {  // the register path's second half
        if constexpr (!WHOLE) {
#pragma unroll
            for (int j = 0; j < SCALE_LOADS; ++j) {
                const int r0 = (j * WAVES + wave) * 32;
                if (r0 < ROWS) {
                    *reinterpret_cast<u32x4*>(scales + (buffer * ROWS + r0 + (lane >> 1)) * kScaleBytes + (lane & 1) * 16) = scale_regs[j];
                }
            }
        }
    };
    find_tile([&](int e) { return scratch[e]; });
    start_tile();
    load_part(0, kWeights, kEnd);  // weights do not wait for the table of rows
    find_rows();
    __syncthreads();
    start_rows();
    load_part(0, kFirst, kWeights);
    load_scales(0);
    store_scales(0);
    ++load_step;
#pragma unroll
    for (int i = 1; i < STAGES - 1; ++i) {
        load_codes(i);
        ++load_step;
    }
    find_tile(offset_of);
    find_rows();

    // addresses of the reads: chunk 2 t + half of row c
    uint32_t read_at[4], scales_at, half8;
    auto set_reads = [&]() {
        const int id = lane_here(), row = id & 31, high = id >> 5;
#pragma unroll
        for (int t = 0; t < 4; ++t) read_at[t] = row * (uint32_t)kStepBytes + (((2 * t + high) ^ ((row >> 1) & 7)) * 16);
        scales_at = row * kScaleBytes + ((row >> 3) & 1) * 16;
        half8 = 8 * high;
    };
    set_reads();
    // Operands of two quarters.  The largest tile with scales through registers has no room for them:
    // there a quarter's operands are read right before it (8192 x 16384 x 4064: 456 -> 412 us when taken up).
    constexpr bool AHEAD = WHOLE || MT * NT < 8;
    u32x4 w[AHEAD ? 2 : 1][NT], x[AHEAD ? 2 : 1][MT];
    u32x2 sw[2][NT], sa[2][MT];
    auto read_codes = [&](int stage, int t) {  // operands of quarter t
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            w[AHEAD ? t & 1 : 0][i] = *reinterpret_cast<const u32x4*>(lds + stage * STAGE + (BM + (wn * NT + i) * 32) * kStepBytes + read_at[t]);
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            x[AHEAD ? t & 1 : 0][j] = *reinterpret_cast<const u32x4*>(lds + stage * STAGE + ((wm * MT + j) * 32) * kStepBytes + read_at[t]);
        }
    };
    // scale bytes of one step of the group; byte 0 and 2 of a word are the lane's
    auto read_scales = [&](int to, int buffer, int step) {
        const uint8_t* from = scales + buffer * ROWS * kScaleBytes + (scales_at ^ (step / 2 * 16)) + step % 2 * 8;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            sw[to][i] = *reinterpret_cast<const u32x2*>(from + (BM + (wn * NT + i) * 32) * kScaleBytes) >> half8;
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            sa[to][j] = *reinterpret_cast<const u32x2*>(from + ((wm * MT + j) * 32) * kScaleBytes) >> half8;
        }
    };
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((STAGES - 2) * LOADS) : "memory");
    load_codes(STAGES - 1);
    ++load_step;
    read_scales(0, 0, 0);
    if (AHEAD) read_codes(0, 0);
    int buffer = 0;
    // Stores count with the loads, in order of issue.  The loads that a tile's first barrier waits for
    // were issued before the stores of the tile before it, which may run on there: `stored` says that
    // there were at least STORES of them (no block was cut).
    constexpr int STORES = MT * NT * (DT == kF32 ? 4 : 2);
    static_assert((STAGES - 2) * LOADS + STORES < 64, "the counter's range");
    bool stored = false;
    while (load_tile.n > 0) {
        const TileItem tile = load_tile;
        set_reads();
        // wavefronts whose rows lie behind the tile's leave their products out; the two wavefronts of
        // a SIMD hold different row blocks, so a half-full tile takes half the time
        const bool active = wm * MT * 32 < tile.n;
        f32x16 acc[NT][MT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x16{};
        }
        for (int g = 0; g < steps; g += kGroupSteps) {
            const bool half_g = half_group && g + 2 == steps;
#pragma unroll
            for (int s = 0; s < kGroupSteps; ++s) {
                const bool last = s == kGroupSteps - 1 || (s == 1 && half_g);  // of the group
                auto multiply = [&](auto quarter) {
                    constexpr int t = decltype(quarter)::value;
                    if (!active || (!WHOLE && (g + s) * 256 + t * 64 >= a.K)) return;
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
#pragma unroll
                        for (int j = 0; j < MT; ++j) {
                            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                operand(w[AHEAD ? t & 1 : 0][i]), operand(x[AHEAD ? t & 1 : 0][j]), acc[i][j], kE2M1, kE2M1, 2 * (t & 1),
                                (int)sw[s & 1][i][t >> 1], 2 * (t & 1), (int)sa[s & 1][j][t >> 1]);
                            // keeps the product in this place: without it the compiler moves the
                            // products of a step behind the branches and reads that follow
                            asm volatile("" : "+v"(acc[i][j]));
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                };
                // reads stand before the products that they hide behind; unfenced they sink to their use
                const int next_buffer = SCALE_BUFFERS == 2 ? buffer ^ 1 : 0;
                read_codes(s % STAGES, AHEAD ? 1 : 0);
                if (last) store_scales(next_buffer);
                __builtin_amdgcn_sched_barrier(0);
                multiply(std::integral_constant<int, 0>{});
                read_codes(s % STAGES, AHEAD ? 2 : 1);
                if (!last) read_scales((s + 1) & 1, buffer, s + 1);
                __builtin_amdgcn_sched_barrier(0);
                multiply(std::integral_constant<int, 1>{});
                read_codes(s % STAGES, AHEAD ? 3 : 2);
                __builtin_amdgcn_sched_barrier(0);
                multiply(std::integral_constant<int, 2>{});
                if (!AHEAD) read_codes(s % STAGES, 3);
                // the next step has landed once no more than the loads behind it are left
                if (FULL && s == 0 && stored) {
                    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((STAGES - 2) * LOADS + STORES) : "memory");
                    stored = false;
                } else {
                    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((STAGES - 2) * LOADS) : "memory");
                }
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                if (AHEAD) read_codes((s + 1) % STAGES, 0);
                if (last) read_scales(0, next_buffer, 0);
                __builtin_amdgcn_sched_barrier(0);
                if (FULL && s % 2 == 0 && load_step == 0) {
                    find_tile(offset_of);
                    if (next_tile.n > 0 && wave * kWave < BM) route = route_of(wave * kWave + lane_now());
                }
                // the step loaded here is STAGES ahead: the first of a group brings the group's scales
                if (s == kGroupSteps - STAGES || (s == 0 && half_g)) load_scales(next_buffer);
                load_codes(s % STAGES);
                multiply(std::integral_constant<int, 3>{});
                ++load_step;
                // tiles end with a group or, of two stages, behind its half
                if (((s + STAGES) % kGroupSteps == kGroupSteps - 1 || (STAGES == 2 && s == 3)) && load_step == steps) {
                    start_tile();
                    start_rows();
                }
                if (s == 1 && half_g) break;
            }
            buffer = SCALE_BUFFERS == 2 ? buffer ^ 1 : 0;
        }
        const int id = lane_here();
        if constexpr (FULL) {
            if (next_tile.n > 0 && wave * kWave < BM) set_source(wave * kWave + id, route);
        } else {
            find_tile(offset_of);
            find_rows();
        }
        stored = tile.n >= (wm * MT + MT) * 32 && a.N - tile.n0 >= (wn * NT + NT) * 32;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int m0 = (wm * MT + j) * 32;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int n = tile.n0 + (wn * NT + i) * 32;
                Raw* out = (Raw*)a.out + (int64_t)(tile.row0 + m0) * a.N + n;
                if (tile.n - m0 >= 32 && a.N - n >= 32) {
                    store_block<DT, true>(out, a.N, 32, 32, acc[i][j], id);
                } else {
                    store_block<DT, false>(out, a.N, tile.n - m0, a.N - n, acc[i][j], id);
                }
            }
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may reach LDS behind the workgroup's end
}

// wgs_per_cu: as many as fit by LDS and registers.
template <int DT, int MT, int NT, int WM, int WN, int STAGES>
hipError_t launch_tiled(const MxMatmulArgs& a, int wgs_per_cu, hipStream_t s)
{
    constexpr int BM = 32 * MT * WM, BN = 32 * NT * WN;
    // at most one partial tile for every expert with rows
    const int64_t experts = a.E < a.rows ? a.E : a.rows;
    const int64_t items = (experts + (a.rows - experts) / BM) * ((a.N + BN - 1) / BN);
    int64_t grid = (items + 7) / 8 * 8;
    if (grid > kMxCUs * wgs_per_cu) grid = kMxCUs * wgs_per_cu;
    if (mx_whole(STAGES, a.K, a.a_scales, a.w_scales)) launch(tiled_kernel<DT, MT, NT, WM, WN, STAGES, true>, dim3((unsigned)grid), dim3(64 * WM * WN), s, a);
    else launch(tiled_kernel<DT, MT, NT, WM, WN, STAGES, false>, dim3((unsigned)grid), dim3(64 * WM * WN), s, a);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_by_shape(const MxMatmulArgs& a, hipStream_t s)
{
    switch (mx_tile(a.E, a.N, a.K, a.rows)) {
    case MxTile::k32x64s4: return launch_tiled<DT, 1, 1, 1, 2, 4>(a, 2, s);
    case MxTile::k64x128s4: return launch_tiled<DT, 1, 2, 2, 2, 4>(a, 1, s);
    case MxTile::k128x128s4: return launch_tiled<DT, 2, 2, 2, 2, 4>(a, 1, s);
    case MxTile::k64x128s2: return launch_tiled<DT, 1, 2, 2, 2, 2>(a, 2, s);
    case MxTile::k128x128s2: return launch_tiled<DT, 2, 2, 2, 2, 2>(a, 2, s);
    case MxTile::k256x256s2: break;
    }
    return launch_tiled<DT, 2, 4, 4, 2, 2>(a, 1, s);
}

}  // namespace

hipError_t launch_mx_matmul(const MxMatmulArgs& a, hipStream_t s)
{
    if (a.dtype == kF32) return launch_by_shape<kF32>(a, s);
    if (a.dtype == kBF16) return launch_by_shape<kBF16>(a, s);
    return launch_by_shape<kF16>(a, s);
}

}  // namespace qmoe
