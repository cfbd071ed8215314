// Product of 8-bit rows with 8-bit weights:
//   out[m][n] = x_scales[m] w_scales[n] sum_k x[m][k] w[n][k],
// the sum whole, in 32 bits. It is rounded to float32 and multiplied by the product
// of the scales' mantissas, their exponents are added behind that: three roundings
// of half a step, and neither the product of two scales nor that of one with the sum
// leaves float32's range on the way to a result inside it.
//
// Both kernels take 16 weight rows as the first operand of a matrix instruction
// (16 x 16 results, 64 products each) and 16 rows of x as the second: a lane then
// holds four columns of one row of the result, those of weight rows 4 g to 4 g + 3,
// g = lane / 16.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "kld_answer.h"

namespace kldk {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 multiply(i32x4 w, i32x4 x, i32x4 sum) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, sum, 0, 0, 0);
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__bf16* p, float v) { *p = static_cast<__bf16>(v); }

// A scale as mantissa in [1/2, 1) and exponent; 0, NaN and infinities are their own mantissas.
struct Scale {
    float m;
    int e;
};
__device__ __forceinline__ Scale split(float s) {
    return Scale{__builtin_amdgcn_frexp_mantf(s), __builtin_amdgcn_frexp_expf(s)};
}
// Whether the exponents may be left in: the product of two such scales is a normal number.
__device__ __forceinline__ bool ordinary(float s) {
    return s == 0.0f || (fabsf(s) >= 0x1p-60f && fabsf(s) <= 0x1p60f);
}
__device__ __forceinline__ float scaled(int sum, Scale x, Scale w) {
    return __builtin_amdgcn_ldexpf(static_cast<float>(sum) * (x.m * w.m), x.e + w.e);
}

// Bytes [k, k + 16) of a row, zero from `dim` on; any alignment. A chunk that the end
// cuts is taken from the row's last 16 bytes.
__device__ __forceinline__ i32x4 load16(const int8_t* row, int k, int dim) {
    i32x4 v = {0, 0, 0, 0};
    if (k + 16 <= dim) {
        memcpy(&v, row + k, 16);
    } else if (k < dim) {
        unsigned __int128 last = 0;
        if (dim >= 16) {
            memcpy(&last, row + dim - 16, 16);
            last >>= 8 * (k + 16 - dim);
        } else {
#pragma unroll 1
            for (int i = dim; i-- > k;) last = last << 8 | static_cast<uint8_t>(row[i]);
        }
        memcpy(&v, &last, 16);
    }
    return v;
}

// A value that is the same in all lanes, in a scalar register: the compiler's own 64-bit
// division leaves it in vector registers.
__device__ __forceinline__ int uniform(int64_t x) { return __builtin_amdgcn_readfirstlane(static_cast<int>(x)); }
__device__ __forceinline__ const int8_t* uniform(const int8_t* p) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(u)));
    const uint64_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(u >> 32)));
    return reinterpret_cast<const int8_t*>(hi << 32 | lo);
}

// x, as a value that the compiler takes to be new here: what depends on it is not formed before a
// loop and kept through it.
__device__ __forceinline__ int here(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// 16 bytes per lane, from `each` + `all` past the beginning of `rows`, to LDS from `to` on in the
// order of the lanes. (Not within a template: the host compiler would reject the size there.)
__device__ __forceinline__ void to_lds(int8_t* to, __amdgpu_buffer_rsrc_t rows, int each, int all) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rows, (__attribute__((address_space(3))) void*)to, 16, each, all, 0, 0);
}

// Waits until all but this wave's last kLeft loads to LDS have arrived and its reads are done, and then
// for the other waves: what they loaded so far is there for all, and what they read may be written over.
template <int kLeft>
__device__ __forceinline__ void wait_fills() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((kLeft & 15) | 7 << 4 | (kLeft >> 4) << 14);  // vmcnt(kLeft), lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// ---- few rows: the weights are read once, straight into registers ----

// A workgroup's waves share 16 kCols columns and split the sum: each takes every
// fourth block of 128 bytes of the weight rows and of x (out of the cache), and the
// four partial sums meet in LDS. Nothing is shared before the end, so no wave waits for
// another. Memory bounds it: 4 rows x 2048 by 151936 take 49-51 us, 6.2 TB/s of weights,
// 1 x 4096 by 32000 27 us (23 where the weights stay in the memory-side cache from one call to
// the next). Blocks of 256 bytes take 50 and 27, without the next block on its way 59 and 29,
// with loads past the cache 57 and 27.
constexpr int kWaves = 4;
constexpr int kSteps = 2;  // matrix instructions of 64 bytes each per block
constexpr int kBlock = 64 * kSteps;

template <class O, int kRows, int kCols>
__global__ void __launch_bounds__(kWaves * 64) few_rows_kernel(Int8Args a, int64_t first) {
    __shared__ int part[kWaves][16 * kRows][16 * kCols + 4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int at = lane & 15, group = lane >> 4;
    const int dim = static_cast<int>(a.dim);
    const int64_t tiles = (a.n_cols + 16 * kCols - 1) / (16 * kCols);
    const int64_t task = first + blockIdx.x;
    const int64_t m0 = task / tiles * (16 * kRows), n0 = task % tiles * (16 * kCols);
    const int8_t* x[kRows];
    const int8_t* w[kCols];
#pragma unroll
    for (int i = 0; i < kRows; ++i) x[i] = a.x + min(m0 + 16 * i + at, a.n_rows - 1) * a.x_stride;
#pragma unroll
    for (int j = 0; j < kCols; ++j) w[j] = a.w + min(n0 + 16 * j + at, a.n_cols - 1) * a.w_stride;
    i32x4 sum[kRows][kCols] = {};
    i32x4 wv[2][kSteps][kCols], xv[2][kSteps][kRows];
    const auto load = [&](int b, int k) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int j = 0; j < kCols; ++j) memcpy(&wv[b][s][j], w[j] + k + s * 64 + group * 16, 16);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int i = 0; i < kRows; ++i) memcpy(&xv[b][s][i], x[i] + k + s * 64 + group * 16, 16);
    };
    const auto use = [&](int b) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int i = 0; i < kRows; ++i)
#pragma unroll
                for (int j = 0; j < kCols; ++j) sum[i][j] = multiply(wv[b][s][j], xv[b][s][i], sum[i][j]);
    };
    // whole blocks, the next one on its way while one is multiplied
    int k = wave * kBlock;
    if (k + kBlock <= dim) {
        load(0, k);
        for (;;) {
            k += kWaves * kBlock;
            if (k + kBlock > dim) {
                use(0);
                break;
            }
            load(1, k);
            use(0);
            k += kWaves * kBlock;
            if (k + kBlock > dim) {
                use(1);
                break;
            }
            load(0, k);
            use(1);
        }
    }
    for (; k < dim; k += kWaves * kBlock) {  // the wave that holds the last, shorter block
        for (int s = 0; s < kSteps && k + s * 64 < dim; ++s) {
            i32x4 xv[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) xv[i] = load16(x[i], k + s * 64 + group * 16, dim);
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                const i32x4 wv = load16(w[j], k + s * 64 + group * 16, dim);
#pragma unroll
                for (int i = 0; i < kRows; ++i) sum[i][j] = multiply(wv, xv[i], sum[i][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int j = 0; j < kCols; ++j) *reinterpret_cast<i32x4*>(&part[wave][16 * i + at][16 * j + 4 * group]) = sum[i][j];
    __syncthreads();
    constexpr int kOuts = 16 * kRows * 16 * kCols;
#pragma unroll
    for (int o = threadIdx.x; o < kOuts; o += kWaves * 64) {
        const int r = o / (16 * kCols), c = o % (16 * kCols);
        const int64_t m = m0 + r, n = n0 + c;
        if (m >= a.n_rows || n >= a.n_cols) continue;
        int whole = 0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) whole += part[i][r][c];
        put(static_cast<O*>(a.out) + m * a.out_stride + n, scaled(whole, split(a.x_scales[m]), split(a.w_scales[n])));
    }
}

// ---- many rows: tiles through LDS ----

constexpr int kDepth = 64;  // bytes of a row per stage: one matrix instruction's

// kBM x kBN results per workgroup, kWM x kWN waves. Four stages of kDepth bytes of each
// row in LDS, filled straight from memory: while one is multiplied out of registers, the
// next is read into them and three more are on their way. A row's four chunks of 16 bytes
// are stored in the order chunk ^ (row / 2 & 3): the lanes that read one chunk of eight
// rows then find them in all banks, and the lanes that fill a row still read it whole.
//
// Results leave by 16 bytes per lane, 64 in a row per instruction. For bfloat16 a lane's
// columns in two matrix tiles have to be neighbours, so tiles 2 i and 2 i + 1 take the
// weight rows of 32 in fours, in turn; w's chunks are ordered so that those lie in all
// banks.
//
// 8192 x 2048 by 151936 to bfloat16: 2.74 ms, 1.86 POP/s; 8192 x 8192 by 8192 439 us, 2.50
// (a library's 8-bit product, unscaled, 2.01). At the latter the matrix units are busy for 65 %
// of the cycles, at the former for 43 %: what is left there is the writing of 2.5 GB (without
// it 2.28 ms). 32 x 2048 by 151936, tiles of 64 x 128: 66 us, 4.7 TB/s of weights. 333 x 1000 by
// 32001 to float32, rows 1024 bytes apart: 29.6 us, fifteen stages straight to LDS and the sixteenth
// by registers, 252 tiles for 256 compute units that each begin with nothing in LDS and end in the
// storing of 43 MB (matrix units busy for a third of the cycles); rows 1000 bytes apart, all by
// registers, 44 us. Two stages of 128 bytes took 533 us at
// 8192^3; one tile per workgroup 2.87 ms at the first size; four waves of 128 x 128 spill; stores past the cache take
// 2.75 ms, but 3.45 instead of 3.14 for float32; workgroups started at different times 2.76, but 512 to 543 at 8192^3.
//
// kRegisters: rows that start anywhere; they pass through registers, as the last, shorter
// stage of any row does. kLines: rows of x and w start at multiples of 16 bytes, and 256 of
// them lie within 2^31. kStream: kLines, and rows of whole groups of four stages: a
// workgroup takes tile after tile, and the fills go on from one to the next, so that a
// tile's first stages arrive while the results of the one before are stored.
enum Feed { kRegisters, kLines, kStream };

struct Tile {
    int64_t m0, n0;
    int last_m, last_n;  // rows of x and w in it, less one
};

template <class O, int kBM, int kBN, int kWM, int kWN, Feed kFeed>
__global__ void __launch_bounds__(kWM* kWN * 64)
    tile_kernel(Int8Args a, int64_t first, int64_t tasks, int64_t tiles_m, int64_t tiles_n) {
    constexpr int kThreads = kWM * kWN * 64;
    constexpr int kTM = kBM / kWM / 16, kTN = kBN / kWN / 16;  // matrix tiles of a wave
    constexpr int kFillRows = kThreads / 4;                    // rows that the workgroup fills at once
    constexpr int kStage = (kBM + kBN) * kDepth;
    // separate arrays, so that the compiler knows a fill of one from a read of another
    __shared__ __attribute__((aligned(1024))) int8_t stage0[kStage];
    __shared__ __attribute__((aligned(1024))) int8_t stage1[kFeed != kRegisters ? kStage : 16];
    __shared__ __attribute__((aligned(1024))) int8_t stage2[kFeed != kRegisters ? kStage : 16];
    __shared__ __attribute__((aligned(1024))) int8_t stage3[kFeed != kRegisters ? kStage : 16];
    const int thread = threadIdx.x;
    const int lane = thread & 63, wave = __builtin_amdgcn_readfirstlane(thread >> 6);
    const int dim = static_cast<int>(a.dim);

    // Consecutive workgroups go to the eight dies in turn: each die gets one run of the
    // tasks, ordered so that the tiles it holds at a time share rows and columns.
    const int64_t die = blockIdx.x % 8, turn = blockIdx.x / 8;
    const int64_t each = tasks / 8, more = tasks % 8;
    const int64_t end = first + (die + 1) * each + min(die + 1, more);
    const int64_t each_block = gridDim.x / 8 + (die < gridDim.x % 8);  // the die's workgroups
    int64_t task = first + die * each + min(die, more) + turn;
    const auto tile_of = [&](int64_t task) __attribute__((always_inline)) {
        constexpr int64_t kGroup = 8;
        const int64_t group = task / (kGroup * tiles_n), in_group = task % (kGroup * tiles_n);
        const int64_t group_m = min(kGroup, tiles_m - group * kGroup);
        Tile t;
        t.m0 = int64_t{uniform(group * kGroup + in_group % group_m)} * kBM;
        t.n0 = int64_t{uniform(in_group / group_m)} * kBN;
        t.last_m = uniform(min(a.n_rows - t.m0, int64_t{kBM})) - 1;
        t.last_n = uniform(min(a.n_cols - t.n0, int64_t{kBN})) - 1;
        return t;
    };
    if (task >= end) return;  // more workgroups than tasks

    // The chunks' order in row r of w, and which row of 16 (32) is the r-th of matrix tile j
    constexpr int kRun = 16 / sizeof(O);
    const auto w_order = [](int r) { return kRun == 4 ? r >> 1 & 3 : (r >> 1 & 1) | (r >> 2 & 2); };
    const auto w_row = [](int j, int r) {
        return kRun == 4 ? 16 * j + r : 32 * (j >> 1) + 4 * (j & 1) + 8 * (r >> 2) + (r & 3);
    };
    // What this thread fills: chunk `slot` of rows fill_row + i kFillRows, from chunk x_chunk / 16 in memory.
    // Rows past the last one are the last one again; their results are not stored.
    const int fill_row = thread >> 2, slot = thread & 3;
    const int x_chunk = (slot ^ (fill_row >> 1 & 3)) * 16, w_chunk = (slot ^ w_order(fill_row)) * 16;
    constexpr int kFillM = kBM / kFillRows, kFillN = kBN / kFillRows;
    static_assert(kFillM * kFillRows == kBM && kFillN * kFillRows == kBN && kFillRows % 16 == 0, "");
    const int8_t *x0, *w0;  // the tile that is filled
    int x_last, w_last, x_bytes, w_bytes;
    const auto fill_next = [&](const Tile& tile, bool some) __attribute__((always_inline)) {
        x0 = uniform(a.x + tile.m0 * a.x_stride);
        w0 = uniform(a.w + tile.n0 * a.w_stride);
        x_last = tile.last_m;
        w_last = tile.last_n;
        x_bytes = uniform(some ? tile.last_m * static_cast<int>(a.x_stride) + dim : 0);  // none: nothing is read
        w_bytes = uniform(some ? tile.last_n * static_cast<int>(a.w_stride) + dim : 0);
    };
    // of this thread's rows; formed anew each time, there is no room to keep them
    const auto x_from = [&](int row, int i) __attribute__((always_inline)) {
        return min(row + i * kFillRows, x_last) * static_cast<int>(a.x_stride) + x_chunk;
    };
    const auto w_from = [&](int row, int i) __attribute__((always_inline)) {
        return min(row + i * kFillRows, w_last) * static_cast<int>(a.w_stride) + w_chunk;
    };
    const int whole = kFeed != kRegisters ? dim / kDepth : 0;
    // a stage past the last one reads nothing
    const auto fill = [&](int8_t* stage, int any_t) __attribute__((always_inline)) {
        const int t = uniform(any_t), row = here(fill_row);
        const __amdgpu_buffer_rsrc_t x_rows = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<int8_t*>(x0), 0, t < whole ? x_bytes : 0, 0x00027000);
        const __amdgpu_buffer_rsrc_t w_rows = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<int8_t*>(w0), 0, t < whole ? w_bytes : 0, 0x00027000);
#pragma unroll
        for (int i = 0; i < kFillM; ++i)
            to_lds(stage + (i * kFillRows + wave * 16) * kDepth, x_rows, x_from(row, i), t * kDepth);
#pragma unroll
        for (int i = 0; i < kFillN; ++i)
            to_lds(stage + (kBM + i * kFillRows + wave * 16) * kDepth, w_rows, w_from(row, i), t * kDepth);
    };
    const auto fill_by_registers = [&](int8_t* stage, const Tile& tile, int t) {
        int8_t* to = stage + fill_row * kDepth + slot * 16;
#pragma unroll 4
        for (int i = 0; i < kFillM; ++i)
            *reinterpret_cast<i32x4*>(to + i * kFillRows * kDepth) =
                load16(a.x + (tile.m0 + min(fill_row + i * kFillRows, tile.last_m)) * a.x_stride, t * kDepth + x_chunk, dim);
#pragma unroll 4
        for (int i = 0; i < kFillN; ++i)
            *reinterpret_cast<i32x4*>(to + (kBM + i * kFillRows) * kDepth) =
                load16(a.w + (tile.n0 + min(fill_row + i * kFillRows, tile.last_n)) * a.w_stride, t * kDepth + w_chunk, dim);
    };

    // what this lane reads: chunk lane / 16 of rows (lane & 15) + 16 i of x, w_row(j, lane & 15) of w
    const int wave_m = wave / kWN * (kBM / kWM), wave_n = wave % kWN * (kBN / kWN);
    const int x_read = (lane & 15) * kDepth + (((lane >> 4) ^ (lane >> 1 & 3)) << 4);
    const int w_read = w_row(0, lane & 15) * kDepth + (((lane >> 4) ^ w_order(w_row(0, lane & 15))) << 4);
    struct Held {
        i32x4 x[kTM], w[kTN];
    };
    const auto take = [&](Held& h, const int8_t* stage) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kTM; ++i)
            h.x[i] = *reinterpret_cast<const i32x4*>(stage + (wave_m + 16 * i) * kDepth + x_read);
#pragma unroll
        for (int j = 0; j < kTN; ++j)
            h.w[j] = *reinterpret_cast<const i32x4*>(stage + (kBM + wave_n + w_row(j, 0)) * kDepth + w_read);
    };
    i32x4 sum[kTM][kTN];
    const auto use = [&](const Held& h) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kTM; ++i)
#pragma unroll
            for (int j = 0; j < kTN; ++j) sum[i][j] = multiply(h.w[j], h.x[i], sum[i][j]);
    };
    // One stage, in registers already. All waves hold it and, once no more than kLeft of their
    // fills are under way, have the next one filled: it is filled anew with stage t and the
    // next one read while it is multiplied. The scheduling groups spread the reads among the
    // matrix instructions; left to itself the compiler reads everything first and waits for it.
    constexpr int kReads = kTM + kTN, kFills = kFillM + kFillN, kUses = kTM * kTN / kReads;
    const auto step = [&](Held& now, Held& next, int8_t* stage, const int8_t* next_stage, int t, auto left)
                          __attribute__((always_inline)) {
        wait_fills<left.value>();
        fill(stage, t);
        take(next, next_stage);
        use(now);
#pragma unroll
        for (int i = 0; i < kReads; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            if (i < kFills) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, kUses, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr std::integral_constant<int, 2 * kFills> two_stages{};
    constexpr std::integral_constant<int, 63> any{};

    // The results of a tile. Its scales are waited for, and with them every fill so far.
    const auto finish = [&](const Tile& tile) __attribute__((always_inline)) {
        const int lane = here(thread) & 63;
        O* out = static_cast<O*>(a.out);
        constexpr int kTiles = kRun / 4, kRuns = kTN / kTiles;  // matrix tiles per run of columns, runs of a lane
        static_assert(kTN % kTiles == 0, "");
        const int64_t n_at = tile.n0 + wave_n + (lane >> 4) * kRun;
        float xs[kTM], ws[kRuns][kRun];
#pragma unroll
        for (int i = 0; i < kTM; ++i) xs[i] = a.x_scales[tile.m0 + min(wave_m + 16 * i + (lane & 15), tile.last_m)];
#pragma unroll
        for (int r = 0; r < kRuns; ++r)
#pragma unroll
            for (int c = 0; c < kRun; ++c) ws[r][c] = a.w_scales[min(n_at + r * 4 * kRun + c, a.n_cols - 1)];
        __builtin_amdgcn_s_waitcnt(15 << 8 | 7 << 4);  // vmcnt(0)
        bool fine = true;
#pragma unroll
        for (int i = 0; i < kTM; ++i) fine = fine && ordinary(xs[i]);
#pragma unroll
        for (int r = 0; r < kRuns; ++r)
#pragma unroll
            for (int c = 0; c < kRun; ++c) fine = fine && ordinary(ws[r][c]);
        const auto store = [&](auto value) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < kTM; ++i) {
                const int row = wave_m + 16 * i + (lane & 15);
                if (row > tile.last_m) break;
                O* to = out + (tile.m0 + row) * a.out_stride;
#pragma unroll
                for (int r = 0; r < kRuns; ++r) {
                    const int64_t n = n_at + r * 4 * kRun;
                    O v[kRun];
#pragma unroll
                    for (int c = 0; c < kRun; ++c)
                        put(&v[c], value(sum[i][r * kTiles + c / 4][c & 3], xs[i], ws[r][c]));
                    if (n + kRun <= a.n_cols) {
                        memcpy(to + n, v, sizeof(v));
                    } else {
#pragma unroll
                        for (int c = 0; c < kRun; ++c)
                            if (n + c < a.n_cols) to[n + c] = v[c];
                    }
                }
            }
        };
        // the same roundings either way
        if (!__ballot(!fine)) store([](int s, float x, float w) { return static_cast<float>(s) * (x * w); });
        else store([](int s, float x, float w) { return scaled(s, split(x), split(w)); });
    };
    const auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kTM; ++i)
#pragma unroll
            for (int j = 0; j < kTN; ++j) sum[i][j] = i32x4{0, 0, 0, 0};
    };

    Tile tile = tile_of(task);
    Held even, odd;
    if (kFeed != kRegisters) {
        fill_next(tile, true);
        fill(stage0, 0);
        fill(stage1, 1);
        fill(stage2, 2);
        fill(stage3, 3);
    }
    if constexpr (kFeed == kStream) {
        wait_fills<0>();
        for (;;) {
            clear();
            take(even, stage0);  // the last step before read it already; kept, it would not leave room for the results
            task += each_block;
            Tile next = tile;
            int t = 4;
            const auto four = [&](auto wait) __attribute__((always_inline)) {
                if (t == whole) {  // the last group of this tile: its stages are filled for the next
                    if (task < end) next = tile_of(task);
                    fill_next(next, task < end);
                    t = 0;
                }
                step(even, odd, stage0, stage1, t, wait);
                step(odd, even, stage1, stage2, t + 1, wait);
                step(even, odd, stage2, stage3, t + 2, wait);
                step(odd, even, stage3, stage0, t + 3, two_stages);
                t += 4;
            };
            // stages 1 to 3 of the tile were waited for before the results of the last one were stored
            four(any);
            for (int i = 4; i < whole; i += 4) four(two_stages);
            finish(tile);
            if (task >= end) break;
            tile = next;
        }
        return;
    }
    clear();
    if (whole > 0) {
        wait_fills<3 * kFills>();
        take(even, stage0);
        int t = 0;
        for (; t + 4 <= whole; t += 4) {
            step(even, odd, stage0, stage1, t + 4, two_stages);
            step(odd, even, stage1, stage2, t + 5, two_stages);
            step(even, odd, stage2, stage3, t + 6, two_stages);
            step(odd, even, stage3, stage0, t + 7, two_stages);
        }
        if (t < whole) step(even, odd, stage0, stage1, t + 4, two_stages);
        if (t + 1 < whole) step(odd, even, stage1, stage2, t + 5, two_stages);
        if (t + 2 < whole) step(even, odd, stage2, stage3, t + 6, two_stages);
        wait_fills<0>();
    }
    for (int t = whole; t * kDepth < dim; ++t) {
        __syncthreads();
        fill_by_registers(stage0, tile, t);
        __syncthreads();
        take(even, stage0);
        use(even);
    }
    finish(tile);
}

template <class O, int kRows, int kCols>
hipError_t launch_few(const Int8Args& a, hipStream_t stream) {
    const int64_t tiles = (a.n_rows + 16 * kRows - 1) / (16 * kRows) * ((a.n_cols + 16 * kCols - 1) / (16 * kCols));
    const int64_t most = max_blocks_per_launch(kWaves * 64);
    for (int64_t first = 0; first < tiles; first += most)
        few_rows_kernel<O, kRows, kCols>
            <<<dim3(static_cast<unsigned int>(std::min(most, tiles - first))), dim3(kWaves * 64), 0, stream>>>(a, first);
    return hipGetLastError();
}

constexpr int64_t kUnits = 256;  // compute units

template <class O, int kBM, int kBN, int kWM, int kWN, bool kMayStream>
hipError_t launch_tiles(const Int8Args& a, hipStream_t stream) {
    const int64_t tiles_m = (a.n_rows + kBM - 1) / kBM, tiles_n = (a.n_cols + kBN - 1) / kBN, tiles = tiles_m * tiles_n;
    constexpr int kThreads = kWM * kWN * 64;
    const int64_t most = max_blocks_per_launch(kThreads);
    const bool lines = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.w)) & 15) == 0 &&
                       ((a.x_stride | a.w_stride) & 15) == 0 && std::max(a.x_stride, a.w_stride) < (int64_t{1} << 31) / 256;
    if constexpr (kMayStream) {
        if (lines && a.dim % (4 * kDepth) == 0 && tiles > kUnits) {
            tile_kernel<O, kBM, kBN, kWM, kWN, kStream><<<dim3(kUnits), dim3(kThreads), 0, stream>>>(a, 0, tiles, tiles_m, tiles_n);
            return hipGetLastError();
        }
    }
    for (int64_t first = 0; first < tiles; first += most) {
        const int64_t tasks = std::min(most, tiles - first);
        const dim3 grid(static_cast<unsigned int>(tasks));
        if (lines) tile_kernel<O, kBM, kBN, kWM, kWN, kLines><<<grid, dim3(kThreads), 0, stream>>>(a, first, tasks, tiles_m, tiles_n);
        else tile_kernel<O, kBM, kBN, kWM, kWN, kRegisters><<<grid, dim3(kThreads), 0, stream>>>(a, first, tasks, tiles_m, tiles_n);
    }
    return hipGetLastError();
}

// Up to 16 rows the weights' way from memory decides: straight into registers; wider columns
// per wave where x is read often (16 x 4096 by 32000: 23.7 us, 28.4 with two; 4 x 2048 by 151936:
// 54.6, 51.5 with two). So it does for 64 rows and few columns, where tiles would leave much of the
// chip idle (64 x 1024 by 1024 4.8 us, tiles of 64 x 64 5.6; 17 x 2048 by 8192 6.2, 7.4; 64 x 11008
// by 4096 22, 29). At the rule's corner, many rows, columns and bytes at once, the tiles
// win (64 x 4096 by 4096 11.3 us, 10.8; 64 x 2048 by 8192 10.4, 7.4; 48 x 8192 by 8192 33, 21), and
// beyond it by far (64 x 4096 by 32000 59, 22).
//
// Among the tiles, the one whose workgroups take the least time: the steps of the compute unit
// that gets the most of them, at what a step of each tile was measured to take there (1024 x 2048
// by 32000 to bfloat16, all units full). The results' width and the number of stages do not enter, since all
// tiles write the same results and their steps grow alike with the stages. So 512 x 4096 by 4096 takes tiles of
// 64 x 128 (16.9 us; 128 x 128 20.1, 256 x 256 45), 32 x 2048 by 151936 as well (65.6; 64 x 64 72.5), 333 x 1000 by
// 32001 to float32 256 x 256 (29.6 us; 128 x 128 30.6, 64 x 128 35.4), 2000 x 1000 by 5000 too (24.4; 26.4, 27.9).
template <class O>
hipError_t launch(const Int8Args& a, hipStream_t stream) {
    if (a.n_rows <= 16)
        return a.n_rows > 8 && a.n_cols >= 16384 ? launch_few<O, 1, 4>(a, stream) : launch_few<O, 1, 2>(a, stream);
    if (a.n_rows <= 64 && a.n_cols <= 8192) return launch_few<O, 2, 2>(a, stream);
    const auto cost = [&](int64_t bm, int64_t bn, int64_t step_ns) {
        const int64_t tiles = (a.n_rows + bm - 1) / bm * ((a.n_cols + bn - 1) / bn);
        return (tiles + kUnits - 1) / kUnits * step_ns;
    };
    const int64_t c64 = cost(64, 64, 170), c64x128 = cost(64, 128, 260), c128 = cost(128, 128, 380),
                  c256 = cost(256, 256, 980);
    const int64_t least = std::min(std::min(c64, c64x128), std::min(c128, c256));
    if (c256 == least) return launch_tiles<O, 256, 256, 2, 4, true>(a, stream);
    if (c128 == least) return launch_tiles<O, 128, 128, 2, 2, false>(a, stream);
    if (c64x128 == least) return launch_tiles<O, 64, 128, 2, 2, false>(a, stream);
    return launch_tiles<O, 64, 64, 2, 2, false>(a, stream);
}

}  // namespace

hipError_t launch_matmul_int8(const Int8Args& a, hipStream_t stream) {
    return a.out_type == kF32 ? launch<float>(a, stream) : launch<__bf16>(a, stream);
}

}  // namespace kldk
