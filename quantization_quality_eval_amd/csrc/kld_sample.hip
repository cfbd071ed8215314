// Drawing one token from each logit row, with temperature, top-k, top-p and min-p.
//
// Logits that are not finite are excluded. With M the largest of the others and
// w_v = exp((z_v - M) / T), tokens are ordered by logit, equal ones by lowest id.
// Kept are the first k of the order; of those the shortest run from its beginning
// that holds a share p of their sum of w; of those the ones with w >= max(m, 2^-64).
// The token is the first kept one, by ids, at which the running sum of the kept w
// passes u times the whole.
//
// With c = 4 log2 e / T a weight is 2^(c z / 4). It is taken as 2^((f + r) / 4), f = rint(c z) and
// |r| <= 1/2: 2^(r / 4) is the token's mantissa, rounded to a whole multiple of 2^-45, and f the
// bin it belongs to, a quarter of a binary unit wide (kld_bins.h). Bins are counted down from
// that of the largest logit of a row or slice, so that a slice's bins are the row's, some whole
// number down. Sums of mantissas in a bin are sums of integers: they depend on no
// order, and their relative error is below 2^-45 whatever the row. Sums over bins are formed in
// float64 in a fixed order.
//
// Launches, over as many rows as the workspace holds (a slice is 8192 tokens):
//   scan  a workgroup per slice: its largest logit, and the count and the sum of mantissas of
//         each of its upper 272 bins (68 binary units; what lies below 2^-64 of the largest
//         weight is dropped), by LDS atomics;
//   plan  a workgroup per row: adds the slices' bins up, finds the bin in which the order is
//         cut first, the logits that belong to that bin, by bisection, and the slices that hold any;
//   list  a workgroup per slice: the tokens between those logits, compared as floats, to a
//         list in memory (at most 16384 a row; a fuller bin is read from the row again);
//   draw  a workgroup per row: cuts the bins by top-k, then top-p, within a bin by a histogram
//         of 256 parts and then by ranking the last 64 tokens; sums what each slice keeps, finds
//         the slice that holds the draw, reads it and draws from it.
// Rows that no limit cuts need the scan and the draw alone: there a slice's sum holds what lies between 2^-64 of
// the largest weight and the last bin's 2^-68 as well, 2^-42 of a row's sum at most, though it is never drawn.
//
// 1024 x 151936 bfloat16 (311 MB), top-p: scan 129 us, plan 14, list 43, draw 71, and 238 us in all
// among other calls; the memory could give the row once in 46 us. The scan is bound by float64
// arithmetic, which runs at half rate here: for each 64 tokens of a SIMD 12 operations of it, of
// which 7 multiply-adds raise a token, beside 5 others and an LDS atomic (2.4 TB/s; bank
// conflicts take a fifth of the LDS' cycles). Float32 would be faster, but its sums err
// by more than the weight of a token near the border of a long row. The list is bound by its second reading of the
// rows (7 TB/s; 218 of the 311 MB come from memory). The draw is bound by latency: two
// workgroups to a CU, each a chain of reductions and barriers. Without limits the 1024 rows take 158 us (scan 127,
// draw 31), at temperature 0 56 (scan 47, memory's rate, draw 8). 64 rows take 27 us without limits
// and 40 to 60 with them, one row of 32000 tokens 35 us: the four launches' own latencies
// (5, 5, 5 and 20 us).
//
// Where a bin that is cut holds more than kList tokens, or top-p cuts one behind a top-k prefix longer than that,
// the draw reads it from the row, slice after slice, in a workgroup by itself: 64 x 151936 with top-p take 200 us at
// a spread of 0.3, 210 with a top-k of 50000 at a spread of 1, and 1.74 ms where all logits are equal, since every
// token then adds to one LDS word; a row of 4194304 equal ones 47 ms.
//
// Measured on the way, 1024 x 151936: bins of a whole unit, whose tokens the draw looked for in
// the rows by itself, 590 us; of a quarter, with two draws to a CU, 340; a list by a workgroup
// per slice 97 to 72 us for 64 rows, in memory rather than in the draw's LDS 320 to 290. A draw of
// 1024 threads was slower.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "kld_answer.h"
#include "kld_bins.h"

namespace kldk {
namespace {

constexpr int kSlice = 8192;        // tokens of a slice
constexpr int kScanThreads = 256;
constexpr int kEach = kSlice / kScanThreads;
constexpr int kCopies = 8;          // of the bins in LDS: lanes that add to one bin wait for each other less
constexpr int kDrawThreads = 512;
constexpr int kDrawEach = kSlice / kDrawThreads;
constexpr int kList = 16384;        // tokens of a row that are listed
constexpr int kSplit = 256;         // parts of a bin, or of a range of logits
constexpr int kFew = 64;            // tokens that a wave ranks
constexpr int kMaxSlices = 512;     // of a row: what the draw knows of each is held in LDS
constexpr double kLeast = 0x1p-64;  // smallest share of the likeliest token's weight that is kept
// A pass over the workspace takes as many rows as fit in this many slices, and in this many bytes or as many as the
// logits have in bfloat16 (the same for float32, so that one workspace serves either type), at least one. So
// 32768 x 60 ask for 232 MB and 8192 x 32000 for 0.5 GB, instead of the 4.5 and 1.2 GB that lists of kList tokens for
// every row and no bound in bytes took, at 1.77 and 0.78 ms instead of 1.81 and 0.94.
constexpr int64_t kPassSlices = 32768, kPassBytes = int64_t{1} << 28;
// Sums that equal each other but for the order of their additions count as equal.
constexpr double kSame = 0x1p-44;

// What the scan leaves of a slice, and the plan for its listing.
struct Info {
    double mass;        // where there are no limits: its sum of weights, over that of its first bin
    unsigned int best;  // order of its largest logit, 0 if none is finite
    int listed;         // whether any token of it belongs to the bins that are listed
};
struct Token {
    unsigned int order;
    unsigned int id_bin;  // id above bit 9, bin
};
static_assert(kBins < 512 && kSampleMaxVocab <= int64_t{kMaxSlices} * kSlice && kSampleMaxVocab <= int64_t{1} << 23, "");
// A row's bins, and the ones whose tokens are listed (none: last < 0).
constexpr int kLaneBins = (kBins + 63) / 64;
struct Plan {
    double mass[kLaneBins * 64];
    int count[kLaneBins * 64];
    int first, last;
    float from, to;      // their logits, [from, to)
    unsigned int best;   // order of the row's largest logit
    int listed;          // tokens so far
};
struct Layout {
    Info* info;              // [rows][slices]
    Plan* plan;              // [rows]
    Token* list;             // [rows][list_of(vocab)]
    double* masses;          // [rows][slices][kBins]: a bin's sum of mantissas, in units
    uint16_t* counts;        // and its count
};
__host__ __device__ inline int64_t slices_of(int64_t vocab) { return (vocab + kSlice - 1) / kSlice; }
constexpr int64_t kSliceBytes = sizeof(Info) + kBins * (sizeof(double) + sizeof(uint16_t));
__host__ __device__ inline int64_t list_of(int64_t vocab) { return vocab < kList ? vocab : kList; }
inline int64_t row_bytes(int64_t vocab) {
    return slices_of(vocab) * kSliceBytes + static_cast<int64_t>(sizeof(Plan)) + list_of(vocab) * static_cast<int64_t>(sizeof(Token));
}
// How many rows the workspace holds: more for more rows, so that one that serves a batch serves a smaller one.
inline int64_t held_rows(int64_t vocab, int64_t n_rows) {
    const int64_t bytes = std::max(kPassBytes, n_rows * vocab * 2);
    return std::max<int64_t>(1, std::min({n_rows, kPassSlices / slices_of(vocab), bytes / row_bytes(vocab)}));
}

template <class E>
struct Elem;
template <>
struct Elem<uint16_t> {
    static constexpr int kPer = 8;  // per 16 bytes
    static __device__ __forceinline__ float get(const unsigned int* q, int e) {
        return __uint_as_float(e & 1 ? q[e >> 1] & 0xffff0000u : q[e >> 1] << 16);
    }
    static __device__ __forceinline__ float widen(uint16_t b) {
        return __uint_as_float(static_cast<unsigned int>(b) << 16);
    }
    static __device__ __forceinline__ uint16_t none() { return 0xff80; }  // -inf
};
template <>
struct Elem<float> {
    static constexpr int kPer = 4;
    static __device__ __forceinline__ float get(const unsigned int* q, int e) { return __uint_as_float(q[e]); }
    static __device__ __forceinline__ float widen(float x) { return x; }
    static __device__ __forceinline__ float none() { return -INFINITY; }
};

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// A slice's tokens in the registers of kScanThreads threads, in 16 bytes each, any alignment; of a
// row's last, shorter slice one by one, places behind its end from its last token so that the loads
// need no branches (32000 tokens: the list 4.4 instead of 7.3 us).
template <class E>
__device__ __forceinline__ int held_id(int slice, int vocab, int i) {
    constexpr int kPer = Elem<E>::kPer;
    const int thread = threadIdx.x, v0 = slice * kSlice;
    return v0 + kSlice <= vocab ? v0 + (i / kPer * kScanThreads + thread) * kPer + i % kPer : v0 + i * kScanThreads + thread;
}
template <class E>
__device__ __forceinline__ void hold_slice(const E* row, int slice, int vocab, float (&z)[kEach]) {
    constexpr int kPer = Elem<E>::kPer;
    if ((slice + 1) * kSlice <= vocab) {
#pragma unroll
        for (int u = 0; u < kEach / kPer; ++u) {
            u32x4 q;
            memcpy(&q, row + held_id<E>(slice, vocab, u * kPer), 16);
            const unsigned int w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < kPer; ++e) z[u * kPer + e] = Elem<E>::get(w, e);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int v = held_id<E>(slice, vocab, i);
            const float x = Elem<E>::widen(row[static_cast<unsigned int>(min(v, vocab - 1))]);
            z[i] = v < vocab ? x : -INFINITY;
        }
    }
}

// Order of logits: that of finite floats, -0 and 0 alike; above 0.
__device__ __forceinline__ unsigned int order_of(float z) {
    const unsigned int u = __float_as_uint(z + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned int o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ bool allowed(float z) { return z < INFINITY && z > -INFINITY; }

// ---- settings ----

enum Mode { kGreedy, kNoLimit, kLimited };

struct Settings {
    Heat heat;
    int64_t k;     // vocab: no limit
    double p;      // 1: no limit
    double least;  // the least share's logarithm, in bins
    Mode mode;
};
__device__ __forceinline__ double setting(const Setting& s, int64_t row) {
    return s.each ? static_cast<double>(s.each[row]) : s.all;
}
__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int64_t row) {
    Settings s;
    const double heat = setting(a.temperature, row), p = setting(a.top_p, row), m = setting(a.min_p, row);
    const int k = a.top_ks ? a.top_ks[row] : a.top_k;
    s.heat = heat_of(heat);
    s.k = k > 0 && k < a.vocab ? k : a.vocab;
    s.p = p < 1.0 ? p : 1.0;
    // less a rounding: a weight that float64 rounds to 1 is 1
    s.least = kPerUnit * (m > kLeast ? log2(fmin(m, 1.0)) - 0x1p-53 : -64.0);
    s.mode = !(heat > 0.0) ? kGreedy : s.k == a.vocab && s.p == 1.0 && !(m > kLeast) ? kNoLimit : kLimited;
    return s;
}

// ---- weights ----

// The scan holds the polynomial's coefficients in scalar registers: left to itself the compiler copies each into
// vector registers before its step.
__device__ __forceinline__ void hold(Raise& raise) {
#pragma unroll
    for (int i = 0; i <= Raise::kDegree; ++i) asm volatile("" : "+s"(raise.c[i]));
}
// What the units of a bin's mantissas weigh.
__device__ __forceinline__ double unit_of(int bin) { return ldexp(scale_of(-bin), -kUnit); }
// The weight of a logit that has a bin.
__device__ __forceinline__ double weight(const Raise& raise, Spot at) { return mantissa_of(raise(at.r)) * scale_of(-at.bin); }

// ---- the scan ----

// Left to itself with its registers (89, 92 for float32): kept to 64 it took 139 us instead of 136 at 1024 x 151936
// bfloat16, 331 instead of 229 at 8192 x 32000.
template <class E>
__global__ void __launch_bounds__(kScanThreads) scan_kernel(SampleArgs a, int64_t first_row, Layout out, int slices) {
    __shared__ unsigned long long bins[(kBins + 1) * kCopies];
    __shared__ float part_max[kScanThreads / 64];
    __shared__ double part_sum[kScanThreads / 64];
    const int64_t task = blockIdx.x;
    const int64_t row = first_row + task / slices;
    const int slice = static_cast<int>(task % slices), thread = threadIdx.x;
    const E* in = static_cast<const E*>(a.logits) + row * a.row_stride;
    float z[kEach];
    hold_slice(in, slice, static_cast<int>(a.vocab), z);
    const Settings s = settings_of(a, row);
    if (s.mode != kGreedy)
        for (int i = thread; i < kBins * kCopies; i += kScanThreads) bins[i] = 0;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kEach; ++i) m = __builtin_elementwise_maximum(m, z[i]);  // a NaN where any is
    if (!(m < INFINITY)) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            z[i] = z[i] < INFINITY ? z[i] : -INFINITY;
            m = fmaxf(m, z[i]);
        }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if ((thread & 63) == 0) part_max[thread >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kScanThreads / 64; ++i) m = fmaxf(m, part_max[i]);
    Info* info = out.info + task;
    const bool none = !(m > -INFINITY);
    if (none || s.mode == kGreedy) {
        if (thread == 0) *info = Info{0.0, none ? 0 : order_of(m), 0};
        return;
    }
    Raise raise;
    hold(raise);
    const Frame frame = frame_of(m, s.heat);
    // Logits that have no bin go to one behind the others.
    const int copy = thread & (kCopies - 1);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const Spot at = spot_of(z[i], frame);
        atomicAdd(&bins[min(static_cast<unsigned int>(at.bin), static_cast<unsigned int>(kBins)) * kCopies + copy],
                  __builtin_bit_cast(unsigned long long, raise(at.r)));
    }
    __syncthreads();
    double sum = 0.0;
    for (int i = thread; i < kBins; i += kScanThreads) {
        uint64_t units = 0;
        int count = 0;
#pragma unroll
        for (int c = 0; c < kCopies; ++c) {
            const uint64_t word = bins[i * kCopies + c];
            units += units_in(word);
            count += count_in(word);
        }
        const double mass = static_cast<double>(units);
        if (s.mode == kLimited) {
            out.masses[task * kBins + i] = mass;
            out.counts[task * kBins + i] = static_cast<uint16_t>(count);
        } else {
            sum += mass * unit_of(i);
        }
    }
    if (s.mode == kNoLimit) {
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
        if ((thread & 63) == 0) part_sum[thread >> 6] = sum;
        __syncthreads();
        for (int i = 1; i < kScanThreads / 64; ++i) sum += part_sum[i];
    }
    if (thread == 0) *info = Info{sum, order_of(m), 0};
}
static_assert(kSlice / kCopies <= kWordTokens && kScanThreads % kCopies == 0 && kSlice < 1 << 16, "");

// ---- the draw ----

constexpr int kDrawWaves = kDrawThreads / 64;
static_assert(kDrawThreads >= kBins, "a thread adds up a bin of the slices");
// The end of the kept run within a bin: tokens above `order` are kept and the first `ties` of the
// ones that equal it (by ids); `mass` is what they weigh, over 2^base.
struct Cut {
    unsigned int order;
    int ties;
    double mass;
};

// Of the words in which a cut sums a part, up to a whole row's tokens: 52 and 64 bits.
constexpr int kLowBits = 19, kCountAt = 41;
static_assert(kSampleMaxVocab <= int64_t{1} << 22 && kSampleMaxVocab < int64_t{1} << (64 - kCountAt) && 22 + kLowBits <= kCountAt &&
              kUnit + 1 - kLowBits + 22 <= 53, "");

struct Shared {
    // of the slices
    int shift[kMaxSlices];                                     // the row's bin of its largest logit
    int in_range[kMaxSlices];                                  // whether any token of it is in the range below
    unsigned long long mass[kMaxSlices];                       // kept in the last bin, ties apart
    unsigned int ties[kMaxSlices];
    double kept[kMaxSlices];
    // the row's bins
    double bin_mass[kLaneBins * 64];
    int bin_count[kLaneBins * 64];
    unsigned long long split_high[kSplit], split_low[kSplit];
    unsigned int few[kFew];
    int few_count;
    unsigned int least, most;
    float from, to;      // the range of logits that is looked at, [from, to)
    Cut cut;
    int slice;           // that holds the draw,
    double rest, total;  // what is left of it there, and the sum of all kept
    double part_d[kDrawWaves];
    int part_i[kDrawWaves], part_j[kDrawWaves];
};

// x of another lane (a DPP control), 0 where the control gives none.
template <int kCtrl, int kRows>
__device__ __forceinline__ int moved(int x) {
    return __builtin_amdgcn_update_dpp(0, x, kCtrl, kRows, 0xf, false);
}
template <int kCtrl, int kRows>
__device__ __forceinline__ unsigned int moved(unsigned int x) {
    return static_cast<unsigned int>(moved<kCtrl, kRows>(static_cast<int>(x)));
}
template <int kCtrl, int kRows>
__device__ __forceinline__ double moved(double x) {
    return __hiloint2double(moved<kCtrl, kRows>(__double2hiint(x)), moved<kCtrl, kRows>(__double2loint(x)));
}
// One value of all lanes up to each: within rows of 16 lanes from 1, 2, 4, 8 lanes before, then from the
// last lane of the row and of the half before.
template <class T, class Join>
__device__ __forceinline__ T joined_to(T x, Join join) {
    x = join(x, moved<0x111, 0xf>(x));
    x = join(x, moved<0x112, 0xf>(x));
    x = join(x, moved<0x114, 0xf>(x));
    x = join(x, moved<0x118, 0xf>(x));
    x = join(x, moved<0x142, 0xa>(x));
    return join(x, moved<0x143, 0xc>(x));
}
template <class T>
__device__ __forceinline__ T wave_sum_to(T x) {
    return joined_to(x, [](T a, T b) { return a + b; });
}
__device__ __forceinline__ unsigned int from_lane(unsigned int x, int lane) {
    return static_cast<unsigned int>(__builtin_amdgcn_readlane(static_cast<int>(x), lane));
}
__device__ __forceinline__ int from_lane(int x, int lane) { return __builtin_amdgcn_readlane(x, lane); }
__device__ __forceinline__ uint64_t from_lane(uint64_t x, int lane) {
    return static_cast<uint64_t>(from_lane(static_cast<unsigned int>(x >> 32), lane)) << 32 | from_lane(static_cast<unsigned int>(x), lane);
}
__device__ __forceinline__ double from_lane(double x, int lane) {
    return __hiloint2double(from_lane(__double2hiint(x), lane), from_lane(__double2loint(x), lane));
}
__device__ __forceinline__ unsigned int wave_most(unsigned int x) {
    return from_lane(joined_to(x, [](unsigned int a, unsigned int b) { return a > b ? a : b; }), 63);
}
// Sum over the workgroup's threads up to this one, in a fixed order.
template <class T>
__device__ __forceinline__ T sum_to(T x, T* part) {
    const int wave = threadIdx.x >> 6;
    x = wave_sum_to(x);
    if ((threadIdx.x & 63) == 63) part[wave] = x;
    __syncthreads();
    T before = 0;
    for (int i = 0; i < wave; ++i) before += part[i];
    return before + x;
}

// A place in a sequence of counted and weighed things, and what lies before it.
struct Place {
    int at;
    int count;
    double mass;
};
// Lane l holds kOf things each, those from l kOf on, counted and weighed. The first that holds
// something and, with what lies before it, reaches what is sought, or (a rounding short) the last one
// that holds something; -1 if none does. The same in all lanes.
template <int kOf, class Reached>
__device__ __forceinline__ Place first_reached(const int (&n)[kOf], const double (&w)[kOf], Reached reached) {
    const int lane = threadIdx.x & 63;
    int all_n = 0;
    double all_w = 0.0;
#pragma unroll
    for (int i = 0; i < kOf; ++i) all_n += n[i], all_w += w[i];
    int at_n = wave_sum_to(all_n) - all_n;
    double at_w = wave_sum_to(all_w) - all_w;
    Place first{-1, 0, 0.0}, last{-1, 0, 0.0};
#pragma unroll
    for (int i = 0; i < kOf; ++i) {
        if (n[i] != 0) {
            last = Place{lane * kOf + i, at_n, at_w};
            if (first.at < 0 && reached(at_n + n[i], at_w + w[i])) first = last;
        }
        at_n += n[i];
        at_w += w[i];
    }
    const uint64_t some = __ballot(last.at >= 0), found = __ballot(first.at >= 0);
    if (!some) return Place{-1, 0, 0.0};
    const int from = found ? __builtin_ctzll(found) : 63 - __builtin_clzll(some);
    const Place mine = found ? first : last;
    return Place{from_lane(mine.at, from), from_lane(mine.count, from), from_lane(mine.mass, from)};
}

template <class E>
struct Row {
    const E* in;
    int vocab;
    int slices;
    Settings s;
    Frame frame;  // by the largest logit
    const double* masses;    // of its slices' bins
    const uint16_t* counts;
    const Token* list;     // of its bins list_first to list_last
    int listed;
    Raise raise;
    Shared& sh;

    // This thread's kDrawEach consecutive tokens of a slice.
    static constexpr int kQuads = kDrawEach / Elem<E>::kPer;
    struct Raw {
        u32x4 q[kQuads];
    };
    __device__ __forceinline__ int id_of(int slice, int e) const {
        return slice * kSlice + static_cast<int>(threadIdx.x) * kDrawEach + e;
    }
    __device__ __forceinline__ Raw read(int slice) const {
        Raw raw;
        const int v = id_of(slice, 0);
        if ((slice + 1) * kSlice <= vocab) {
            memcpy(&raw, in + v, sizeof(raw));
        } else {
            E e[kDrawEach];
#pragma unroll
            for (int i = 0; i < kDrawEach; ++i) {
                const E x = in[static_cast<unsigned int>(min(v + i, vocab - 1))];
                e[i] = v + i < vocab ? x : Elem<E>::none();
            }
            memcpy(&raw, e, sizeof(raw));
        }
        return raw;
    }
    static __device__ __forceinline__ float get(const Raw& raw, int e) {
        const u32x4 q = raw.q[e / Elem<E>::kPer];
        const unsigned int w[4] = {q.x, q.y, q.z, q.w};
        return Elem<E>::get(w, e % Elem<E>::kPer);
    }
    __device__ __forceinline__ Spot at(float z) const { return spot_of(z, frame); }
    // Whether a token passes min-p.
    __device__ __forceinline__ bool enough(float z) const {
        return (static_cast<double>(z) - static_cast<double>(frame.most)) * s.heat.per >= s.least;
    }
    // The logits of bins first to last, [from, to), and the slices that hold any. Bins fall as logits rise.
    __device__ __forceinline__ void set_range(int first, int last) const {
        __syncthreads();
        if (threadIdx.x < 2) {
            const int bin = threadIdx.x == 0 ? last : first - 1;
            // the lowest logit whose bin is `bin` or one before it. It is next to where c z reaches the
            // bin's edge, unless c is too small or too large for that to be told.
            unsigned int below = order_of(-INFINITY), above = order_of(INFINITY);
            const auto reaches = [&](unsigned int o) { return bin_of(value_of(o), frame) <= bin; };
            if (bin >= 0) {  // before the first there is none: infinity
                const float near = static_cast<float>((frame.top - kWhole - bin - 0.5) * (1.0 / frame.per));
                if (fabsf(near) < 1e30f && fabsf(near) > 1e-30f) {
                    const unsigned int o = order_of(near);
                    if (reaches(o + 2)) above = o + 2;
                    else below = o + 2;
                    if (above == o + 2 && !reaches(o - 2)) below = o - 2;
                }
#pragma unroll 1
                while (above - below > 1) {
                    const unsigned int middle = below + (above - below) / 2;
                    if (reaches(middle)) above = middle;
                    else below = middle;
                }
            }
            (threadIdx.x == 0 ? sh.from : sh.to) = value_of(above);
        }
        for (int i = threadIdx.x; i < slices; i += kDrawThreads) {
            const int local = last - sh.shift[i];
            sh.in_range[i] = local >= 0 && (first < last || counts[static_cast<int64_t>(i) * kBins + local] != 0);
        }
        __syncthreads();
    }
    __device__ __forceinline__ int next_in_range(int i) const {
        do ++i;
        while (i < slices && !sh.in_range[i]);
        return i;
    }
    // f(order, slice) for the tokens in the range set last, out of the row.
    template <class F>
    __device__ __forceinline__ void each_in_range(F f) const {
        const float from = sh.from, to = sh.to;
#pragma unroll 1
        for (int i = next_in_range(-1); i < slices; i = next_in_range(i)) {
            const Raw raw = read(i);
            unsigned int in = 0;
#pragma unroll
            for (int e = 0; e < kDrawEach; ++e) {
                const float z = get(raw, e);
                in |= static_cast<unsigned int>(z >= from && z < to) << e;
            }
            for (; in; in &= in - 1) f(order_of(Elem<E>::widen(this->in[id_of(i, __builtin_ctz(in))])), i);
        }
    }
    // f(order, slice) for the tokens of a bin, out of the list or, where they are not in it, of the row (their
    // range set last).
    template <class F>
    __device__ __forceinline__ void each_of(int bin, bool in_list, F f) const {
        if (in_list) {
#pragma unroll 1
            for (int i = threadIdx.x; i < listed; i += kDrawThreads) {
                const Token t = list[i];
                if (static_cast<int>(t.id_bin & 511) == bin) f(t.order, static_cast<int>(t.id_bin >> 9) / kSlice);
            }
        } else {
            each_in_range(f);
        }
    }

    // Cuts a bin where its tokens, in order, number `want_count` or weigh `want_mass` (the other one is out
    // of reach). They are divided by their weight, then as long as a part holds more than kFew by their
    // order, and the last few are ranked.
    __device__ __forceinline__ Cut cut(int bin, bool in_list, int want_count, double want_mass) const {
        const auto each = [&](auto f) __attribute__((always_inline)) {
            each_of(bin, in_list, [&](unsigned int o, int) __attribute__((always_inline)) { f(o); });
        };
        const double unit = unit_of(bin);  // sums are in whole units of the bin
        const double want = want_mass * (1.0 - kSame);
        const auto units = [&](unsigned int o) __attribute__((always_inline)) { return units_of(raise(at(value_of(o)).r)); };
        // A part's mantissas are summed in two words, without their last bits and those alone below a count of them.
        const auto count_of = [&](int part) __attribute__((always_inline)) { return static_cast<int>(sh.split_low[part] >> kCountAt); };
        const int thread = threadIdx.x, lane = thread & 63;
        unsigned int lo = 0, hi = ~0u;
        int down = -1;  // -1: by weight
        const auto part_of = [&](unsigned int o) __attribute__((always_inline)) {  // the largest logits first
            if (down >= 0) return kSplit - 1 - static_cast<int>((o - lo) >> down);
            const int part = static_cast<int>((0.5 - at(value_of(o)).r) * kSplit);
            return max(0, min(kSplit - 1, part));
        };
        int above = 0;
        double above_mass = 0.0;
        for (;;) {
            __syncthreads();
            if (thread < kSplit) sh.split_high[thread] = 0, sh.split_low[thread] = 0;
            if (thread == 0) sh.few_count = 0, sh.least = ~0u, sh.most = 0;
            __syncthreads();
            each([&](unsigned int o) __attribute__((always_inline)) {
                if (o < lo || o > hi) return;
                const int part = part_of(o);
                const unsigned long long u = units(o);
                atomicAdd(&sh.split_high[part], u >> kLowBits);
                atomicAdd(&sh.split_low[part], (u & ((1ull << kLowBits) - 1)) + (1ull << kCountAt));
            });
            __syncthreads();
            constexpr int kOf = kSplit / 64;
            int n[kOf];
            double w[kOf];
#pragma unroll
            for (int i = 0; i < kOf; ++i) {
                n[i] = count_of(lane * kOf + i);
                const double low = static_cast<double>(sh.split_low[lane * kOf + i] & ((1ull << kCountAt) - 1));
                w[i] = fma(static_cast<double>(sh.split_high[lane * kOf + i]), 1 << kLowBits, low) * unit;
            }
            const Place found = first_reached(n, w, [&](int count, double mass) {
                return above + count >= want_count || above_mass + mass >= want;
            });
            const int in_part = count_of(max(found.at, 0));
            above += found.count;
            above_mass += found.mass;
            const bool few = in_part <= kFew;
            each([&](unsigned int o) __attribute__((always_inline)) {
                if (o < lo || o > hi || part_of(o) != found.at) return;
                if (few) sh.few[atomicAdd(&sh.few_count, 1)] = o;
                else atomicMin(&sh.least, o), atomicMax(&sh.most, o);
            });
            __syncthreads();
            if (!few && sh.least != sh.most) {
                lo = sh.least;
                hi = sh.most;
                down = 0;
                while ((hi - lo) >> down >= kSplit) ++down;
                continue;
            }
            if (thread < 64) {
                // each lane's token: how many there are above it and what they weigh, how many equal it
                const unsigned int mine = few ? (lane < in_part ? sh.few[lane] : 0) : lane == 0 ? sh.least : 0;
                const uint64_t weighs = mine != 0 ? units(mine) : 0;
                int before = 0, same = few ? 0 : in_part;
                uint64_t before_units = 0;
                if (few)
#pragma unroll 1
                    for (int i = 0; i < in_part; ++i) {
                        const unsigned int o = from_lane(mine, i);
                        const uint64_t u = from_lane(weighs, i);
                        before += o > mine;
                        before_units += o > mine ? u : 0;
                        same += o == mine;
                    }
                const int count = above + before;
                const double mass = above_mass + static_cast<double>(before_units) * unit, each_mass = static_cast<double>(weighs) * unit;
                // the first logit that reaches it, or (a rounding short) the last
                const bool reached = count + same >= want_count || mass + same * each_mass >= want;
                const unsigned int first = wave_most(mine != 0 && reached ? mine : 0);
                const unsigned int last = ~wave_most(mine != 0 ? ~mine : 0);
                if (mine != 0 && mine == (first ? first : last)) {
                    int ties = min(same, want_count - count);
                    if (want < INFINITY) ties = static_cast<int>(fmin(ties, ceil((want - mass) / each_mass)));
                    ties = max(1, ties);
                    // equal lanes write the same
                    sh.cut = Cut{mine, ties, mass + ties * each_mass};
                }
            }
            __syncthreads();
            return sh.cut;
        }
    }
    // Adds a token of a bin to what its slice keeps of it; ties are counted apart.
    __device__ __forceinline__ void keep(bool cut_bin, Cut c, bool by_least, bool ties_pass, unsigned int o, int slice) const {
        const float z = value_of(o);
        if ((!cut_bin || o > c.order) && (!by_least || enough(z)))
            atomicAdd(&sh.mass[slice], static_cast<unsigned long long>(units_of(raise(at(z).r))));
        else if (ties_pass && o == c.order) atomicAdd(&sh.ties[slice], 1u);
    }
};

// What the workgroup needs to know of a row's slices, in LDS. False: no logit of the row is finite, or one
// has to be taken that equals the largest (of the slice `greedy`).
template <class E>
__device__ __forceinline__ bool open_row(Row<E>& r, const Info* info, int* greedy) {
    const int thread = threadIdx.x, lane = thread & 63;
    Shared& sh = r.sh;
    // the largest logit and the first slice that holds it, in every wave
    unsigned int best = 0, holder = 0;
    for (int i = lane; i < r.slices; i += 64) {
        const unsigned int o = info[i].best;
        if (o > best) best = o, holder = ~i;
    }
    const unsigned int mine = best;
    best = wave_most(best);
    *greedy = -1;
    if (best == 0) return false;
    r.frame = frame_of(value_of(best), r.s.heat);
    r.frame = Frame{from_lane(r.frame.per, 0), from_lane(r.frame.top, 0), from_lane(r.frame.low, 0), r.frame.most};  // scalar registers
    if (r.s.mode == kGreedy) {
        *greedy = static_cast<int>(~wave_most(mine == best ? holder : 0));
        return false;
    }
    for (int i = thread; i < r.slices; i += kDrawThreads) {
        const Info x = info[i];
        const float most = x.best != 0 ? value_of(x.best) : -INFINITY;
        const int shift = bin_of(most, r.frame);
        sh.shift[i] = shift;
        sh.mass[i] = 0;
        sh.ties[i] = 0;
        if (r.s.mode == kNoLimit) sh.kept[i] = shift < kBins && r.enough(most) ? x.mass * scale_of(-shift) : 0.0;
    }
    __syncthreads();
    return true;
}
// The slices' bins, added up.
template <class E>
__device__ __forceinline__ void add_bins(const Row<E>& r) {
    const int thread = threadIdx.x;
    if (thread < kLaneBins * 64) {
        double mass = 0.0;
        int count = 0;
        if (thread < kBins) {
#pragma unroll 8
            for (int i = 0; i < r.slices; ++i) {
                const int at = thread - r.sh.shift[i];
                const int64_t from = static_cast<int64_t>(i) * kBins + max(at, 0);  // read in any case: no branches
                const double w = r.masses[from];
                const int n = r.counts[from];
                mass += at >= 0 ? w : 0.0;
                count += at >= 0 ? n : 0;
            }
        }
        r.sh.bin_mass[thread] = mass * unit_of(thread);
        r.sh.bin_count[thread] = count;
    }
    __syncthreads();
}
// How many tokens the row's bins hold, and what they weigh.
__device__ __forceinline__ void all_of(const Shared& sh, int* count, double* mass) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    double w = 0.0;
#pragma unroll
    for (int h = 0; h < kLaneBins; ++h) {
        n += sh.bin_count[lane * kLaneBins + h];
        w += sh.bin_mass[lane * kLaneBins + h];
    }
    *count = from_lane(wave_sum_to(n), 63);
    *mass = from_lane(wave_sum_to(w), 63);
}
// The bin, of those up to `limit`, in which the order reaches k tokens or the weight p; in every wave.
__device__ __forceinline__ Place bin_of_limit(const Shared& sh, int limit, int k, double p) {
    const int lane = threadIdx.x & 63;
    int n[kLaneBins];
    double w[kLaneBins];
#pragma unroll
    for (int h = 0; h < kLaneBins; ++h) {
        n[h] = lane * kLaneBins + h <= limit ? sh.bin_count[lane * kLaneBins + h] : 0;
        w[h] = sh.bin_mass[lane * kLaneBins + h];
    }
    return first_reached(n, w, [&](int count, double mass) { return count >= k || mass >= p * (1.0 - kSame); });
}
// The bin that min-p falls in.
template <class E>
__device__ __forceinline__ int bin_of_least(const Row<E>& r) {
    return min(kBins - 1, -static_cast<int>(rint(r.at(r.frame.most).r + r.s.least)));
}
// Where the tokens of a bin are listed those of earlier ones may be too: with top-p to come behind top-k its
// bin is among them.
__device__ __forceinline__ int first_to_list(const Settings& s, int stage, int bin, int before, int in_bin) {
    return in_bin <= kList && stage == 0 && s.p < 1.0 && before + in_bin <= kList ? 0 : bin;
}

// Whether min-p cuts the order before the bin in which top-k or top-p does, and nothing else hangs on where.
__device__ __forceinline__ bool passed_by_least(const Settings& s, int stage, int bin, int bin_least) {
    return bin > bin_least && (stage == 1 || (stage == 0 && !(s.p < 1.0)));
}

template <class E>
__device__ __forceinline__ Row<E> row_of(const SampleArgs& a, const Layout& ws, int64_t row, int64_t here, int slices,
                                         Shared& sh) {
    return Row<E>{static_cast<const E*>(a.logits) + row * a.row_stride, static_cast<int>(a.vocab), slices,
                  settings_of(a, row), Frame{}, ws.masses + here * slices * kBins, ws.counts + here * slices * kBins, ws.list + here * list_of(a.vocab), 0, Raise(), sh};
}

// The bin in which a row is cut first, the logits that belong to it and the slices that hold any.
template <class E>
__global__ void __launch_bounds__(kDrawThreads) plan_kernel(SampleArgs a, int64_t first_row, Layout ws, int slices) {
    __shared__ Shared sh;
    const int64_t here = blockIdx.x;
    const int thread = threadIdx.x;
    Info* info = ws.info + here * slices;
    Plan* plan = ws.plan + here;
    Row<E> r = row_of<E>(a, ws, first_row + here, here, slices, sh);
    int greedy;
    if (!open_row(r, info, &greedy) || r.s.mode == kNoLimit) {
        if (thread == 0) plan->last = -1;
        return;
    }
    add_bins(r);
    if (thread < kLaneBins * 64) {
        plan->mass[thread] = sh.bin_mass[thread];
        plan->count[thread] = sh.bin_count[thread];
    }
    int all_n;
    double whole;
    all_of(sh, &all_n, &whole);
    int stage = r.s.k < all_n ? 0 : r.s.p < 1.0 ? 1 : 2;
    const int bin_least = bin_of_least(r);
    Place at{bin_least, 0, 0.0};
    if (stage < 2)
        at = bin_of_limit(sh, kBins, stage == 0 ? static_cast<int>(r.s.k) : INT32_MAX,
                          stage == 0 ? INFINITY : fmax(r.s.p, 0.0) * whole);
    if (passed_by_least(r.s, stage, at.at, bin_least)) stage = 2, at.at = bin_least;
    const int in_bin = sh.bin_count[at.at];
    const bool listed = in_bin > 0 && in_bin <= kList;
    const int first = first_to_list(r.s, stage, at.at, at.count, in_bin);
    if (listed) {
        r.set_range(first, at.at);
        for (int i = thread; i < slices; i += kDrawThreads)
            info[i].listed = sh.in_range[i];
    }
    if (thread == 0) {
        plan->first = first;
        plan->last = listed ? at.at : -1;
        plan->from = sh.from;
        plan->to = sh.to;
        plan->best = order_of(r.frame.most);
        plan->listed = 0;
    }
}

// The tokens that belong to it, a slice per workgroup. Eight waves to a SIMD: 48 us for 1024 x 151936 bfloat16, with
// the 90 registers that the compiler takes by itself 63.
template <class E>
__global__ void __launch_bounds__(kScanThreads, 8) list_kernel(SampleArgs a, int64_t first_row, Layout ws, int slices) {
    const int64_t task = blockIdx.x, here = task / slices, row = first_row + here;
    const int slice = static_cast<int>(task % slices), thread = threadIdx.x, lane = thread & 63;
    Plan* plan = ws.plan + here;
    const int first = plan->first, last = plan->last, some = ws.info[task].listed;
    const float from = plan->from, below = plan->to;
    const unsigned int best = plan->best;
    if (last < 0 || !some) return;
    const E* in = static_cast<const E*>(a.logits) + row * a.row_stride;
    const int vocab = static_cast<int>(a.vocab);
    float z[kEach];
    hold_slice(in, slice, vocab, z);
    unsigned int mine = 0;
    static_assert(kEach == 32, "");
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        mine |= static_cast<unsigned int>(z[i] >= from && z[i] < below) << i;
    }
    if (!__ballot(mine != 0)) return;
    const int n = __popc(mine), to = wave_sum_to(n);
    int put = 0;
    if (lane == 63) put = atomicAdd(&plan->listed, to);
    put = from_lane(put, 63) + to - n;
    Frame frame{};
    if (first < last) frame = frame_of(value_of(best), settings_of(a, row).heat);
    Token* list = ws.list + here * list_of(vocab);
    // a lane has few: they are read again rather than picked out of registers
    for (; mine; mine &= mine - 1, ++put) {
        const int id = held_id<E>(slice, vocab, __builtin_ctz(mine));
        const float z = Elem<E>::widen(in[id]);
        const int bin = first < last ? spot_of(z, frame).bin : last;
        if (put < list_of(vocab)) list[put] = Token{order_of(z), static_cast<unsigned int>(id) << 9 | bin};
    }
}

template <class E>
__global__ void __launch_bounds__(kDrawThreads, 4) draw_kernel(SampleArgs a, int64_t first_row, Layout ws, int slices) {
    __shared__ Shared sh;
    __shared__ float logit[kSlice];  // of the slice that holds the draw
    const int64_t here = blockIdx.x, row = first_row + here;
    const int thread = threadIdx.x, lane = thread & 63, wave = thread >> 6;
    Row<E> r = row_of<E>(a, ws, row, here, slices, sh);
    hold(r.raise);
    const Settings& s = r.s;
    const auto finish = [&](int token, double logp) {
        a.tokens_out[row] = token;
        a.logp_out[row] = static_cast<float>(logp);
    };
    int greedy;
    if (!open_row(r, ws.info + here * slices, &greedy)) {
        if (greedy < 0) {
            if (thread == 0) finish(-1, -INFINITY);
            return;
        }
        const auto raw = r.read(greedy);
        if (thread == 0) sh.least = ~0u;
        __syncthreads();
        unsigned int at = ~0u;
#pragma unroll
        for (int e = kDrawEach - 1; e >= 0; --e)
            if (allowed(r.get(raw, e)) && r.get(raw, e) == r.frame.most) at = r.id_of(greedy, e);
        if (at != ~0u) atomicMin(&sh.least, at);
        __syncthreads();
        if (thread == 0) finish(static_cast<int>(sh.least), 0.0);
        return;
    }
    const int bin_least = bin_of_least(r);
    int last_bin = bin_least;  // the last bin that any token is kept of
    Cut cut{0, 0, 0.0};        // and where it is cut, if anywhere but by min-p
    bool cut_bin = false;

    if (s.mode == kLimited) {
        const Plan* plan = ws.plan + here;
        if (thread < kLaneBins * 64) {
            sh.bin_mass[thread] = plan->mass[thread];
            sh.bin_count[thread] = plan->count[thread];
        }
        const int list_first = plan->last >= 0 ? plan->first : 1, list_last = plan->last;
        r.listed = plan->listed;
        __syncthreads();
        int all_n;
        double whole;  // what top-k leaves
        all_of(sh, &all_n, &whole);
        // The order is cut by top-k, then by top-p, each in the bin where it reaches its limit; then what each
        // slice keeps of the last bin is summed.
        int limit_bin = kBins;
#pragma unroll 1
        for (int stage = 0; stage < 3; ++stage) {
            if (stage == 0 ? s.k >= all_n : stage == 1 && !(s.p < 1.0)) continue;
            const int k = stage == 0 ? static_cast<int>(s.k) : INT32_MAX;
            const double p = stage == 1 ? fmax(s.p, 0.0) * whole : INFINITY;
            Place at{0, 0, 0.0};
            if (stage < 2) {
                at = bin_of_limit(sh, limit_bin, k, p);
                if (passed_by_least(s, stage, at.at, bin_least)) continue;
            } else {
                if (cut_bin && limit_bin <= bin_least) last_bin = limit_bin;
                else cut_bin = false;
                at.at = last_bin;
                if (sh.bin_count[last_bin] == 0) break;
            }
            const int bin = at.at;
            const bool in_list = bin >= list_first && bin <= list_last;
            if (!in_list) r.set_range(bin, bin);
            if (stage < 2) {
                const Cut c = r.cut(bin, in_list, stage == 0 ? k - at.count : INT32_MAX, p - at.mass);
                if (stage == 0) whole = at.mass + c.mass;
                const bool later = cut_bin && bin == limit_bin &&
                                   (c.order < cut.order || (c.order == cut.order && c.ties > cut.ties));
                if (!later) cut = c;
                limit_bin = bin;
                cut_bin = true;
            } else {
                const bool by_least = last_bin == bin_least;
                const bool ties_pass = cut_bin && (!by_least || r.enough(value_of(cut.order)));
                r.each_of(bin, in_list, [&](unsigned int o, int slice) __attribute__((always_inline)) {
                    r.keep(cut_bin, cut, by_least, ties_pass, o, slice);
                });
            }
        }
        // What each slice keeps of the bins above: a wave per slice, a lane per bin (those from
        // the 64th on belong to the first lanes again)
        for (int i = wave; i < slices; i += kDrawWaves) {
            const int down = sh.shift[i];
            double above = 0.0;
            for (int b = lane; b + down < last_bin; b += 64)
                above += r.masses[static_cast<int64_t>(i) * kBins + b] * unit_of(b + down);
#pragma unroll
            for (int o = 32; o >= 1; o >>= 1) above += __shfl_xor(above, o);
            if (lane == 0) sh.kept[i] = above;
        }
        __syncthreads();
    }

    // The slices' sums and ties, in their order, by the first wave: 64 at a time.
    if (wave == 0) {
        const double cut_weight = cut_bin ? weight(r.raise, r.at(value_of(cut.order))) : 0.0;
        double total = 0.0;
        int ties_before = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < slices; i0 += 64) {
            const int i = i0 + lane;
            const int ties = i < slices ? static_cast<int>(sh.ties[i]) : 0;
            const int ties_to = wave_sum_to(ties);
            const int taken = max(0, min(ties, cut.ties - (ties_before + ties_to - ties)));
            double kept = 0.0;
            if (i < slices) {
                kept = sh.kept[i] + static_cast<double>(sh.mass[i]) * unit_of(last_bin) + taken * cut_weight;
                sh.kept[i] = kept;
                sh.ties[i] = taken;
            }
            ties_before += from_lane(ties_to, 63);
            total += from_lane(wave_sum_to(kept), 63);
        }
        const float u = a.uniforms[row];
        const double target = static_cast<double>(u > 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f) * total * (1.0 + kSame);
        double before = 0.0;
        Place at{-1, 0, 0.0};
        int slice = -1;
#pragma unroll 1
        for (int i0 = 0; i0 < slices; i0 += 64) {
            const int i = i0 + lane;
            const double kept[1] = {i < slices ? sh.kept[i] : 0.0};
            const int some[1] = {kept[0] > 0.0};
            bool passes = false;
            const Place here = first_reached(some, kept, [&](int, double mass) { return before + mass > target; });
            if (here.at >= 0) {
                slice = i0 + here.at;
                at = Place{here.at, 0, before + here.mass};
                passes = at.mass + from_lane(kept[0], here.at) > target;
            }
            before += from_lane(wave_sum_to(kept[0]), 63);
            if (passes) break;
        }
        if (lane == 0) sh.slice = max(slice, 0), sh.rest = target - at.mass, sh.total = total;
    }
    __syncthreads();
    const int slice = sh.slice, take = static_cast<int>(sh.ties[slice]);
    const double rest = sh.rest, total = sh.total;

    // In that slice the token: each thread has kDrawEach consecutive ones, in LDS (its own place, so that a loop
    // over them is short).
    const auto raw = r.read(slice);
    float* const z = logit + thread;
    int same = 0;
#pragma unroll
    for (int e = 0; e < kDrawEach; ++e) {
        z[e * kDrawThreads] = r.get(raw, e);
        same += cut_bin && allowed(r.get(raw, e)) && order_of(r.get(raw, e)) == cut.order;
    }
    const int seen_before = cut_bin ? sum_to(same, sh.part_i) - same : 0;
    int seen = seen_before;
    const auto kept = [&](int e) __attribute__((always_inline)) {
        const float mine = z[e * kDrawThreads];
        if (!(mine < INFINITY)) return 0.0;
        const Spot at = r.at(mine);
        if (at.bin > last_bin) return 0.0;
        if (at.bin == last_bin) {
            const unsigned int o = order_of(mine);
            if (cut_bin && (o < cut.order || (o == cut.order && seen++ >= take))) return 0.0;
            if (last_bin == bin_least && !r.enough(mine)) return 0.0;
        }
        return weight(r.raise, at);
    };
    double sum = 0.0;
#pragma unroll 1
    for (int e = 0; e < kDrawEach; ++e) sum += kept(e);
    const double to = sum_to(sum, sh.part_d);
    // the first thread that passes, or (a rounding short) the last that keeps any
    const uint64_t some = __ballot(sum > 0.0), passing = __ballot(sum > 0.0 && to > rest);
    if (lane == 0) {
        sh.part_i[wave] = passing ? wave * 64 + __builtin_ctzll(passing) : -1;
        sh.part_j[wave] = some ? wave * 64 + 63 - __builtin_clzll(some) : -1;
    }
    __syncthreads();
    int chosen = -1;
    bool passed = false;
    for (int i = 0; i < kDrawWaves; ++i) {
        if (passed) continue;
        passed = sh.part_i[i] >= 0;
        chosen = passed ? sh.part_i[i] : max(chosen, sh.part_j[i]);
    }
    if (thread != chosen) return;
    // its first token that passes, or its last kept one
    double run = to - sum, w = 0.0;
    int at = 0;
    seen = seen_before;
#pragma unroll 1
    for (int e = 0; e < kDrawEach && !(w > 0.0 && run > rest); ++e) {
        const double mine = kept(e);
        if (!(mine > 0.0)) continue;
        run += mine;
        w = mine;
        at = e;
    }
    finish(r.id_of(slice, at), log(w / total));
}

template <class E>
hipError_t launch(const SampleArgs& a, void* workspace, hipStream_t stream) {
    const int64_t slices = slices_of(a.vocab);
    const int64_t most = held_rows(a.vocab, a.n_rows), passes = (a.n_rows + most - 1) / most;
    const int64_t rows = (a.n_rows + passes - 1) / passes;  // passes of even size
    Layout ws;
    ws.info = static_cast<Info*>(workspace);
    ws.plan = reinterpret_cast<Plan*>(ws.info + rows * slices);
    ws.list = reinterpret_cast<Token*>(ws.plan + rows);
    ws.masses = reinterpret_cast<double*>(ws.list + rows * list_of(a.vocab));
    ws.counts = reinterpret_cast<uint16_t*>(ws.masses + rows * slices * kBins);
    const bool limits = a.temperature.each || a.top_ks || a.top_p.each || a.min_p.each ||
                        (a.temperature.all > 0.0 &&
                         ((a.top_k > 0 && a.top_k < a.vocab) || a.top_p.all < 1.0 || a.min_p.all > kLeast));
    const int n_slices = static_cast<int>(slices);
    for (int64_t first = 0; first < a.n_rows; first += rows) {
        const int64_t n = std::min(rows, a.n_rows - first);
        const dim3 each_row(static_cast<unsigned int>(n)), each_slice(static_cast<unsigned int>(n * slices));
        scan_kernel<E><<<each_slice, dim3(kScanThreads), 0, stream>>>(a, first, ws, n_slices);
        if (limits) {
            plan_kernel<E><<<each_row, dim3(kDrawThreads), 0, stream>>>(a, first, ws, n_slices);
            list_kernel<E><<<each_slice, dim3(kScanThreads), 0, stream>>>(a, first, ws, n_slices);
        }
        draw_kernel<E><<<each_row, dim3(kDrawThreads), 0, stream>>>(a, first, ws, n_slices);
    }
    return hipGetLastError();
}

}  // namespace

int64_t sample_workspace_bytes(int, int64_t vocab, int64_t n_rows) {
    return held_rows(vocab, n_rows) * row_bytes(vocab);
}

hipError_t launch_sample(const SampleArgs& a, void* workspace, hipStream_t stream) {
    return a.type == kF32 ? launch<float>(a, workspace, stream) : launch<uint16_t>(a, workspace, stream);
}

}  // namespace kldk
