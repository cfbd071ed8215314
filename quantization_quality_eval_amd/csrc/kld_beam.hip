// Beam selection: the K best continuations of each item over its beams and the
// whole vocabulary.
//
// With s_w the score of beam w and z its logit row, a live beam offers token v
// at s_w + z_v - lse_w, lse_w = log sum exp z over the row's finite entries; a
// finished beam offers itself alone, at s_w. Of one beam's candidates the order
// is that of its logits (equal logits: the lowest id first).
//
// Two launches. The scan streams every live row once and keeps nothing but the
// sum of its exponentials and the largest logit of each group of consecutive
// elements (128 of bfloat16, 64 of float32). The merge forms the item's
// normalisers, bounds the K-th best group from below, reads the groups that
// reach the bound again -- every chosen candidate is in one of them, as K of them
// hold a candidate that good -- and ranks their elements in float64. The
// normalisers come from float32 exponentials; where two neighbours of the
// ranking, of different beams, are closer than those can tell, or the last chosen
// and any candidate of another beam behind it, the item's workgroup reads the rows
// concerned again in float64 and ranks once more.
//
// Measured on MI355X (kernel times). 128 items x 8 beams of 151936 bfloat16, one
// beam in eight finished, K = 16: scan 50 us, 272 MB at 5.4 TB/s, of which about 30
// us are vector instructions; merge 14 us. The same in float32: 116 us in all, 545 MB at
// 4.7 TB/s. 32 x 4, K = 8: 8.7 + 11 us. 4 rows of 32000: 3.8 + 8.8 us. Candidate lists kept by the scan's waves cost 62 to 72 us for
// the largest case instead of 50: a list has a handful of arrivals per tile for
// most of a row, and each cost more instructions than the tile's exponentials.
#include <float.h>
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kld_vocab.h"

namespace kldk {
namespace {

constexpr int kWaves = 4;            // waves per scan workgroup; they share nothing
constexpr int kChunks = 4;           // 16-byte chunks per lane and tile
constexpr int kTile = 64 * kChunks;  // chunks of a tile
constexpr int kGroupChunks = 16;     // chunks of a group: those of 16 neighbouring lanes
constexpr int kTileGroups = kTile / kGroupChunks;
constexpr int64_t kTargetWaves = 8192;  // of a scan: 4096 and 16384 are 7% slower and 2% faster for
                                        // the largest case above, 9% and 4% slower for the second
constexpr int kMergeThreads = 512;   // 256 and 1024 take up to 4 us more
constexpr int kMergeList = 1024;     // candidates the merge ranks at once
constexpr int kHold = 6;             // quadruples of groups that a merge thread keeps in registers
constexpr int kNear = 512;           // groups that the merge reads again at most

constexpr float kLog2e = 1.44269504088896340736f;
// A sum's reference is its largest logit in binary units, rounded up to a whole
// number: going over to a higher one multiplies the sum by a power of two, exactly,
// however often a rising row does so. Bounds of the reference (logits of 2^20 and
// -2^15). Logits above the first, or rows that lie below the second altogether, would
// lose their sums in float32: the merge takes such rows in float64.
constexpr float kMostRef = 1512776.0f;
constexpr float kLeastRef = -47275.0f;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Sum of a slice: sum 2^(z log2e - ref) over its finite logits, ref a whole number. A
// NaN sum: the slice holds logits past kMostRef.
struct Slice {
    double sum;
    float ref;
    int unused;
};

struct Layout {
    Slice* slice;  // [rows][slices]
    float* top;    // [rows][groups], in the order of their elements
};

template <class E>
struct Elem;
template <>
struct Elem<uint16_t> {
    static constexpr int kPer = 8;  // elements per chunk
    static constexpr unsigned int kNone = 0xff80ff80u;
    static __device__ __forceinline__ float get(const u32x4& c, int e) {
        const unsigned int w = c[e >> 1];
        return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
    }
};
template <>
struct Elem<float> {
    static constexpr int kPer = 4;
    static constexpr unsigned int kNone = 0xff800000u;
    static __device__ __forceinline__ float get(const u32x4& c, int e) { return __uint_as_float(c[e]); }
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float(static_cast<unsigned int>(b) << 16); }

// A row: `head` elements before the first 16-byte boundary, whole chunks, and
// the elements behind the last of them; the ones outside the chunks are loose.
template <class E>
struct Row {
    const E* p;
    int head;
    int chunks;
    int tail_at;
    int loose;
    __device__ __forceinline__ Row(const E* row, int64_t vocab) : p(row) {
        constexpr int kPer = Elem<E>::kPer;
        const int to_chunk = static_cast<int>(-(reinterpret_cast<uintptr_t>(row) / sizeof(E)) & (kPer - 1));
        head = to_chunk < vocab ? to_chunk : static_cast<int>(vocab);
        chunks = static_cast<int>((vocab - head) / kPer);
        tail_at = head + chunks * kPer;
        loose = head + static_cast<int>(vocab - tail_at);
    }
    __device__ __forceinline__ int loose_id(int i) const { return i < head ? i : tail_at + (i - head); }
};

// Signed order of float values (none is NaN), its own inverse on the bits.
__device__ __forceinline__ int signed_order(int bits) { return bits ^ ((bits >> 31) & 0x7fffffff); }
// Maximum over the 16 lanes of a row: with the neighbour, the other pair of the
// quad, the other quad of the half, the other half. On integers it is one
// instruction a step; on floats the compiler quiets both operands first.
template <int kCtrl>
__device__ __forceinline__ int max_with(int x) {
    return max(x, __builtin_amdgcn_mov_dpp(x, kCtrl, 0xf, 0xf, true));
}
__device__ __forceinline__ int row_max(float x) {
    return max_with<0x140>(max_with<0x141>(max_with<0x4e>(max_with<0xb1>(signed_order(__float_as_int(x))))));
}

__device__ __forceinline__ float ref_of(float z) { return ceilf(z * kLog2e); }
// A sum over the reference `from`, over `to` >= from. 2^-4096 of it is nothing: that
// takes in references of infinity too.
__device__ __forceinline__ double over(double sum, float from, float to) {
    return ldexp(sum, static_cast<int>(fmaxf(from - to, -4096.0f)));
}

// One wave per slice of a row, a tile of 2048 (1024) elements at a time with the
// next in flight; waves share nothing. Per lane a running reference and sum: the
// exponentials of a tile are added in float32, tiles in float64. A tile costs
// about five vector instructions per element (unpack, maximum, scale, exponential,
// add); with 4 KB per wave in flight memory bounds it.
template <class E>
__global__ void __launch_bounds__(kWaves * 64)
    beam_scan_kernel(const E* __restrict__ logits, int64_t vocab, int64_t row_stride, int64_t rows, int slices,
                     int tiles, int tiles_per_slice, const float* __restrict__ scores,
                     const uint8_t* __restrict__ finished, Layout out) {
    constexpr int kPer = Elem<E>::kPer;
    constexpr int kEach = kChunks * kPer;  // elements per lane and tile
    const int lane = threadIdx.x & 63;
    const int64_t task = static_cast<int64_t>(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = task / slices;
    if (row >= rows) return;
    const int slice = static_cast<int>(task - row * slices);
    const Row<E> in(logits + row * row_stride, vocab);
    const u32x4* body = reinterpret_cast<const u32x4*>(in.p + in.head) + lane;
    const int t0 = slice * tiles_per_slice;
    const int t1 = t0 + tiles_per_slice < tiles ? t0 + tiles_per_slice : tiles;

    u32x4 r[kChunks];
    const auto load = [&](int tile) {
        const int c0 = tile * kTile;
        if (c0 + kTile <= in.chunks) {
#pragma unroll
            for (int u = 0; u < kChunks; ++u) r[u] = __builtin_nontemporal_load(body + c0 + u * 64);
        } else {
            const int left = in.chunks - c0 - lane;
#pragma unroll
            for (int u = 0; u < kChunks; ++u) {
                const unsigned int none = Elem<E>::kNone;
                r[u] = u32x4{none, none, none, none};
                if (u * 64 < left) r[u] = __builtin_nontemporal_load(body + c0 + u * 64);
            }
        }
    };
    if (t0 < t1) load(t0);
    // a row that offers nothing: known after its first tile is on its way
    if (!isfinite(scores[row]) || (finished && finished[row])) return;

    // the first four lanes of each row of 16 store its maxima, a chunk each
    float* top = out.top + (row * tiles + t0) * kTileGroups + (lane & 3) * (kTileGroups / kChunks) + (lane >> 4);
    float ref = kLeastRef;  // of this lane, in binary units
    double sum = 0.0;
    for (int tile = t0; tile < t1; ++tile) {
        float x[kEach];
#pragma unroll
        for (int u = 0; u < kChunks; ++u)
#pragma unroll
            for (int e = 0; e < kPer; ++e) x[u * kPer + e] = Elem<E>::get(r[u], e);
        if (tile + 1 < t1) load(tile + 1);
        float best[kChunks], part, to;
        for (bool clean = false;; clean = true) {
#pragma unroll
            for (int u = 0; u < kChunks; ++u) {
                best[u] = x[u * kPer];
#pragma unroll
                for (int e = 1; e < kPer; ++e) best[u] = fmaxf(best[u], x[u * kPer + e]);
            }
            to = fmaxf(ref, ref_of(fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3]))));
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < kEach; ++i) acc[i & 3] += __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], kLog2e, -to));
            part = (acc[0] + acc[1]) + (acc[2] + acc[3]);
            // a NaN or an infinity among the logits makes the sum NaN: exclude them
            if (clean || !__ballot(!(part >= 0.0f))) break;
#pragma unroll
            for (int i = 0; i < kEach; ++i) x[i] = isfinite(x[i]) ? x[i] : -INFINITY;
        }
        sum = over(sum, ref, to) + static_cast<double>(part);
        ref = to;
        int mine = row_max(best[0]);
#pragma unroll
        for (int u = 1; u < kChunks; ++u) {
            const int q = row_max(best[u]);
            mine = (lane & 3) == u ? q : mine;
        }
        static_assert(kChunks == 4 && kGroupChunks == 16, "");
        if ((lane & 12) == 0) *top = __int_as_float(signed_order(mine));
        top += kTileGroups;
    }
    if (slice == 0 && lane < in.loose) {
        const float z = widen(in.p[in.loose_id(lane)]);
        if (isfinite(z)) {
            const float to = fmaxf(ref, ref_of(z));
            sum = over(sum, ref, to) + static_cast<double>(__builtin_amdgcn_exp2f(__builtin_fmaf(z, kLog2e, -to)));
            ref = to;
        }
    }
    float whole = ref;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) whole = fmaxf(whole, __shfl_xor(whole, o));
    sum = over(sum, ref, whole);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
    if (lane == 0) out.slice[row * slices + slice] = Slice{whole <= kMostRef ? sum : static_cast<double>(NAN), whole, 0};
}

// A scored candidate and the order of the selection. For a group, z is its
// largest logit and v its place among the row's groups.
struct Scored {
    double s;
    float z;
    int w;
    int v;
};
__device__ __forceinline__ bool before(const Scored& a, const Scored& b) {
    if (a.s != b.s) return a.s > b.s;
    if (a.w != b.w) return a.w < b.w;
    if (a.z != b.z) return a.z > b.z;
    return a.v < b.v;
}

__device__ __forceinline__ unsigned int order_of(float z) {
    const unsigned int u = __float_as_uint(z + 0.0f);  // -0 and 0 are alike
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned int o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
// Values that `few` and that `many` of the wave's lanes reach, at most 1/128 of its
// distance from the wave's largest below the few-th and the many-th largest; -inf where
// fewer lanes hold a finite one. The upper 16 bits of a distance are enough; those of the
// value itself are not, its size being that of a score: steps of 4 to 8 at -600 let
// thousands of groups reach the bound (11 ms instead of 65 us for the largest case
// above), and all 32 bits cost each call 0.9 us.
__device__ __forceinline__ float2 reached_by(float x, int few, int many) {
    const int rows = row_max(x);  // of each 16 lanes
    const int best = max(max(__builtin_amdgcn_readlane(rows, 0), __builtin_amdgcn_readlane(rows, 16)),
                         max(__builtin_amdgcn_readlane(rows, 32), __builtin_amdgcn_readlane(rows, 48)));
    const float top = __int_as_float(signed_order(best));
    if (!(top > -INFINITY)) return float2{-INFINITY, -INFINITY};
    const unsigned int o = order_of(x - top);
    unsigned int a = 0, b = 0;
#pragma unroll 2
    for (unsigned int bit = 1u << 31; bit >= 1u << 16; bit >>= 1) {
        a |= __popcll(__ballot(o >= (a | bit))) >= few ? bit : 0;
        b |= __popcll(__ballot(o >= (b | bit))) >= many ? bit : 0;
    }
    // a distance is NaN below the lowest finite one; it and its sum with the largest are
    // off by 2^-24 of themselves, which is taken off
    const auto below = [&](float d) {
        return d > -INFINITY ? (top + d) - 0x1p-22f * (fabsf(top) + fabsf(d)) : -INFINITY;
    };
    return float2{below(value_of(a)), below(value_of(b))};
}

// kRetake: live, its normaliser is to be taken in float64. kExact: it was.
enum : int { kEmpty, kLive, kFinished, kRetake, kExact };

// log2 of a positive normal number, off by less than 3 x 2^-24: its exponent, and
// the float32 logarithm of its mantissa in [1, 2).
__device__ __forceinline__ double log2_of(double x) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x));
    const double mantissa = __longlong_as_double(static_cast<long long>((u & 0xfffffffffffffull) | 0x3ff0000000000000ull));
    return static_cast<double>(static_cast<int>(u >> 52) - 1023) +
           static_cast<double>(__builtin_amdgcn_logf(static_cast<float>(mantissa)));
}

struct Merge {
    float score[kBeamMaxBeams];
    double lse[kBeamMaxBeams];
    float shift[kBeamMaxBeams];  // score - lse, rounded; NaN where that passes float32's range; -inf for a
                                 // beam that offers no logits
    int state[kBeamMaxBeams];
    f32x4 quad[kNear];           // quadruples with groups worth reading,
    int2 quad_at[kNear];         // their beams and first groups
    int2 near[kNear];            // those groups: beam, place
    double list_s[kMergeList];   // candidates: score,
    uint64_t list_k[kMergeList]; // beam and logit, the first of equal scores with the least,
    int list_v[kMergeList];      // id
    Scored ranked[kBeamMaxSelect];
    Scored pick[kMergeThreads / 64];
    double part[kMergeThreads / 64];
    float bound[kMergeThreads / 64][2];
    int count, quad_count, near_count, again;
    __device__ __forceinline__ void set_shift(int w) {
        const float x = static_cast<float>(score[w] - lse[w]);
        shift[w] = !live(w) ? -INFINITY : fabsf(x) < INFINITY ? x : NAN;
    }
    __device__ __forceinline__ bool live(int w) const { return state[w] == kLive || state[w] == kExact; }
    __device__ __forceinline__ Scored scored(float z, int w, int v) const {
        return Scored{score[w] + (static_cast<double>(z) - lse[w]), z, w, v};
    }
    __device__ __forceinline__ void add(const Scored& c) {
        const int at = atomicAdd(&count, 1);
        if (at >= kMergeList) return;
        list_s[at] = c.s;
        list_k[at] = (static_cast<uint64_t>(c.w) << 32) | ~order_of(c.z);
        list_v[at] = c.v;
    }
    // The beam's normaliser is too coarse for the order: it is taken again.
    __device__ __forceinline__ void ask(int w) {
        if (state[w] == kLive) state[w] = kRetake, again = 1;
    }
    // Whether a candidate that was not chosen may belong before the last chosen one. It
    // need not be the next in order: others of the last one's beam, equal logits for
    // instance, can stand between.
    __device__ __forceinline__ void ask_near(const Scored& last, double s, int w, double tol) {
        if (w == last.w || last.s - s > tol || s > last.s || (s == last.s && w < last.w)) return;
        ask(w);
        ask(last.w);
    }
    // The list's first m entries in order; four lanes per entry count the ones
    // before it, without a branch: equal logits of one beam are common.
    __device__ __forceinline__ void rank(int n, int m) {
        const int t = threadIdx.x;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += kMergeThreads / 4) {
            const int i = i0 + (t >> 2), q = i < n ? i : 0;
            const double s = list_s[q];
            const uint64_t k = list_k[q];
            const int v = list_v[q];
            int at = 0;
#pragma unroll 4
            for (int j = t & 3; j < n; j += 4) {
                const double os = list_s[j];
                const uint64_t ok = list_k[j];
                const int ov = list_v[j];
                at += (os > s) | ((os == s) & ((ok < k) | ((ok == k) & (ov < v))));
            }
            at += __shfl_xor(at, 1);
            at += __shfl_xor(at, 2);
            if (i < n && (t & 3) == 0 && at < m)
                ranked[at] = Scored{s, value_of(~static_cast<unsigned int>(k)), static_cast<int>(k >> 32), v};
        }
    }
};

// The item as its workgroup sees it.
template <class E>
struct Item {
    const E* rows;
    int64_t row_stride;
    int64_t vocab;
    int n_beams;
    int groups;
    int eos;
    const float* tops;
    __device__ __forceinline__ Row<E> row(int w) const { return Row<E>(rows + w * row_stride, vocab); }
    // Candidates that no group holds: finished beams and loose elements.
    template <class F>
    __device__ __forceinline__ void each_loose(const Merge& s, F&& f) const {
#pragma unroll 1
        for (int i = threadIdx.x; i < n_beams * 16; i += kMergeThreads) {
            const int w = i >> 4, q = i & 15;
            if (s.state[w] == kFinished) {
                if (q == 0) f(Scored{static_cast<double>(s.score[w]), 0.0f, w, eos});
            } else if (s.live(w)) {
                const Row<E> r = row(w);
                if (q >= r.loose) continue;
                const int v = r.loose_id(q);
                const float z = widen(r.p[v]);
                if (isfinite(z)) f(s.scored(z, w, v));
            }
        }
    }
};

// The rare parts of the merge stand in functions of their own, so that what
// every call runs stays small: a merge is as long as its instructions take to
// arrive.

// Normalisers in float64, of every beam whose state asks for it.
template <class E>
__device__ __attribute__((noinline)) void retake(Merge& s, const Item<E>& item) {
    constexpr int kW = kMergeThreads / 64;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    for (int w = 0; w < item.n_beams; ++w) {
        if (s.state[w] != kRetake) continue;
        const Row<E> row = item.row(w);
        float most = -INFINITY;
        double sum = 0.0;
        for (int i = t; i < item.groups; i += kMergeThreads)
            most = fmaxf(most, item.tops[static_cast<int64_t>(w) * item.groups + i]);
        if (t < row.loose) {
            const float z = widen(row.p[row.loose_id(t)]);
            if (isfinite(z)) most = fmaxf(most, z);
        }
        for (int o = 32; o >= 1; o >>= 1) most = fmaxf(most, __shfl_xor(most, o));
        __syncthreads();
        if (lane == 0) s.part[wave] = most;
        __syncthreads();
        for (int q = 0; q < kW; ++q) most = fmaxf(most, static_cast<float>(s.part[q]));
        for (int64_t i = most > -INFINITY ? t : item.vocab; i < item.vocab; i += kMergeThreads) {
            const float z = widen(row.p[i]);
            if (isfinite(z)) sum += exp(static_cast<double>(z) - most);
        }
        for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
        __syncthreads();
        if (lane == 0) s.part[wave] = sum;
        __syncthreads();
        if (t == 0) {
            sum = 0.0;
            for (int q = 0; q < kW; ++q) sum += s.part[q];
            s.lse[w] = most + log(sum);
            s.state[w] = most > -INFINITY ? kExact : kEmpty;  // empty: every logit is excluded
            s.set_shift(w);
        }
    }
    __syncthreads();
}

// Too many candidates near one another (long ties): the first m <= most one
// after the other. A group is looked into where its largest logit beats what
// the thread has found. One more pass asks for the beams with candidates near the
// last one. Returns m.
template <class E>
__device__ __attribute__((noinline)) int pick_slowly(Merge& s, const Item<E>& item, int most, double tol) {
    constexpr int kW = kMergeThreads / 64, kPer = Elem<E>::kPer, kOfGroup = kGroupChunks * kPer;
    const Scored none{-INFINITY, -INFINITY, 0x7fffffff, 0x7fffffff};
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    // f(candidate) for every candidate of the groups whose largest logit passes at(z, w)
    const auto each = [&](auto&& at, auto&& f) {
        for (int w = 0; w < item.n_beams; ++w) {
            if (!s.live(w)) continue;
            const Row<E> row = item.row(w);
            for (int i = t; i < item.groups; i += kMergeThreads) {
                const float z = item.tops[static_cast<int64_t>(w) * item.groups + i];
                if (!(z > -INFINITY) || !at(z, w)) continue;
                for (int e = 0; e < kOfGroup; ++e) {
                    const int64_t v = row.head + int64_t{i} * kOfGroup + e;
                    if (v >= row.tail_at) break;
                    const float x = widen(row.p[v]);
                    if (isfinite(x)) f(s.scored(x, w, static_cast<int>(v)));
                }
            }
        }
        item.each_loose(s, f);
    };
    for (int j = 0; j < most; ++j) {
        Scored best = none;
        const auto consider = [&](const Scored& c) {
            if ((j == 0 || before(s.ranked[j - 1], c)) && before(c, best)) best = c;
        };
        each([&](float z, int w) { return s.scored(z, w, 0).s > best.s || (best.w == w && z > best.z); }, consider);
        for (int d = 32; d >= 1; d >>= 1) {
            const Scored other{__shfl_xor(best.s, d), __shfl_xor(best.z, d), __shfl_xor(best.w, d),
                               __shfl_xor(best.v, d)};
            if (before(other, best)) best = other;
        }
        __syncthreads();
        if (lane == 0) s.pick[wave] = best;
        __syncthreads();
        for (int q = 0; q < kW; ++q)
            if (before(s.pick[q], best)) best = s.pick[q];
        if (best.w == none.w) return j;
        if (t == 0) s.ranked[j] = best;
        __syncthreads();
    }
    const Scored last = s.ranked[most - 1];
    each([&](float z, int w) { return w != last.w && last.s - s.scored(z, w, 0).s <= tol; },
         [&](const Scored& c) { s.ask_near(last, c.s, c.w, tol); });
    return most;
}

// One workgroup per item. Latency bounds it: three dependent reads (sums and
// maxima, then the best groups) and nine barriers, at 1 to 2 us per step for few
// groups; nothing in it is repeated per logit.
template <class E>
__global__ void __launch_bounds__(kMergeThreads)
    beam_merge_kernel(const E* __restrict__ logits, int64_t vocab, int64_t row_stride, int n_beams, int slices,
                      int group, int tiles, int loose, int64_t first_item, int k, double tol, const float* scores, const uint8_t* finished, int eos,
                      Layout in, float* scores_out, int32_t* __restrict__ parents_out,
                      int32_t* __restrict__ tokens_out, uint8_t* finished_out) {
    constexpr int kW = kMergeThreads / 64;
    constexpr int kPer = Elem<E>::kPer;
    __shared__ Merge s;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int groups = tiles * kTileGroups;
    const int64_t this_item = first_item + blockIdx.x, first_beam = this_item * n_beams;
    const Item<E> item{logits + first_beam * row_stride, row_stride, vocab, n_beams, groups, eos,
                       in.top + first_beam * groups};

    // The largest logits of the groups, four at a time, or one where that leaves
    // threads idle; a thread's first kHold stay in registers.
    const int wide = n_beams * groups <= kMergeThreads * kHold ? 1 : 4;
    const int per = groups / wide, total = n_beams * per;
    const auto tops_of = [&](int i) {
        if (wide == 4) return reinterpret_cast<const f32x4*>(item.tops)[i];
        return f32x4{item.tops[i], -INFINITY, -INFINITY, -INFINITY};
    };
    f32x4 held[kHold];
    int beam[kHold];
#pragma unroll
    for (int q = 0; q < kHold; ++q) {
        const int i = t + q * kMergeThreads;
        held[q] = f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (i < total) held[q] = tops_of(i);
    }
    // normalisers, `group` lanes per beam; scores and flags are read before anything is written
#pragma unroll 1
    for (int w0 = 0; w0 < n_beams; w0 += kMergeThreads / group) {
        const int w = w0 + t / group, g = t % group;
        if (w >= n_beams) continue;
        const Slice* parts = in.slice + (first_beam + w) * slices;
        Slice q{0.0, kLeastRef, 0};
        if (g < slices) q = parts[g];  // not written if the beam is not live: not used then
        const float score = scores[first_beam + w];
        const bool ended = finished && finished[first_beam + w];
        const int st = !isfinite(score) ? kEmpty : ended ? kFinished : kLive;
        float ref = q.ref;
        double sum = q.sum;
#pragma unroll 1
        for (int i = g + group; i < slices; i += group) {
            q = parts[i];
            const float to = fmaxf(ref, q.ref);
            sum = over(sum, ref, to) + over(q.sum, q.ref, to);
            ref = to;
        }
        float to = ref;
#pragma unroll 1
        for (int o = group >> 1; o >= 1; o >>= 1) to = fmaxf(to, __shfl_xor(to, o));
        sum = over(sum, ref, to);
#pragma unroll 1
        for (int o = group >> 1; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
        if (g == 0) {
            // a row that reaches its reference holds a logit less than a unit below it, and its sum 1/2; one
            // below 1/4: all of the row lies below kLeastRef, or is excluded
            const bool sound = st == kLive && sum > 0.25;
            s.score[w] = score;
            s.state[w] = st == kLive && !sound ? kRetake : st;
            s.lse[w] = sound ? (static_cast<double>(to) + log2_of(sum)) / static_cast<double>(kLog2e) : 0.0;
            s.set_shift(w);
        }
    }
#pragma unroll
    for (int q = 0; q < kHold; ++q) {
        const int i = t + q * kMergeThreads;
        beam[q] = i < total ? static_cast<int>(static_cast<unsigned int>(i) / static_cast<unsigned int>(per)) : 0;
    }
    const auto best_of = [](const f32x4& q) { return fmaxf(fmaxf(q[0], q[1]), fmaxf(q[2], q[3])); };
    __syncthreads();
    static_assert(kBeamMaxBeams <= 64, "a lane per beam");
    if (__ballot(lane < n_beams && s.state[lane] == kRetake)) retake(s, item);

    int m;
    // Every further round has taken at least one more row in float64.
    for (;;) {
        // What k groups reach: each of the waves holds `share` lanes that reach the least
        // of their bounds, or one wave holds k. z + shift is formed in float32 here; shift
        // and sum are off by 2^-24 of themselves, which is taken off the bounds. A sum that
        // cannot be formed (NaN) or that passes float32's range claims nothing, and nothing
        // is left out for it: whether a token is excluded is a matter of its logit alone.
        float mine = -INFINITY;
        const auto look = [&](const f32x4& q, int w) {
            const float shift = s.shift[w], sc = best_of(q) + shift;
            mine = fmaxf(mine, sc - 0x1p-22f * (fabsf(sc) + fabsf(shift)));
        };
#pragma unroll
        for (int q = 0; q < kHold; ++q) {
            if (q * kMergeThreads >= total) break;
            look(held[q], beam[q]);
        }
#pragma unroll 1
        for (int i = t + kHold * kMergeThreads; i < total; i += kMergeThreads) look(tops_of(i), i / per);
        const float2 reached = reached_by(mine, (k + kW - 1) / kW, k);
        if (lane == 0) s.bound[wave][0] = reached.x, s.bound[wave][1] = reached.y;
        if (t == 0) s.count = s.quad_count = s.near_count = s.again = 0;
        __syncthreads();
        float least_f = s.bound[0][0], alone = s.bound[0][1];
#pragma unroll
        for (int q = 1; q < kW; ++q) {
            least_f = fminf(least_f, s.bound[q][0]);
            alone = fmaxf(alone, s.bound[q][1]);
        }
        least_f = fmaxf(least_f, alone);
        // the groups that may reach it, or come near it, by the same sums
        const auto reach = [&](float shift) {
            return least_f - 0x1p-22f * (fabsf(least_f) + fabsf(shift)) - 2.0f * static_cast<float>(tol);
        };
        const auto reaches = [&](const f32x4& q, int w) {
            const float shift = s.shift[w], best = best_of(q);
            return shift != -INFINITY && best > -INFINITY && !(best + shift < reach(shift));
        };
        const auto take = [&](const f32x4& q, int i, int w) {
            if (!reaches(q, w)) return;
            const int at = atomicAdd(&s.quad_count, 1);
            if (at >= kNear) return;
            s.quad[at] = q;
            s.quad_at[at] = int2{w, (i - w * per) * wide};
        };
#pragma unroll
        for (int q = 0; q < kHold; ++q) {
            if (q * kMergeThreads >= total) break;
            take(held[q], t + q * kMergeThreads, beam[q]);
        }
#pragma unroll 1
        for (int i = t + kHold * kMergeThreads; i < total; i += kMergeThreads) take(tops_of(i), i, i / per);
        __syncthreads();
        const int quads = s.quad_count;
#pragma unroll 1
        for (int i = t; i < min(quads, kNear) * 4; i += kMergeThreads) {
            const float z = reinterpret_cast<const float*>(s.quad)[i];
            const int2 q = s.quad_at[i >> 2];
            const float shift = s.shift[q.x];
            if (z > -INFINITY && !(z + shift < reach(shift))) {
                const int at = atomicAdd(&s.near_count, 1);
                if (at < kNear) s.near[at] = int2{q.x, q.y + (i & 3)};
            }
        }
        __syncthreads();
        const int near = s.near_count;
        bool fits = quads <= kNear && near <= kNear;
        if (fits) {
            // their elements
#pragma unroll 1
            for (int i = t; i < near * kGroupChunks; i += kMergeThreads) {
                const int2 g = s.near[i / kGroupChunks];
                const Row<E> row = item.row(g.x);
                const int64_t c = int64_t{g.y} * kGroupChunks + i % kGroupChunks;
                if (c >= row.chunks) continue;
                const u32x4 x = reinterpret_cast<const u32x4*>(row.p + row.head)[c];
                const float shift = s.shift[g.x], from = reach(shift);
                const int v = row.head + static_cast<int>(c) * kPer;
#pragma unroll 1
                for (int j = 0; j < 4; ++j) {
                    const unsigned int word = j < 2 ? (j == 0 ? x[0] : x[1]) : (j == 2 ? x[2] : x[3]);
#pragma unroll
                    for (int e = 0; e < kPer / 4; ++e) {
                        const float z = Elem<E>::get(u32x4{word, 0, 0, 0}, e);
                        if (isfinite(z) && !(z + shift < from)) s.add(s.scored(z, g.x, v + j * (kPer / 4) + e));
                    }
                }
            }
            if (loose)
                item.each_loose(s, [&](const Scored& c) {
                    if (!(static_cast<float>(c.s) < reach(s.shift[c.w]))) s.add(c);
                });
            else if (t < n_beams && s.state[t] == kFinished)
                s.add(Scored{static_cast<double>(s.score[t]), 0.0f, t, eos});
            __syncthreads();
            const int n = s.count;
            fits = n <= kMergeList;
            m = n < k ? n : k;
            if (fits) s.rank(n, m);
            __syncthreads();
            // the list holds whatever comes within tol of the last place
            if (fits && m == k) {
                const Scored last = s.ranked[k - 1];
#pragma unroll 1
                for (int i = t; i < n; i += kMergeThreads)
                    s.ask_near(last, s.list_s[i], static_cast<int>(s.list_k[i] >> 32), tol);
            }
        }
        if (!fits) m = pick_slowly(s, item, k, tol);
        if (t + 1 < m) {
            const Scored x = s.ranked[t], y = s.ranked[t + 1];
            if (x.w != y.w && x.s - y.s <= tol) {
                s.ask(x.w);
                s.ask(y.w);
            }
        }
        __syncthreads();
        if (!s.again) break;
        retake(s, item);
    }

    if (t < k) {
        const int64_t at = this_item * k + t;
        const bool some = t < m;
        const Scored c = s.ranked[some ? t : 0];
        scores_out[at] = some ? static_cast<float>(c.s) : -INFINITY;
        parents_out[at] = some ? c.w : -1;
        tokens_out[at] = some ? c.v : -1;
        finished_out[at] = some && (s.state[c.w] == kFinished || c.v == eos);
    }
}

struct Shape {
    int tiles;  // of every row, also of one that begins inside a chunk
    int tiles_per_slice;
    int slices;
};

// Slices of a row: enough waves to fill the chip, none with less than a tile.
Shape shape_of(int type, int64_t vocab, int64_t rows) {
    const int64_t per_tile = int64_t{kTile} * (type == kBF16 ? 8 : 4);
    const int64_t tiles = (vocab + per_tile - 1) / per_tile;
    int64_t slices = (kTargetWaves + rows - 1) / rows;
    if (slices > tiles) slices = tiles;
    const int64_t per = (tiles + slices - 1) / slices;
    return Shape{static_cast<int>(tiles), static_cast<int>(per), static_cast<int>((tiles + per - 1) / per)};
}

int64_t align16(int64_t b) { return (b + 15) & ~int64_t{15}; }

template <class E>
hipError_t launch_typed(const BeamArgs& a, void* workspace, hipStream_t stream) {
    const int64_t rows = a.n_items * a.n_beams;
    const Shape sh = shape_of(a.type, a.vocab, rows);
    Layout lay;
    lay.slice = static_cast<Slice*>(workspace);
    lay.top = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                       align16(rows * sh.slices * static_cast<int64_t>(sizeof(Slice))));
    const E* logits = static_cast<const E*>(a.logits);
    const int64_t blocks = (rows * sh.slices + kWaves - 1) / kWaves;
    beam_scan_kernel<E><<<dim3(static_cast<unsigned>(blocks)), kWaves * 64, 0, stream>>>(
        logits, a.vocab, a.row_stride, rows, sh.slices, sh.tiles, sh.tiles_per_slice, a.scores, a.finished, lay);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // Twice what a float32 normaliser may be off, in nats and units of 2^-24: the
    // exponentials' arguments, rounded by one unit of themselves, average at most
    // log2 V + 2 (a distribution's mean -log2 p, and a sum of 1/4 at least) times ln 2;
    // an exponential is off by 2 units; 8 and 2 additions by one each; the logarithm by
    // 3 ln 2; log2 e by a quarter of the entropy, 0.16 log2 V: 16 + 0.86 log2 V. Tiles,
    // lanes and slices are joined exactly, in float64 and by powers of two.
    const double tol = 2.0 * 0x1p-24 * (24.0 + log2(static_cast<double>(a.vocab)));
    // whether a row may have elements outside its chunks
    constexpr int kPer = Elem<E>::kPer;
    const int loose = reinterpret_cast<uintptr_t>(logits) % 16 != 0 || a.row_stride % kPer != 0 || a.vocab % kPer != 0;
    int group = 1;  // lanes that join one beam's slices
    while (group < sh.slices && group < 64) group *= 2;
    const int64_t per = max_blocks_per_launch(kMergeThreads);
    for (int64_t first = 0; first < a.n_items; first += per) {
        const int64_t n = a.n_items - first < per ? a.n_items - first : per;
        beam_merge_kernel<E><<<dim3(static_cast<unsigned>(n)), kMergeThreads, 0, stream>>>(
            logits, a.vocab, a.row_stride, a.n_beams, sh.slices, group, sh.tiles, loose, first, a.n_select, tol,
            a.scores, a.finished, a.eos, lay, a.scores_out, a.parents_out, a.tokens_out, a.finished_out);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

int64_t beam_workspace_bytes(int type, int64_t vocab, int64_t n_items, int n_beams, int) {
    const int64_t rows = n_items * n_beams;
    if (rows == 0) return 0;
    const Shape sh = shape_of(type, vocab, rows);
    return align16(rows * sh.slices * static_cast<int64_t>(sizeof(Slice))) +
           rows * sh.tiles * kTileGroups * static_cast<int64_t>(sizeof(float));
}

hipError_t launch_beam_select(const BeamArgs& a, void* workspace, hipStream_t stream) {
    return a.type == kBF16 ? launch_typed<uint16_t>(a, workspace, stream) : launch_typed<float>(a, workspace, stream);
}

}  // namespace kldk
