// Beam selection: the K best continuations of each item over its beams and the
// whole vocabulary.
//
// With s_w the score of beam w and z its logit row, a live beam offers token v
// at s_w + z_v - lse_w, lse_w = log sum exp z over the row's finite entries; a
// finished beam offers itself alone, at s_w. Of one beam's candidates the order
// is that of its logits (equal logits: the lowest id first), so a row's K
// largest logits hold all that can be chosen from it, and a slice's K largest
// all that can be chosen from the slice.
//
// Two launches. The scan reads every live row once: each wave streams one slice
// of a row, keeps the sum of exponentials against a running maximum and the
// slice's K largest logits. The merge joins the slices of an item's beams,
// forms the normalisers and scores in float64 and ranks the candidates. Its
// normalisers come from float32 exponentials; where two neighbours of the
// ranking, of different beams, are closer than those can tell, the item's
// workgroup reads its rows again in float64 and ranks once more.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kld_vocab.h"

namespace kldk {
namespace {

constexpr int kWaves = 4;        // waves per scan workgroup; they share nothing
constexpr int kChunks = 4;       // 16-byte chunks per lane and tile
constexpr int kTile = 64 * kChunks;  // chunks of a tile
constexpr int kList = 256;       // candidates a wave holds before it must drop some
constexpr int kMergeThreads = 256;
constexpr int kHold = 8;         // candidates a merge thread keeps in registers
constexpr int kMergeList = 1024;  // candidates the merge ranks at once

constexpr float kLog2e = 1.44269504088896340736f;
// Bounds of the float32 reference. Logits above the first, or rows that lie
// below the second altogether, would lose their sums in float32: the merge
// takes such rows in float64.
constexpr float kMostLogit = 1048576.0f;
constexpr float kLeastRef = -32768.0f * kLog2e;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

struct Cand {
    float z;
    int v;  // -1: none
};

// Sum of a slice: sum 2^(z log2e - ref) over its finite logits. A NaN sum:
// the slice holds logits past kMostLogit.
struct Slice {
    double sum;
    float ref;
    int n;  // candidates found in it
};

struct Layout {
    Slice* slice;  // [rows][slices]
    Cand* cand;    // [rows][slices][k]
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
    static __device__ __forceinline__ void set(u32x4& c, int e, uint16_t x) {
        const unsigned int w = c[e >> 1];
        c[e >> 1] = e & 1 ? (w & 0xffffu) | (static_cast<unsigned int>(x) << 16) : (w & 0xffff0000u) | x;
    }
    static __device__ __forceinline__ uint16_t none() { return 0xff80u; }
};
template <>
struct Elem<float> {
    static constexpr int kPer = 4;
    static constexpr unsigned int kNone = 0xff800000u;
    static __device__ __forceinline__ float get(const u32x4& c, int e) { return __uint_as_float(c[e]); }
    static __device__ __forceinline__ void set(u32x4& c, int e, float x) { c[e] = __float_as_uint(x); }
    static __device__ __forceinline__ float none() { return -INFINITY; }
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float(static_cast<unsigned int>(b) << 16); }

// Unsigned order of float values, -0 and 0 alike (none is NaN).
__device__ __forceinline__ unsigned int order_of(float z) {
    const unsigned int u = __float_as_uint(z + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned int o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
// Of two candidates of one row the one with the larger key comes first.
__device__ __forceinline__ uint64_t key_of(float z, int v) {
    return (static_cast<uint64_t>(order_of(z)) << 32) | (0xffffffffu - static_cast<unsigned int>(v));
}

// The k best of the wave's n candidates (n <= kList), in order, at the list's
// front; each lane ranks up to kList / 64 of them against all.
__device__ __forceinline__ int keep_best(uint64_t* list, int n, int k, int lane) {
    constexpr int kMine = kList / 64;
    uint64_t mine[kMine];
    int rank[kMine];
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
        mine[q] = q * 64 + lane < n ? list[q * 64 + lane] : 0;
        rank[q] = 0;
    }
    for (int i = 0; i < n; ++i) {
        const uint64_t other = list[i];
#pragma unroll
        for (int q = 0; q < kMine; ++q)
            if (q * 64 < n) rank[q] += other > mine[q];
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < kMine; ++q)
        if (q * 64 + lane < n && rank[q] < k) list[rank[q]] = mine[q];
    __builtin_amdgcn_wave_barrier();
    return n < k ? n : k;
}

// A value that at least k lanes reach (none: -inf), from the upper 16 bits of
// the k-th largest lane value: the k-th largest of a superset is no smaller.
__device__ __forceinline__ float reached_by(float x, int k) {
    const unsigned int o = order_of(x);
    unsigned int t = 0;
#pragma unroll
    for (int b = 31; b >= 16; --b) {
        const unsigned int c = t | (1u << b);
        if (__popcll(__ballot(o >= c)) >= k) t = c;
    }
    const float v = value_of(t);
    return v > -INFINITY ? v : -INFINITY;   // also where the bits say NaN: fewer than k lanes hold a finite value
}

template <class E>
__global__ void __launch_bounds__(kWaves * 64)
    beam_scan_kernel(const E* __restrict__ logits, int64_t vocab, int64_t row_stride, int64_t rows, int slices,
                     int tiles_per_slice, int k, int drop_at, const float* __restrict__ scores,
                     const uint8_t* __restrict__ finished, Layout out) {
    constexpr int kPer = Elem<E>::kPer;
    constexpr int kEach = kChunks * kPer;  // elements per lane and tile
    __shared__ uint64_t lists[kWaves][kList];
    __shared__ u32x4 stages[kWaves][64 * kChunks];
    __shared__ int owners[kWaves][64];
    const int lane = threadIdx.x & 63;
    const int64_t task = static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6);
    const int64_t row = task / slices;
    if (row >= rows) return;
    const int slice = static_cast<int>(task - row * slices);
    const float score = scores[row];
    if (!isfinite(score) || (finished && finished[row])) return;  // its logits offer nothing
    uint64_t* list = lists[threadIdx.x >> 6];
    u32x4* stage = stages[threadIdx.x >> 6];
    int* owner = owners[threadIdx.x >> 6];

    // chunk c of the row: elements [c kPer - off, c kPer - off + kPer), 16-byte aligned
    const E* p = logits + row * row_stride;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(E));
    const E* base = p - off;
    const int64_t chunks = (vocab + off + kPer - 1) / kPer;
    const int64_t full_from = off ? 1 : 0, full_to = (vocab + off) / kPer;  // chunks that lie in the row as a whole
    const int64_t c_first = static_cast<int64_t>(slice) * tiles_per_slice * kTile;
    int64_t c_last = c_first + static_cast<int64_t>(tiles_per_slice) * kTile;
    if (c_last > chunks) c_last = chunks;

    const auto load = [&](int64_t c0, u32x4(&r)[kChunks]) {
        if (c0 >= full_from && c0 + kTile <= full_to && c0 + kTile <= c_last) {
#pragma unroll
            for (int u = 0; u < kChunks; ++u)
                r[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(base + (c0 + u * 64 + lane) * kPer));
        } else {
#pragma unroll
            for (int u = 0; u < kChunks; ++u) {
                const int64_t c = c0 + u * 64 + lane;
                const unsigned int none = Elem<E>::kNone;
                r[u] = u32x4{none, none, none, none};
                if (c < c_last) {
                    if (c >= full_from && c < full_to) {
                        r[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(base + c * kPer));
                    } else {
#pragma unroll
                        for (int e = 0; e < kPer; ++e) {
                            const int64_t i = c * kPer + e - off;
                            if (i >= 0 && i < vocab) Elem<E>::set(r[u], e, p[i]);
                        }
                    }
                }
            }
        }
    };

    float ref = kLeastRef;  // in binary units
    double sum = 0.0;
    bool wild = false;
    float least = -INFINITY;  // a logit below it is no candidate
    uint64_t least_key = 0;
    int n = 0;
    u32x4 r[kChunks], next[kChunks];
    if (c_first < c_last) load(c_first, r);
    for (int64_t c0 = c_first; c0 < c_last; c0 += kTile) {
        const bool more = c0 + kTile < c_last;
        if (more) load(c0 + kTile, next);

        float best, part, to;
        for (bool clean = false;; clean = true) {
            best = -INFINITY;
#pragma unroll
            for (int u = 0; u < kChunks; ++u) {
#pragma unroll
                for (int e = 0; e < kPer; ++e) best = fmaxf(best, Elem<E>::get(r[u], e));
            }
            to = fmaxf(ref, best * kLog2e);
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int u = 0; u < kChunks; ++u)
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    acc[e & 3] += __builtin_amdgcn_exp2f(__builtin_fmaf(Elem<E>::get(r[u], e), kLog2e, -to));
            part = (acc[0] + acc[1]) + (acc[2] + acc[3]);
            // a NaN among the logits makes the sum NaN, an infinity or a logit too large shows in the largest
            if (clean || !__ballot(!(part >= 0.0f) || !(best <= kMostLogit))) break;
#pragma unroll
            for (int u = 0; u < kChunks; ++u)
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (!isfinite(Elem<E>::get(r[u], e))) Elem<E>::set(r[u], e, Elem<E>::none());
        }
        wild |= !(best <= kMostLogit);
        sum = sum * static_cast<double>(__builtin_amdgcn_exp2f(ref - to)) + static_cast<double>(part);
        ref = to;

        if (c0 == c_first) {
            least = reached_by(best, k);
            least_key = least > -INFINITY ? static_cast<uint64_t>(order_of(least)) << 32 : 0;
        }
        // Lanes that hold a candidate lay their elements side by side, then the
        // whole wave looks at them, one element per lane.
        const bool hit = best >= least && best > -INFINITY;
        const unsigned long long hits = __ballot(hit);
        if (hits) {
            if (hit) {
                const int slot = __popcll(hits & ((1ull << lane) - 1));
                owner[slot] = lane;
#pragma unroll
                for (int u = 0; u < kChunks; ++u) stage[slot * kChunks + u] = r[u];
            }
            __builtin_amdgcn_wave_barrier();
            const int held = __popcll(hits) * kEach;
            for (int i0 = 0; i0 < held; i0 += 64) {
                const int i = i0 + lane;
                const int e = i % kEach;
                const bool there = i < held;
                const float z = there ? widen(reinterpret_cast<const E*>(stage)[i]) : -INFINITY;
                const int64_t chunk = c0 + (e / kPer) * 64 + (there ? owner[i / kEach] : 0);
                const uint64_t key = key_of(z, static_cast<int>(chunk * kPer + e % kPer - off));
                const bool in = z > -INFINITY && key > least_key;
                const unsigned long long b = __ballot(in);
                if (!b) continue;
                if (in) list[n + __popcll(b & ((1ull << lane) - 1))] = key;
                n += __popcll(b);
                __builtin_amdgcn_wave_barrier();
                if (n > kList - 64) {
                    n = keep_best(list, n, k, lane);
                    least_key = list[k - 1];
                    least = value_of(static_cast<unsigned int>(least_key >> 32));
                }
            }
            if (n >= drop_at) {
                n = keep_best(list, n, k, lane);
                if (n == k) {
                    least_key = list[k - 1];
                    least = value_of(static_cast<unsigned int>(least_key >> 32));
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kChunks; ++u) r[u] = next[u];
    }

    n = keep_best(list, n, k, lane);
    if (lane < k) {
        const uint64_t key = lane < n ? list[lane] : 0;
        out.cand[(row * slices + slice) * k + lane] =
            lane < n ? Cand{value_of(static_cast<unsigned int>(key >> 32)),
                            static_cast<int>(0xffffffffu - static_cast<unsigned int>(key))}
                     : Cand{-INFINITY, -1};
    }
    float whole = ref;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) whole = fmaxf(whole, __shfl_xor(whole, o));
    sum *= static_cast<double>(__builtin_amdgcn_exp2f(ref - whole));
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
    wild = __ballot(wild) != 0;
    if (lane == 0) out.slice[row * slices + slice] = Slice{wild ? static_cast<double>(NAN) : sum, whole, n};
}

// A scored candidate and the order of the selection.
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

__device__ __forceinline__ unsigned int order_hi(double s) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(s));
    return static_cast<unsigned int>((u >> 63 ? ~u : u | (uint64_t{1} << 63)) >> 32);
}
__device__ __forceinline__ double value_hi(unsigned int o) {
    const uint64_t u = static_cast<uint64_t>(o) << 32;
    return __longlong_as_double(static_cast<long long>(u >> 63 ? u ^ (uint64_t{1} << 63) : ~u));
}

template <class E>
__global__ void __launch_bounds__(kMergeThreads)
    beam_merge_kernel(const E* __restrict__ logits, int64_t vocab, int64_t row_stride, int n_beams, int slices,
                      int group, int k, double tol, const float* scores, const uint8_t* finished, int eos, Layout in,
                      float* scores_out, int32_t* __restrict__ parents_out, int32_t* __restrict__ tokens_out,
                      uint8_t* finished_out) {
    constexpr int kW = kMergeThreads / 64;
    enum { kEmpty, kLive, kFinished, kRetake, kExact };  // kRetake: live, its normaliser is to be taken in float64
    __shared__ float score[kBeamMaxBeams];
    __shared__ double lse[kBeamMaxBeams];
    __shared__ int state[kBeamMaxBeams];
    __shared__ Scored list[kMergeList];
    __shared__ Scored ranked[kBeamMaxSelect + 1];
    __shared__ double dred[kW];
    __shared__ unsigned int bound[kW];
    __shared__ Scored pick[kW];
    __shared__ int count, again;
    const int64_t item = blockIdx.x;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int per = slices * k, total = n_beams * per;
    const Cand* cands = in.cand + item * total;
    const Slice* parts = in.slice + item * n_beams * slices;

    // the first kHold candidates of a thread stay in registers
    Cand held[kHold];
    int beam[kHold];
#pragma unroll
    for (int c = 0; c < kHold; ++c) {
        const int i = t + c * kMergeThreads;
        beam[c] = i < total ? i / per : -1;
        if (i < total) held[c] = cands[i];
    }

    // normalisers, `group` lanes per beam; scores and flags are read before anything is written
    for (int w0 = 0; w0 < n_beams; w0 += kMergeThreads / group) {
        const int w = w0 + t / group, g = t % group;
        if (w >= n_beams) continue;
        const float s = scores[item * n_beams + w];
        const int st = !isfinite(s) ? kEmpty : finished && finished[item * n_beams + w] ? kFinished : kLive;
        float ref = kLeastRef;
        double sum = 0.0;
        int found = 0;
        if (st == kLive) {
            for (int i = g; i < slices; i += group) {
                const Slice q = parts[w * slices + i];
                const float to = fmaxf(ref, q.ref);
                sum = sum * static_cast<double>(__builtin_amdgcn_exp2f(ref - to)) +
                      q.sum * static_cast<double>(__builtin_amdgcn_exp2f(q.ref - to));
                ref = to;
                found |= q.n;
            }
            float to = ref;
            for (int o = group >> 1; o >= 1; o >>= 1) to = fmaxf(to, __shfl_xor(to, o));
            sum *= static_cast<double>(__builtin_amdgcn_exp2f(ref - to));
            ref = to;
            for (int o = group >> 1; o >= 1; o >>= 1) {
                sum += __shfl_xor(sum, o);
                found |= __shfl_xor(found, o);
            }
        }
        if (g == 0) {
            score[w] = s;
            // a sum below 1/2 never reached its reference: all of the row lies below kLeastRef
            const bool sound = sum > 0.5;
            state[w] = st == kLive && found && !sound ? kRetake : st;
            lse[w] = sound ? (static_cast<double>(ref) + log2(sum)) / static_cast<double>(kLog2e) : 0.0;
        }
    }
    __syncthreads();

    const auto scored = [&](int i, int w, const Cand& x, Scored& c) {  // false: there is no such candidate
        const int st = state[w];
        if (st == kFinished) {
            c = Scored{static_cast<double>(score[w]), 0.0f, w, eos};
            return i == w * per;
        }
        c = Scored{score[w] + (static_cast<double>(x.z) - lse[w]), x.z, w, x.v};
        return st != kEmpty && x.v >= 0;
    };
    const auto each = [&](auto&& f) {
        Scored c;
#pragma unroll
        for (int q = 0; q < kHold; ++q)
            if (beam[q] >= 0 && scored(t + q * kMergeThreads, beam[q], held[q], c)) f(c);
        for (int i = t + kHold * kMergeThreads; i < total; i += kMergeThreads)
            if (scored(i, i / per, cands[i], c)) f(c);
    };

    // Every further round has taken at least one more row in float64.
    for (;;) {
        for (int w = 0; w < n_beams; ++w) {
            if (state[w] != kRetake) continue;
            float m = -INFINITY;
            for (int i = t; i < slices; i += kMergeThreads) {
                const Cand c = cands[(w * slices + i) * k];
                if (c.v >= 0) m = fmaxf(m, c.z);
            }
#pragma unroll
            for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
            __syncthreads();
            if (lane == 0) dred[wave] = m;
            __syncthreads();
            for (int q = 0; q < kW; ++q) m = fmaxf(m, static_cast<float>(dred[q]));
            double sum = 0.0;
            const E* p = logits + (item * n_beams + w) * row_stride;
            for (int64_t i = t; i < vocab; i += kMergeThreads) {
                const float z = widen(p[i]);
                if (isfinite(z)) sum += exp(static_cast<double>(z) - m);
            }
#pragma unroll
            for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
            __syncthreads();
            if (lane == 0) dred[wave] = sum;
            __syncthreads();
            if (t == 0) {
                sum = 0.0;
                for (int q = 0; q < kW; ++q) sum += dred[q];
                lse[w] = m + log(sum);
                state[w] = kExact;
            }
        }
        __syncthreads();

        // a score that k candidates reach, then the candidates near or above it
        double mine = -INFINITY;
        each([&](const Scored& c) { mine = fmax(mine, c.s); });
        const unsigned int o = mine > -INFINITY ? order_hi(mine) : 0;
        unsigned int b = 0;
#pragma unroll
        for (int bit = 31; bit >= 8; --bit) {
            const unsigned int c = b | (1u << bit);
            if (__popcll(__ballot(o >= c)) >= k) b = c;
        }
        if (lane == 0) bound[wave] = b;
        if (t == 0) count = again = 0;
        __syncthreads();
        b = 0;
#pragma unroll
        for (int q = 0; q < kW; ++q) b = bound[q] > b ? bound[q] : b;
        const double least = b ? value_hi(b) - tol : -INFINITY;
        each([&](const Scored& c) {
            if (c.s >= least) {
                const int at = atomicAdd(&count, 1);
                if (at < kMergeList) list[at] = c;
            }
        });
        __syncthreads();
        const int n = count;
        const int m = n < k + 1 ? n : k + 1;
        if (n <= kMergeList) {
            for (int i0 = 0; i0 < n; i0 += kMergeThreads / 4) {  // four lanes per candidate
                const int i = i0 + (t >> 2);
                int rank = 0;
                Scored c{};
                if (i < n) {
                    c = list[i];
                    for (int j = t & 3; j < n; j += 4) rank += before(list[j], c);
                }
                rank += __shfl_xor(rank, 1);
                rank += __shfl_xor(rank, 2);
                if (i < n && (t & 3) == 0 && rank < m) ranked[rank] = c;
            }
        } else {
            // too many near one another (long ties): one after the other
            const Scored none{-INFINITY, -INFINITY, 0x7fffffff, 0x7fffffff};
            for (int j = 0; j < m; ++j) {
                Scored best = none;
                each([&](const Scored& c) {
                    if ((j == 0 || before(ranked[j - 1], c)) && before(c, best)) best = c;
                });
#pragma unroll
                for (int d = 32; d >= 1; d >>= 1) {
                    const Scored other{__shfl_xor(best.s, d), __shfl_xor(best.z, d), __shfl_xor(best.w, d),
                                       __shfl_xor(best.v, d)};
                    if (before(other, best)) best = other;
                }
                if (lane == 0) pick[wave] = best;
                __syncthreads();
                if (t == 0) {
                    for (int q = 1; q < kW; ++q)
                        if (before(pick[q], best)) best = pick[q];
                    ranked[j] = best;
                }
                __syncthreads();
            }
        }
        __syncthreads();
        if (t + 1 < m && ranked[t].w != ranked[t + 1].w && ranked[t].s - ranked[t + 1].s <= tol)
            for (int q = 0; q < 2; ++q)
                if (state[ranked[t + q].w] == kLive) {
                    state[ranked[t + q].w] = kRetake;
                    again = 1;
                }
        __syncthreads();
        if (!again) break;
    }

    if (t < k) {
        const int64_t at = item * k + t;
        const bool some = t < count;
        const Scored c = ranked[some ? t : 0];
        scores_out[at] = some ? static_cast<float>(c.s) : -INFINITY;
        parents_out[at] = some ? c.w : -1;
        tokens_out[at] = some ? c.v : -1;
        finished_out[at] = some && (state[c.w] == kFinished || c.v == eos);
    }
}

struct Shape {
    int slices;
    int tiles_per_slice;
};

// Slices of a row: enough waves to fill the chip, none shorter than a tile.
Shape shape_of(int type, int64_t vocab, int64_t rows) {
    const int64_t per_tile = int64_t{64} * kChunks * (type == kBF16 ? 8 : 4);
    const int64_t tiles = (vocab + 15) / per_tile + 1;  // a row that starts inside a chunk may touch one tile more
    int64_t slices = (4096 + rows - 1) / rows;
    if (slices > tiles) slices = tiles;
    const int64_t per = (tiles + slices - 1) / slices;
    return Shape{static_cast<int>((tiles + per - 1) / per), static_cast<int>(per)};
}

int64_t align16(int64_t b) { return (b + 15) & ~int64_t{15}; }

template <class E>
hipError_t launch_typed(const BeamArgs& a, void* workspace, hipStream_t stream) {
    const int64_t rows = a.n_items * a.n_beams;
    const Shape sh = shape_of(a.type, a.vocab, rows);
    Layout lay;
    lay.slice = static_cast<Slice*>(workspace);
    lay.cand = reinterpret_cast<Cand*>(static_cast<char*>(workspace) +
                                       align16(rows * sh.slices * static_cast<int64_t>(sizeof(Slice))));
    const E* logits = static_cast<const E*>(a.logits);
    const int drop_at = a.n_select * 2 > 32 ? a.n_select * 2 : 32;
    const int64_t blocks = (rows * sh.slices + kWaves - 1) / kWaves;
    beam_scan_kernel<E><<<dim3(static_cast<unsigned>(blocks)), kWaves * 64, 0, stream>>>(
        logits, a.vocab, a.row_stride, rows, sh.slices, sh.tiles_per_slice, a.n_select, drop_at, a.scores, a.finished,
        lay);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // Twice what a float32 normaliser may be off, in nats: the exponentials'
    // arguments, rounded by 2^-24 of themselves, average at most log2 V (a
    // distribution's mean -log2 p) times ln 2; an exponential is off by 2^-23,
    // a sum of 8 and 2 more additions by 2^-24 each, log2 e by 2^-26 of the
    // entropy.
    const double tol = 2.0 * 0x1p-24 * (24.0 + log2(static_cast<double>(a.vocab)));
    int group = 1;  // lanes that join one beam's slices
    while (group < sh.slices && group < 64) group *= 2;
    beam_merge_kernel<E><<<dim3(static_cast<unsigned>(a.n_items)), kMergeThreads, 0, stream>>>(
        logits, a.vocab, a.row_stride, a.n_beams, sh.slices, group, a.n_select, tol, a.scores, a.finished, a.eos, lay,
        a.scores_out, a.parents_out, a.tokens_out, a.finished_out);
    return hipGetLastError();
}

}  // namespace

int64_t beam_workspace_bytes(int type, int64_t vocab, int64_t n_items, int n_beams, int n_select) {
    const int64_t rows = n_items * n_beams;
    if (rows == 0) return 0;
    const Shape sh = shape_of(type, vocab, rows);
    return align16(rows * sh.slices * static_cast<int64_t>(sizeof(Slice))) +
           rows * sh.slices * n_select * static_cast<int64_t>(sizeof(Cand));
}

hipError_t launch_beam_select(const BeamArgs& a, void* workspace, hipStream_t stream) {
    return a.type == kBF16 ? launch_typed<uint16_t>(a, workspace, stream) : launch_typed<float>(a, workspace, stream);
}

}  // namespace kldk
