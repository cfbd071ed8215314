// Embedding lookup with scaling, and its gradient by sorted tokens.
//
// Lookup: out[n] = scale * table[t_n]; a negative id gives a zero row, an id
// past the vocabulary a NaN row.
//
// Gradient: dtable[v] = scale * sum over { n : t_n = v } of grad[n]. A sort of
// the positions by their id makes each row's sum one run of the sorted order,
// added up in an order that depends on the tokens alone:
//   1. group: the positions grouped by id, each id's in increasing order. Few
//      positions: wave p of P owns the ids v with v mod P = p; it reads every
//      id, counts its own and the ones of the waves before it, and writes its
//      positions; no wave waits for another. More: a counting sort by v mod P
//      first (count, scatter), after which a workgroup sorts one residue's.
//   2. sum: the sorted order is cut into pieces of 8 to 32 positions; a workgroup
//      adds up the runs of one piece for one tile of columns. A run that lies
//      in the piece is done; of a run that reaches past it the piece's part is
//      kept in float32. Further workgroups of the launch set the rows that no
//      position names to zero.
//   3. join: the parts of each run that was cut, in order.
//
// Measured on MI355X. Lookup of 16384 rows of 151936 x 2048 bfloat16 into float32: 33
// us for 164 MB (5.0 TB/s; one row per thread instead of four: 49). Gradient of 16384
// positions x 4096 bfloat16 into a bfloat16 table of 32000: 100 us in all, of which
// the sort takes 16, the sum and the zeros 60 to 74 (396 MB) and the join 8; of
// 65536 positions x 256 into float32 x 151936: 69 us (sort 25, sum 27, join 8); of 100
// positions: 12 us in three launches. Large sums are bound by memory, small ones by
// the launches, which depend on one another.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "kld_vocab.h"

namespace kldk {
namespace {

constexpr int kThreads = 256;
constexpr int kOwned = 512;  // ids one wave owns at most

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float(static_cast<unsigned int>(b) << 16); }

// float -> bfloat16 bits, round to nearest even; NaN stays NaN. One instruction for two.
__device__ __forceinline__ uint16_t to_bf16(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}
// V consecutive elements as one load or store (V * sizeof(E) is 2 to 16 bytes).
template <class E, int V>
struct alignas(V * sizeof(E)) Vec {
    E x[V];
};

// V float64 results, each rounded once to nearest even. On its way to bfloat16 a
// value is rounded to float32 first; as the midpoints of bfloat16 are float32 values,
// that takes no value across one, but may put a value onto one that lies beside it.
// Only there (one value in 65536) is the float64 looked at again: it says which side,
// and a step of the float32 to that side rounds as it does.
template <class EO, int V>
__device__ __forceinline__ Vec<EO, V> rounded(const double (&x)[V]) {
    Vec<EO, V> o;
    if constexpr (sizeof(EO) == 4) {
#pragma unroll
        for (int e = 0; e < V; ++e) o.x[e] = static_cast<float>(x[e]);
    } else {
        unsigned int u[V];
        bool midpoint = false;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            u[e] = __float_as_uint(static_cast<float>(x[e]));
            midpoint |= (u[e] & 0xffffu) == 0x8000u;
        }
        if (midpoint) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if ((u[e] & 0xffffu) != 0x8000u) continue;
                const double here = fabs(static_cast<double>(__uint_as_float(u[e]))), from = fabs(x[e]);
                u[e] += (here < from) - (here > from);
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) o.x[e] = to_bf16(__uint_as_float(u[e]));
    }
    return o;
}

// How a launch covers rows and columns: `lanes` threads (a power of two from 64
// to kThreads) of V elements each take one tile of a row's columns, tile after
// tile, row unit after row unit; `first`: the launch's first workgroup.
struct Cover {
    int64_t first;
    int lanes;
    int tiles;
};
struct Place {
    int64_t unit;
    int64_t col;
};
template <int V>
__device__ __forceinline__ Place place_of(const Cover& c) {
    const int64_t i = (c.first + blockIdx.x) * (kThreads / c.lanes) + threadIdx.x / c.lanes;
    return Place{i / c.tiles, (i % c.tiles * c.lanes + threadIdx.x % c.lanes) * V};
}

template <int V>
Cover cover_of(int64_t dim) {
    Cover c{0, 64, 1};
    while (c.lanes < kThreads && int64_t{c.lanes} * V < dim) c.lanes *= 2;
    c.tiles = static_cast<int>((dim + int64_t{c.lanes} * V - 1) / (int64_t{c.lanes} * V));
    return c;
}

// Launch f(c, blocks) until `units` row units are covered.
template <class F>
hipError_t launch_cover(Cover c, int64_t units, F&& f) {
    const int64_t in_block = kThreads / c.lanes, per = max_blocks_per_launch(kThreads);
    const int64_t n = (units * c.tiles + in_block - 1) / in_block;
    for (; c.first < n; c.first += per) {
        f(c, dim3(static_cast<unsigned>(n - c.first < per ? n - c.first : per)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Whether rows of `dim` elements can be accessed V elements at a time.
bool allows(int v, int64_t dim, const void* p, int64_t stride, size_t size) {
    return dim % v == 0 && stride % v == 0 && reinterpret_cast<uintptr_t>(p) % (v * size) == 0;
}
// Elements of 16 bytes of the wider type.
template <class A, class B>
constexpr int widest() {
    return sizeof(A) + sizeof(B) == 4 ? 8 : 4;
}

// ---- lookup ----

constexpr int kRows = 4;              // rows a thread of a large lookup takes
constexpr int64_t kFullWaves = 8192;  // what a large lookup leaves at least

// R consecutive positions per row unit, their rows in flight together.
template <class ET, class EO, int V, int R>
__global__ void __launch_bounds__(kThreads)
    embed_kernel(const ET* __restrict__ table, int64_t vocab, int64_t dim, int64_t table_stride,
                 const int32_t* __restrict__ tokens, int64_t n_tokens, double scale, EO* __restrict__ out,
                 int64_t out_stride, Cover c) {
    const Place at = place_of<V>(c);
    const int64_t n0 = at.unit * R;
    if (n0 >= n_tokens || at.col >= dim) return;
    int32_t t[R];
    Vec<ET, V> x[R];
#pragma unroll
    for (int q = 0; q < R; ++q) t[q] = n0 + q < n_tokens ? tokens[n0 + q] : -1;
#pragma unroll
    for (int q = 0; q < R; ++q)
        if (t[q] >= 0 && t[q] < vocab)
            x[q] = *reinterpret_cast<const Vec<ET, V>*>(table + t[q] * table_stride + at.col);
#pragma unroll
    for (int q = 0; q < R; ++q) {
        if (n0 + q >= n_tokens) break;
        double z[V];
        if (t[q] >= 0 && t[q] < vocab) {
#pragma unroll
            for (int e = 0; e < V; ++e) z[e] = static_cast<double>(widen(x[q].x[e])) * scale;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) z[e] = t[q] < 0 ? 0.0 : static_cast<double>(NAN);
        }
        *reinterpret_cast<Vec<EO, V>*>(out + (n0 + q) * out_stride + at.col) = rounded<EO, V>(z);
    }
}

// ---- gradient ----

// Positions per piece of the sum: 32 where that makes waves enough to fill the
// chip, down to 8 where it does not (adding 8192 x 1000 float32: 20 us with 32, 15
// with 16, 14 with 8; 16384 x 4096 bfloat16: the join takes 9 us with 32, 12 with 16).
constexpr int kMostPiece = 32;
constexpr int kLeastPiece = 8;
constexpr int64_t kPieceWaves = 4096;
constexpr int kAhead = 8;     // rows in flight per thread; 16 cost registers (85 -> 107 us, 16384 x 4096)
constexpr int kZeroRows = 8;  // rows of the table that a thread zeroes
static_assert(kMostPiece < 64, "a lane per position and one more");

// The counting sort of many positions.
constexpr int kLgBuckets = 10;
constexpr int kBuckets = 1 << kLgBuckets;
constexpr int kBucketIds = 1024;      // ids of one bucket at most
constexpr int kSortThreads = 1024;
constexpr int kMostChunks = 32;       // workgroups of its first two launches
constexpr int64_t kChunkTokens = 1024;  // positions of one of them at least
// Up to here every wave reads every id: 12 us in all for 256 positions against 17
// sorted, 16 and 18 for 1024, 22 and 19 for 2048.
constexpr int64_t kFewTokens = 1536;

struct GradSpace {
    int32_t* total;    // positions with a valid id
    int32_t* perm;     // n_tokens: positions grouped by id
    int32_t* word;     // n_tokens + 1: their ids, then -1
    int32_t* count;    // positions of id v at [(v mod P) * owned + v / P]
    float* part;       // [pieces][2][dim]: a piece's part of the run that enters it, of the run that leaves it
    int lg;            // log2 P
    int owned;         // ids per residue
    int piece;         // positions per piece
    int pieces;
    // counting sort only (chunks > 0)
    int chunks;
    int64_t chunk_tokens;
    int32_t* hist;     // [chunks][kBuckets]
    int32_t* start;    // kBuckets + 1: where each bucket begins
    int32_t* bperm;    // n_tokens: positions by bucket
    int32_t* bword;    // n_tokens: their ids
};

int64_t align16(int64_t b) { return (b + 15) & ~int64_t{15}; }

GradSpace grad_space(void* ws, int64_t vocab, int64_t dim, int64_t n_tokens, int64_t* bytes) {
    GradSpace g{};
    const bool sort = n_tokens > kFewTokens && vocab <= int64_t{kBuckets} * kBucketIds;
    g.lg = kLgBuckets;
    if (!sort)
        while ((int64_t{kOwned} << g.lg) < vocab) ++g.lg;
    g.owned = static_cast<int>((vocab + (int64_t{1} << g.lg) - 1) >> g.lg);
    g.piece = kMostPiece;
    while (g.piece > kLeastPiece && n_tokens / g.piece * ((dim + 255) / 256) < kPieceWaves) g.piece /= 2;
    g.pieces = static_cast<int>((n_tokens + g.piece - 1) / g.piece);
    int64_t at = 0;
    const auto take = [&](int64_t n) {  // ws is null where only the size is asked for
        char* q = ws ? static_cast<char*>(ws) + at : nullptr;
        at += align16(n * 4);
        return q;
    };
    g.total = reinterpret_cast<int32_t*>(take(1));
    g.perm = reinterpret_cast<int32_t*>(take(n_tokens));
    g.word = reinterpret_cast<int32_t*>(take(n_tokens + 1));
    g.count = reinterpret_cast<int32_t*>(take(static_cast<int64_t>(g.owned) << g.lg));
    g.part = reinterpret_cast<float*>(take(2 * g.pieces * ((dim + 3) & ~int64_t{3})));
    if (sort) {
        g.chunk_tokens = (n_tokens + kMostChunks - 1) / kMostChunks;
        if (g.chunk_tokens < kChunkTokens) g.chunk_tokens = kChunkTokens;
        g.chunk_tokens = (g.chunk_tokens + kSortThreads - 1) / kSortThreads * kSortThreads;
        g.chunks = static_cast<int>((n_tokens + g.chunk_tokens - 1) / g.chunk_tokens);
        g.hist = reinterpret_cast<int32_t*>(take(int64_t{g.chunks} * kBuckets));
        g.start = reinterpret_cast<int32_t*>(take(kBuckets + 1));
        g.bperm = reinterpret_cast<int32_t*>(take(n_tokens));
        g.bword = reinterpret_cast<int32_t*>(take(n_tokens));
    }
    if (bytes) *bytes = at;
    return g;
}

// Exclusive prefix over the lanes of a wave; *sum: the total.
__device__ __forceinline__ int wave_prefix(int c, int lane, int* sum) {
    int incl = c;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(incl, o);
        if (lane >= o) incl += up;
    }
    *sum = __shfl(incl, 63);
    return incl - c;
}

// Between LDS writes of a wave's lanes and reads of them by its other lanes. The
// hardware runs a wave's LDS operations in order; the fences, which cost no
// instruction, keep the compiler to that order as well.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The wave's lanes of `valid` that hold the same key (of `bits` bits) as this one.
__device__ __forceinline__ unsigned long long same_key(unsigned long long valid, int key, int bits) {
    unsigned long long m = valid;
    for (int b = 0; b < bits; ++b) {
        const unsigned long long ones = __ballot((key >> b) & 1);
        m &= (key >> b) & 1 ? ones : ~ones;
    }
    return m;
}

__global__ void __launch_bounds__(kThreads)
    group_kernel(const int32_t* __restrict__ tokens, int64_t n_tokens, int64_t vocab, GradSpace g) {
    constexpr int kTake = 8;  // ids per lane in flight
    __shared__ int cnt[kThreads / 64][kOwned];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t p = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + wave;
    int* own = cnt[wave];
    const int64_t mask = (int64_t{1} << g.lg) - 1;
    const unsigned long long below = (1ull << lane) - 1;
    const auto each = [&](auto&& f) {  // all ids in order, 64 at a time
        for (int64_t b = 0; b < n_tokens; b += 64 * kTake) {
            int32_t t[kTake];
#pragma unroll
            for (int q = 0; q < kTake; ++q) {
                const int64_t n = b + q * 64 + lane;
                t[q] = n < n_tokens ? tokens[n] : -1;
            }
#pragma unroll
            for (int q = 0; q < kTake; ++q) f(b + q * 64 + lane, t[q]);
        }
    };
    for (int j = lane; j < g.owned; j += 64) own[j] = 0;
    wave_sync();
    int less = 0;
    each([&](int64_t, int32_t t) {
        const bool ok = t >= 0 && t < vocab;
        less += __popcll(__ballot(ok && (t & mask) < p));
        if (ok && (t & mask) == p) atomicAdd(&own[t >> g.lg], 1);
    });
    wave_sync();
    int sum = less;  // exclusive prefix over the owned ids, after the ids of the waves before
    for (int j0 = 0; j0 < g.owned; j0 += 64) {
        const int j = j0 + lane;
        const int c = j < g.owned ? own[j] : 0;
        int all;
        const int before = wave_prefix(c, lane, &all);
        if (j < g.owned) {
            g.count[p * g.owned + j] = c;
            own[j] = sum + before;
        }
        sum += all;
    }
    wave_sync();
    if (p == mask && lane == 0) {
        *g.total = sum;
        g.word[sum] = -1;
    }
    each([&](int64_t n, int32_t t) {
        unsigned long long m = __ballot(t >= 0 && t < vocab && (t & mask) == p);
        const int id = t >> g.lg;
        while (m) {
            const int x = __shfl(id, __builtin_ctzll(m));
            const unsigned long long same = __ballot(id == x) & m;
            const int at = own[x];
            wave_sync();
            if ((same >> lane) & 1) {
                const int to = at + __popcll(same & below);
                g.perm[to] = static_cast<int32_t>(n);
                g.word[to] = t;
            }
            if (lane == 0) own[x] = at + __popcll(same);
            wave_sync();
            m &= ~same;
        }
    });
}

// Positions of each residue in each chunk.
__global__ void __launch_bounds__(kSortThreads)
    bucket_count_kernel(const int32_t* __restrict__ tokens, int64_t n_tokens, int64_t vocab, GradSpace g) {
    __shared__ int hist[kBuckets];
    hist[threadIdx.x] = 0;
    __syncthreads();
    const int64_t n0 = blockIdx.x * g.chunk_tokens;
    const int64_t n1 = n0 + g.chunk_tokens < n_tokens ? n0 + g.chunk_tokens : n_tokens;
    for (int64_t n = n0 + threadIdx.x; n < n1; n += kSortThreads) {
        const int32_t t = tokens[n];
        if (t >= 0 && t < vocab) atomicAdd(&hist[t & (kBuckets - 1)], 1);
    }
    __syncthreads();
    g.hist[static_cast<int64_t>(blockIdx.x) * kBuckets + threadIdx.x] = hist[threadIdx.x];
}

// A chunk's positions into their buckets, in order: each wave counts its part
// of the chunk, the counts of all waves and chunks before give each wave its
// places, and equal residues within 64 positions follow one another by lane.
__global__ void __launch_bounds__(kSortThreads)
    bucket_scatter_kernel(const int32_t* __restrict__ tokens, int64_t n_tokens, int64_t vocab, GradSpace g) {
    constexpr int kW = kSortThreads / 64;
    static_assert(kSortThreads == kBuckets, "a thread per bucket");
    __shared__ int place[kW][kBuckets];
    __shared__ int sums[kW];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    for (int w = 0; w < kW; ++w) place[w][t] = 0;
    int before = 0, all = 0;  // positions of bucket t in the chunks before, in all chunks
#pragma unroll 8
    for (int c = 0; c < g.chunks; ++c) {
        const int h = g.hist[static_cast<int64_t>(c) * kBuckets + t];
        before += c < static_cast<int>(blockIdx.x) ? h : 0;
        all += h;
    }
    __syncthreads();
    const int64_t part = g.chunk_tokens / kW;
    const int64_t n0 = blockIdx.x * g.chunk_tokens + wave * part;
    const int64_t n1 = n0 + part < n_tokens ? n0 + part : n_tokens;
    for (int64_t n = n0 + lane; n < n1; n += 64) {
        const int32_t x = tokens[n];
        if (x >= 0 && x < vocab) atomicAdd(&place[wave][x & (kBuckets - 1)], 1);
    }
    int sum;
    int start = wave_prefix(all, lane, &sum);
    if (lane == 0) sums[wave] = sum;
    __syncthreads();
    for (int w = 0; w < wave; ++w) start += sums[w];
    if (blockIdx.x == 0) {
        g.start[t] = start;
        if (t == kBuckets - 1) {
            g.start[kBuckets] = start + all;
            *g.total = start + all;
            g.word[start + all] = -1;
        }
    }
    int at = start + before;
#pragma unroll
    for (int w = 0; w < kW; ++w) {
        const int c = place[w][t];
        place[w][t] = at;
        at += c;
    }
    __syncthreads();
    for (int64_t b = n0; b < n1; b += 64) {
        const int64_t n = b + lane;
        const int32_t x = n < n1 ? tokens[n] : -1;
        const bool ok = x >= 0 && x < vocab;
        const int key = x & (kBuckets - 1);
        const unsigned long long same = same_key(__ballot(ok), key, kLgBuckets);
        const int first = ok ? place[wave][key] : 0;
        wave_sync();
        if (ok) {
            const int to = first + __popcll(same & ((1ull << lane) - 1));
            g.bperm[to] = static_cast<int32_t>(n);
            g.bword[to] = x;
            if (same >> lane == 1) place[wave][key] = to + 1;  // the last of its residue
        }
        wave_sync();
    }
}

// One bucket's positions grouped by id, in order, the same way.
__global__ void __launch_bounds__(kThreads) bucket_group_kernel(GradSpace g, int id_bits) {
    constexpr int kW = kThreads / 64;
    __shared__ int place[kW][kBucketIds];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int bucket = blockIdx.x;
    const int i0 = g.start[bucket], n = g.start[bucket + 1] - i0;
    for (int w = 0; w < kW; ++w)
        for (int j = t; j < g.owned; j += kThreads) place[w][j] = 0;
    __syncthreads();
    const int part = ((n + kW - 1) / kW + 63) & ~63;
    const int a = wave * part < n ? wave * part : n, b = a + part < n ? a + part : n;
#pragma unroll 4
    for (int i = a + lane; i < b; i += 64) atomicAdd(&place[wave][g.bword[i0 + i] >> kLgBuckets], 1);
    __syncthreads();
    if (wave == 0) {
        int sum = i0;
        for (int j0 = 0; j0 < g.owned; j0 += 64) {
            const int j = j0 + lane;
            int c[kW], all = 0, total;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                c[w] = j < g.owned ? place[w][j] : 0;
                all += c[w];
            }
            int at = sum + wave_prefix(all, lane, &total);
            if (j < g.owned) {
                g.count[bucket * g.owned + j] = all;
#pragma unroll
                for (int w = 0; w < kW; ++w) {
                    place[w][j] = at;
                    at += c[w];
                }
            }
            sum += total;
        }
    }
    __syncthreads();
    constexpr int kTake = 4;  // loads in flight
    for (int i1 = a; i1 < b; i1 += 64 * kTake) {
        int x[kTake], n_of[kTake];
#pragma unroll
        for (int q = 0; q < kTake; ++q) {
            const int i = i1 + q * 64 + lane;
            x[q] = i < b ? g.bword[i0 + i] : -1;
            n_of[q] = i < b ? g.bperm[i0 + i] : 0;
        }
#pragma unroll
        for (int q = 0; q < kTake; ++q) {
            const bool ok = x[q] >= 0;
            if (!__ballot(ok)) break;
            const int key = x[q] >> kLgBuckets;
            const unsigned long long same = same_key(__ballot(ok), key, id_bits);
            const int first = ok ? place[wave][key] : 0;
            wave_sync();
            if (ok) {
                const int to = first + __popcll(same & ((1ull << lane) - 1));
                g.perm[to] = n_of[q];
                g.word[to] = x[q];
                if (same >> lane == 1) place[wave][key] = to + 1;
            }
            wave_sync();
        }
    }
}

hipError_t launch_group(const EmbedGradArgs& a, const GradSpace& g, hipStream_t s) {
    if (g.chunks == 0) {
        group_kernel<<<dim3(static_cast<unsigned>((int64_t{1} << g.lg) / (kThreads / 64))), kThreads, 0, s>>>(
            a.tokens, a.n_tokens, a.vocab, g);
        return hipGetLastError();
    }
    const dim3 chunks(static_cast<unsigned>(g.chunks));
    bucket_count_kernel<<<chunks, kSortThreads, 0, s>>>(a.tokens, a.n_tokens, a.vocab, g);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    bucket_scatter_kernel<<<chunks, kSortThreads, 0, s>>>(a.tokens, a.n_tokens, a.vocab, g);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    int id_bits = 0;
    while ((1 << id_bits) < g.owned) ++id_bits;
    bucket_group_kernel<<<dim3(kBuckets), kThreads, 0, s>>>(g, id_bits);
    return hipGetLastError();
}

template <class EG, class EO>
struct GradIn {
    const EG* grad;
    int64_t grad_stride;
    int64_t dim;
    double scale;
    EO* out;
    int64_t out_stride;
    int64_t vocab;
    bool accumulate;
    bool past_cache;
};

// V zeros; non-temporal where table and gradient together do not fit the
// memory-side cache: a bfloat16 table of 262 MB and 134 MB of gradient take 100 us
// so, 109 otherwise, while two micro-batches of 33 MB into a float32 table of 128 MB
// take 96 and 90 us: there the second finds the first's rows in the cache.
constexpr int64_t kCacheBytes = int64_t{256} << 20;
template <class E, int V>
__device__ __forceinline__ void zero(E* p, bool past_cache) {
    if constexpr (V * sizeof(E) == 16) {
        typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
        if (past_cache) {
            __builtin_nontemporal_store(u32x4{0u, 0u, 0u, 0u}, reinterpret_cast<u32x4*>(p));
            return;
        }
    }
    *reinterpret_cast<Vec<E, V>*>(p) = Vec<E, V>{};
}

// A finished sum into its row: scaled in float64, added to what is there when
// accumulating, rounded once.
template <class EG, class EO, int V, class S>
__device__ __forceinline__ void finish(const GradIn<EG, EO>& a, int32_t word, int64_t col, const S (&acc)[V]) {
    Vec<EO, V>* o = reinterpret_cast<Vec<EO, V>*>(a.out + word * a.out_stride + col);
    Vec<EO, V> v{};
    if (a.accumulate) v = *o;
    double s[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        s[e] = static_cast<double>(acc[e]) * a.scale;
        if (a.accumulate) s[e] += static_cast<double>(widen(v.x[e]));
    }
    *o = rounded<EO, V>(s);
}

template <class EG, class EO, int V>
__global__ void __launch_bounds__(kThreads) run_sum_kernel(GradIn<EG, EO> a, GradSpace g, Cover c) {
    const Place at = place_of<V>(c);
    const int piece = __builtin_amdgcn_readfirstlane(static_cast<int>(at.unit));  // one per wave
    const int64_t col = at.col;
    const int lane = threadIdx.x & 63;
    if (piece >= g.pieces) {
        if (a.accumulate || col >= a.dim) return;  // the last workgroup may reach past the pieces
        const int64_t mask = (int64_t{1} << g.lg) - 1;
        const int64_t v0 = (at.unit - g.pieces) * kZeroRows;
        int named[kZeroRows];
#pragma unroll
        for (int q = 0; q < kZeroRows; ++q) {
            const int64_t v = v0 + q;
            named[q] = v < a.vocab ? g.count[(v & mask) * g.owned + (v >> g.lg)] : 1;
        }
#pragma unroll
        for (int q = 0; q < kZeroRows; ++q)
            if (named[q] == 0) zero<EO, V>(a.out + (v0 + q) * a.out_stride + col, a.past_cache);
        return;
    }
    // lane l holds the piece's l-th position and its id; lane n the id behind the piece
    const int total = *g.total;
    const int i0 = piece * g.piece;
    if (i0 >= total) return;
    const int n = i0 + g.piece < total ? g.piece : total - i0;
    const int words = lane <= n ? g.word[i0 + lane] : -1;
    const int perms = lane < n ? g.perm[i0 + lane] : 0;
    bool entered = i0 > 0 && g.word[i0 - 1] == __builtin_amdgcn_readlane(words, 0);
    // lanes past the row's end stay: the others read their positions
    const bool mine = col < a.dim;
    const int64_t wide = (a.dim + 3) & ~int64_t{3};
    const EG* from = a.grad + col;
    float acc[V] = {};
#pragma unroll 1
    for (int i = 0; i < n; i += kAhead) {
        Vec<EG, V> row[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            if (i + q >= n) break;
            const int64_t at_row = __builtin_amdgcn_readlane(perms, i + q) * a.grad_stride;
            row[q] = Vec<EG, V>{};
            if (mine) row[q] = *reinterpret_cast<const Vec<EG, V>*>(from + at_row);
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            if (i + q >= n) break;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += widen(row[q].x[e]);
            const int word = __builtin_amdgcn_readlane(words, i + q);
            const bool ends = __builtin_amdgcn_readlane(words, i + q + 1) != word;
            if (!ends && i + q + 1 < n) continue;
            if (!mine) {
            } else if (ends && !entered) {
                finish<EG, EO, V>(a, word, col, acc);
            } else {
                float* to = g.part + (int64_t{piece} * 2 + (entered ? 0 : 1)) * wide + col;
#pragma unroll
                for (int e = 0; e < V; ++e) to[e] = acc[e];
            }
            entered = false;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = 0.0f;
        }
    }
}

// Runs that leave the piece they begin in: their parts added in float64, each
// of the workgroup's waves a share of them in order, then the shares.
template <class EG, class EO, int V>
__global__ void __launch_bounds__(kThreads) run_join_kernel(GradIn<EG, EO> a, GradSpace g, Cover c) {
    constexpr int kW = kThreads / 64;
    __shared__ double shares[kW][64][V];
    const int64_t block = c.first + blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t piece = block / c.tiles, col = (block % c.tiles * 64 + lane) * V;
    const int64_t i0 = piece * g.piece, i1 = i0 + g.piece;  // below n_tokens: the last piece has no unit
    // read together, judged after: most units end here (6.9 us to 6.6 for 8192 tokens
    // of 1000 columns); past the total the words hold anything and decide nothing
    const int64_t total = *g.total;
    const int32_t word = g.word[i1 - 1], behind = g.word[i1], first = g.word[i0], ahead = i0 > 0 ? g.word[i0 - 1] : -1;
    if (i1 >= total || behind != word) return;   // no run leaves this piece
    if (first == word && ahead == word) return;  // it began before
    const bool in_run = lane < g.piece && g.word[i0 + lane] == word;  // the piece's last positions
    const int64_t begin = i1 - __popcll(__ballot(in_run));
    const int64_t mask = (int64_t{1} << g.lg) - 1;
    const int64_t end = begin + g.count[(word & mask) * g.owned + (word >> g.lg)];
    const int64_t wide = (a.dim + 3) & ~int64_t{3};
    const int64_t last = (end - 1) / g.piece, per = (last - piece + kW) / kW;  // parts `piece` to `last`
    const int64_t q0 = piece + wave * per, q1 = q0 + per < last + 1 ? q0 + per : last + 1;
    double sum[V] = {};
    if (col < a.dim) {
#pragma unroll 8
        for (int64_t q = q0; q < q1; ++q) {
            const float* p = g.part + (q * 2 + (q == piece ? 1 : 0)) * wide + col;
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += p[e];
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) shares[wave][lane][e] = sum[e];
    __syncthreads();
    if (wave != 0 || col >= a.dim) return;
#pragma unroll
    for (int w = 1; w < kW; ++w)
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] += shares[w][lane][e];
    finish<EG, EO, V>(a, word, col, sum);
}

template <class EG, class EO, int V>
hipError_t grad_vec(const EmbedGradArgs& a, const GradSpace& g, hipStream_t s) {
    const GradIn<EG, EO> in{static_cast<const EG*>(a.grad), a.grad_stride, a.dim,   a.scale,
                            static_cast<EO*>(a.out),        a.out_stride,  a.vocab, a.accumulate,
                            a.vocab * a.dim * static_cast<int64_t>(sizeof(EO)) +
                                    a.n_tokens * a.dim * static_cast<int64_t>(sizeof(EG)) > kCacheBytes};
    const int64_t zero_units = a.accumulate ? 0 : (a.vocab + kZeroRows - 1) / kZeroRows;
    const hipError_t e = launch_cover(cover_of<V>(a.dim), g.pieces + zero_units, [&](const Cover& c, dim3 blocks) {
        run_sum_kernel<EG, EO, V><<<blocks, kThreads, 0, s>>>(in, g, c);
    });
    if (e != hipSuccess || g.pieces < 2) return e;
    // a whole workgroup per unit of 64 V columns
    const Cover join{0, kThreads, static_cast<int>((a.dim + 64 * V - 1) / (64 * V))};
    return launch_cover(join, g.pieces - 1, [&](const Cover& c, dim3 blocks) {
        run_join_kernel<EG, EO, V><<<blocks, kThreads, 0, s>>>(in, g, c);
    });
}

template <class EG, class EO>
hipError_t grad_typed(const EmbedGradArgs& a, const GradSpace& g, hipStream_t s) {
    const hipError_t e = launch_group(a, g, s);
    if (e != hipSuccess) return e;
    const auto both = [&](int v) {
        return allows(v, a.dim, a.grad, a.grad_stride, sizeof(EG)) && allows(v, a.dim, a.out, a.out_stride, sizeof(EO));
    };
    constexpr int kMost = widest<EG, EO>();
    if (both(kMost)) return grad_vec<EG, EO, kMost>(a, g, s);
    if (both(2)) return grad_vec<EG, EO, 2>(a, g, s);
    return grad_vec<EG, EO, 1>(a, g, s);
}

template <class ET, class EO>
hipError_t embed_typed(const void* table, int64_t vocab, int64_t dim, int64_t table_stride, const int32_t* tokens,
                       int64_t n_tokens, double scale, void* out, int64_t out_stride, hipStream_t s) {
    const auto run = [&](auto v) {
        constexpr int V = decltype(v)::value;
        const Cover c = cover_of<V>(dim);
        // several rows per thread once that leaves waves enough to fill the chip
        const auto with = [&](auto r) {
            constexpr int R = decltype(r)::value;
            return launch_cover(c, (n_tokens + R - 1) / R, [&](const Cover& part, dim3 blocks) {
                embed_kernel<ET, EO, V, R><<<blocks, kThreads, 0, s>>>(
                    static_cast<const ET*>(table), vocab, dim, table_stride, tokens, n_tokens, scale,
                    static_cast<EO*>(out), out_stride, part);
            });
        };
        if (n_tokens / kRows * c.tiles * (c.lanes / 64) >= kFullWaves) return with(std::integral_constant<int, kRows>{});
        return with(std::integral_constant<int, 1>{});
    };
    const auto both = [&](int v) {
        return allows(v, dim, table, table_stride, sizeof(ET)) && allows(v, dim, out, out_stride, sizeof(EO));
    };
    constexpr int kMost = widest<ET, EO>();
    if (both(kMost)) return run(std::integral_constant<int, kMost>{});
    if (both(2)) return run(std::integral_constant<int, 2>{});
    return run(std::integral_constant<int, 1>{});
}

}  // namespace

hipError_t launch_embed(int table_type, int out_type, const void* table, int64_t vocab, int64_t dim,
                        int64_t table_stride, const int32_t* tokens, int64_t n_tokens, double scale, void* out,
                        int64_t out_stride, hipStream_t s) {
    if (table_type == kBF16)
        return out_type == kBF16
                   ? embed_typed<uint16_t, uint16_t>(table, vocab, dim, table_stride, tokens, n_tokens, scale, out, out_stride, s)
                   : embed_typed<uint16_t, float>(table, vocab, dim, table_stride, tokens, n_tokens, scale, out, out_stride, s);
    return out_type == kBF16
               ? embed_typed<float, uint16_t>(table, vocab, dim, table_stride, tokens, n_tokens, scale, out, out_stride, s)
               : embed_typed<float, float>(table, vocab, dim, table_stride, tokens, n_tokens, scale, out, out_stride, s);
}

int64_t embed_grad_workspace_bytes(int64_t vocab, int64_t dim, int64_t n_tokens) {
    int64_t bytes = 0;
    (void)grad_space(nullptr, vocab, dim, n_tokens, &bytes);
    return bytes;
}

hipError_t launch_embed_grad(const EmbedGradArgs& a, void* workspace, hipStream_t s) {
    const GradSpace g = grad_space(workspace, a.vocab, a.dim, a.n_tokens, nullptr);
    if (a.grad_type == kBF16)
        return a.out_type == kBF16 ? grad_typed<uint16_t, uint16_t>(a, g, s) : grad_typed<uint16_t, float>(a, g, s);
    return a.out_type == kBF16 ? grad_typed<float, uint16_t>(a, g, s) : grad_typed<float, float>(a, g, s);
}

}  // namespace kldk
