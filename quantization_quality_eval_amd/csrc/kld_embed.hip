// Embedding lookup with scaling, and its gradient by sorted tokens.
//
// Lookup: out[n] = scale * table[t_n]; a negative id gives a zero row, an id
// past the vocabulary a NaN row.
//
// Gradient: dtable[v] = scale * sum over { n : t_n = v } of grad[n]. A sort of
// the positions by their id makes each row's sum one run of the sorted order,
// added up in the order of the positions, so results do not depend on timing:
//   1. group: wave p of P owns the ids v with v mod P = p. It reads every id,
//      counts its own and the ones of the waves before it, and writes its
//      positions grouped by id, each id's in increasing order. No wave waits
//      for another.
//   2. one workgroup per run and column tile adds the run's rows in float32.
//   3. rows of the table that no position names are set to zero.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kld_vocab.h"

namespace kldk {
namespace {

constexpr int kThreads = 256;
constexpr int kOwned = 512;  // ids one wave owns at most

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float(static_cast<unsigned int>(b) << 16); }

// float -> bfloat16 bits, round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint16_t to_bf16(float x) {
    const unsigned int u = __float_as_uint(x);
    if ((u & 0x7fffffffu) > 0x7f800000u) return static_cast<uint16_t>((u >> 16) | 0x40u);
    return static_cast<uint16_t>((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = to_bf16(x); }

template <class ET, class EO>
__global__ void __launch_bounds__(kThreads)
    embed_kernel(const ET* __restrict__ table, int64_t vocab, int64_t dim, int64_t table_stride,
                 const int32_t* __restrict__ tokens, double scale, EO* __restrict__ out, int64_t out_stride) {
    const int64_t n = blockIdx.x;
    const int32_t t = tokens[n];
    EO* o = out + n * out_stride;
    for (int64_t c = threadIdx.x; c < dim; c += kThreads) {
        float x = 0.0f;
        if (t >= vocab) x = NAN;
        else if (t >= 0) x = static_cast<float>(static_cast<double>(widen(table[t * table_stride + c])) * scale);
        put(o + c, x);
    }
}

// ---- gradient ----

struct GradSpace {
    int32_t* total;    // positions with a valid id
    int32_t* perm;     // n_tokens: positions grouped by id
    int32_t* word;     // n_tokens: their ids
    int32_t* count;    // P * owned: positions of id p + P j at [p * owned + j]
    int lg;            // log2 P
    int owned;         // ids per wave
};

int group_lg(int64_t vocab) {
    int lg = 10;
    while ((int64_t{kOwned} << lg) < vocab) ++lg;
    return lg;
}

int64_t align16(int64_t b) { return (b + 15) & ~int64_t{15}; }

GradSpace grad_space(void* ws, int64_t vocab, int64_t n_tokens, int64_t* bytes) {
    GradSpace g{};
    g.lg = group_lg(vocab);
    g.owned = static_cast<int>((vocab + (int64_t{1} << g.lg) - 1) >> g.lg);
    char* p = static_cast<char*>(ws);
    int64_t at = 0;
    const auto take = [&](int64_t n) {
        int32_t* q = reinterpret_cast<int32_t*>(p + at);
        at += align16(n * static_cast<int64_t>(sizeof(int32_t)));
        return q;
    };
    g.total = take(1);
    g.perm = take(n_tokens);
    g.word = take(n_tokens);
    g.count = take(static_cast<int64_t>(g.owned) << g.lg);
    if (bytes) *bytes = at;
    return g;
}

__global__ void __launch_bounds__(kThreads)
    group_kernel(const int32_t* __restrict__ tokens, int64_t n_tokens, int64_t vocab, GradSpace g) {
    __shared__ int cnt[kThreads / 64][kOwned];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t p = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + wave;
    int* own = cnt[wave];
    const int64_t mask = (int64_t{1} << g.lg) - 1;
    const unsigned long long below = (1ull << lane) - 1;
    for (int j = lane; j < g.owned; j += 64) own[j] = 0;
    __builtin_amdgcn_wave_barrier();
    int less = 0;
    for (int64_t b = 0; b < n_tokens; b += 64) {
        const int64_t n = b + lane;
        const int32_t t = n < n_tokens ? tokens[n] : -1;
        const bool ok = t >= 0 && t < vocab;
        less += __popcll(__ballot(ok && (t & mask) < p));
        unsigned long long m = __ballot(ok && (t & mask) == p);
        const int id = t >> g.lg;
        while (m) {
            const int x = __shfl(id, __builtin_ctzll(m));
            const unsigned long long same = __ballot(id == x) & m;
            if (lane == 0) own[x] += __popcll(same);
            m &= ~same;
        }
    }
    __builtin_amdgcn_wave_barrier();
    int sum = less;  // exclusive prefix over the owned ids, after the ids of the waves before
    for (int j0 = 0; j0 < g.owned; j0 += 64) {
        const int j = j0 + lane;
        const int c = j < g.owned ? own[j] : 0;
        int incl = c;
        for (int o = 1; o < 64; o <<= 1) {
            const int up = __shfl_up(incl, o);
            if (lane >= o) incl += up;
        }
        if (j < g.owned) {
            g.count[p * g.owned + j] = c;
            own[j] = sum + incl - c;
        }
        sum += __shfl(incl, 63);
    }
    __builtin_amdgcn_wave_barrier();
    if (p == mask && lane == 0) *g.total = sum;
    for (int64_t b = 0; b < n_tokens; b += 64) {
        const int64_t n = b + lane;
        const int32_t t = n < n_tokens ? tokens[n] : -1;
        const bool ok = t >= 0 && t < vocab;
        unsigned long long m = __ballot(ok && (t & mask) == p);
        const int id = t >> g.lg;
        while (m) {
            const int x = __shfl(id, __builtin_ctzll(m));
            const unsigned long long same = __ballot(id == x) & m;
            const int at = own[x];
            __builtin_amdgcn_wave_barrier();
            if ((same >> lane) & 1) {
                const int to = at + __popcll(same & below);
                g.perm[to] = static_cast<int32_t>(n);
                g.word[to] = t;
            }
            if (lane == 0) own[x] = at + __popcll(same);
            __builtin_amdgcn_wave_barrier();
            m &= ~same;
        }
    }
}

template <class EG, class EO>
__global__ void __launch_bounds__(kThreads)
    run_sum_kernel(const EG* __restrict__ grad, int64_t grad_stride, int64_t dim, double scale, GradSpace g,
                   EO* __restrict__ out, int64_t out_stride, bool accumulate) {
    const int64_t i = blockIdx.x;
    const int64_t total = *g.total;
    if (i >= total) return;
    const int32_t t = g.word[i];
    if (i > 0 && g.word[i - 1] == t) return;
    EO* o = out + t * out_stride;
    for (int64_t c = threadIdx.x; c < dim; c += kThreads) {
        float acc = 0.0f;
        for (int64_t k = i; k < total && g.word[k] == t; ++k) acc += widen(grad[g.perm[k] * grad_stride + c]);
        double x = static_cast<double>(acc) * scale;
        if (accumulate) x += static_cast<double>(widen(o[c]));
        put(o + c, static_cast<float>(x));
    }
}

template <class EO>
__global__ void __launch_bounds__(kThreads)
    zero_rows_kernel(int64_t vocab, int64_t dim, GradSpace g, EO* __restrict__ out, int64_t out_stride) {
    const int64_t mask = (int64_t{1} << g.lg) - 1;
    for (int64_t v = blockIdx.x; v < vocab; v += gridDim.x) {
        if (g.count[(v & mask) * g.owned + (v >> g.lg)] != 0) continue;
        for (int64_t c = threadIdx.x; c < dim; c += kThreads) put(out + v * out_stride + c, 0.0f);
    }
}

template <class EG, class EO>
hipError_t grad_typed(const EmbedGradArgs& a, const GradSpace& g, hipStream_t s) {
    group_kernel<<<dim3(static_cast<unsigned>((int64_t{1} << g.lg) / (kThreads / 64))), kThreads, 0, s>>>(
        a.tokens, a.n_tokens, a.vocab, g);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (!a.accumulate) {
        zero_rows_kernel<EO><<<dim3(static_cast<unsigned>(a.vocab < 16384 ? a.vocab : 16384)), kThreads, 0, s>>>(
            a.vocab, a.dim, g, static_cast<EO*>(a.out), a.out_stride);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.n_tokens > 0)
        run_sum_kernel<EG, EO><<<dim3(static_cast<unsigned>(a.n_tokens)), kThreads, 0, s>>>(
            static_cast<const EG*>(a.grad), a.grad_stride, a.dim, a.scale, g, static_cast<EO*>(a.out), a.out_stride,
            a.accumulate);
    return hipGetLastError();
}

template <class ET, class EO>
hipError_t embed_typed(const void* table, int64_t vocab, int64_t dim, int64_t table_stride, const int32_t* tokens,
                       int64_t n_tokens, double scale, void* out, int64_t out_stride, hipStream_t s) {
    const int64_t per = max_blocks_per_launch(kThreads);
    for (int64_t done = 0; done < n_tokens; done += per) {
        const int64_t n = n_tokens - done < per ? n_tokens - done : per;
        embed_kernel<ET, EO><<<dim3(static_cast<unsigned>(n)), kThreads, 0, s>>>(
            static_cast<const ET*>(table), vocab, dim, table_stride, tokens + done, scale,
            static_cast<EO*>(out) + done * out_stride, out_stride);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
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

int64_t embed_grad_workspace_bytes(int64_t vocab, int64_t, int64_t n_tokens) {
    int64_t bytes = 0;
    (void)grad_space(nullptr, vocab, n_tokens, &bytes);
    return bytes;
}

hipError_t launch_embed_grad(const EmbedGradArgs& a, void* workspace, hipStream_t s) {
    const GradSpace g = grad_space(workspace, a.vocab, a.n_tokens, nullptr);
    if (a.grad_type == kBF16)
        return a.out_type == kBF16 ? grad_typed<uint16_t, uint16_t>(a, g, s) : grad_typed<uint16_t, float>(a, g, s);
    return a.out_type == kBF16 ? grad_typed<float, uint16_t>(a, g, s) : grad_typed<float, float>(a, g, s);
}

}  // namespace kldk
