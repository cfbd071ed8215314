// Beam selection: the K best continuations of each item over its beams and the
// whole vocabulary.
//
// With s_w the score of beam w and z its logit row, a live beam offers token v
// at s_w + z_v - lse_w, lse_w = log sum exp z over the row's finite entries; a
// finished beam offers itself alone, at s_w. Of one beam's candidates the order
// is that of its logits (equal logits: the lowest id first), so a row's K
// largest logits hold all that can be chosen from it.
//
// Two launches: one workgroup per row forms the row's normaliser (float64) and
// its K largest logits, one workgroup per item merges them.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kld_vocab.h"

namespace kldk {
namespace {

constexpr int kThreads = 256;

struct Cand {
    float z;
    int v;  // -1: none
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float(static_cast<unsigned int>(b) << 16); }

// A logit as the selection sees it: everything that is not finite is -inf.
template <class E>
__device__ __forceinline__ float logit(const E* p) {
    const float z = widen(*p);
    return isfinite(z) ? z : -INFINITY;
}

// Whether candidate (za, va) comes before (zb, vb); none comes last.
__device__ __forceinline__ bool before(float za, int va, float zb, int vb) {
    if (va < 0 || vb < 0) return va >= 0;
    return za > zb || (za == zb && va < vb);
}

template <class E>
__global__ void __launch_bounds__(kThreads)
    beam_rows_kernel(const E* __restrict__ logits, int64_t vocab, int64_t row_stride, int k,
                     const float* __restrict__ scores, const uint8_t* __restrict__ finished, double* __restrict__ lse,
                     Cand* __restrict__ cand) {
    __shared__ float sm[kThreads];
    __shared__ int si[kThreads];
    __shared__ double sd[kThreads];
    const int64_t r = blockIdx.x;
    const int t = threadIdx.x;
    if (!isfinite(scores[r]) || (finished && finished[r])) return;  // its logits offer nothing
    const E* row = logits + r * row_stride;
    float m = -INFINITY;
    for (int64_t i = t; i < vocab; i += kThreads) m = fmaxf(m, logit(row + i));
    sm[t] = m;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        if (t < o) sm[t] = fmaxf(sm[t], sm[t + o]);
        __syncthreads();
    }
    m = sm[0];
    __syncthreads();
    double sum = 0;
    if (m > -INFINITY)
        for (int64_t i = t; i < vocab; i += kThreads) sum += exp(static_cast<double>(logit(row + i)) - m);
    sd[t] = sum;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        if (t < o) sd[t] += sd[t + o];
        __syncthreads();
    }
    if (t == 0) lse[r] = m > -INFINITY ? m + log(sd[0]) : 0.0;
    float pz = INFINITY;
    int pv = -1;
    for (int j = 0; j < k; ++j) {
        float bz = -INFINITY;
        int bv = -1;
        for (int64_t i = t; i < vocab; i += kThreads) {
            const float z = logit(row + i);
            const int v = static_cast<int>(i);
            if (z > -INFINITY && (z < pz || (z == pz && v > pv)) && before(z, v, bz, bv)) bz = z, bv = v;
        }
        sm[t] = bz;
        si[t] = bv;
        __syncthreads();
        for (int o = kThreads / 2; o > 0; o >>= 1) {
            if (t < o && before(sm[t + o], si[t + o], sm[t], si[t])) sm[t] = sm[t + o], si[t] = si[t + o];
            __syncthreads();
        }
        pz = sm[0];
        pv = si[0];
        __syncthreads();
        if (t == 0) cand[r * k + j] = Cand{pz, pv};
        if (pv < 0) {  // the row is used up (uniform: pv is shared)
            for (int q = j + 1 + t; q < k; q += kThreads) cand[r * k + q] = Cand{-INFINITY, -1};
            break;
        }
    }
}

__global__ void __launch_bounds__(64)
    beam_merge_kernel(int w_n, int k, const float* scores, const uint8_t* finished, int eos,
                      const double* __restrict__ lse, const Cand* __restrict__ cand, float* scores_out,
                      int32_t* __restrict__ parents_out, int32_t* __restrict__ tokens_out, uint8_t* finished_out) {
    // lane w holds beam w: its next candidate in order. Read before anything is
    // written: scores_out may be scores, finished_out finished.
    const int64_t item = blockIdx.x;
    const int w = threadIdx.x;
    const int64_t r = item * w_n + w;
    const bool here = w < w_n;
    const float s = here ? scores[r] : -INFINITY;
    const bool alive = here && isfinite(s);
    const bool fin = alive && finished && finished[r];
    const double c = alive && !fin ? lse[r] : 0.0;
    int next = 0;
    for (int j = 0; j < k; ++j) {
        double best = -INFINITY;
        int tok = -1;
        if (fin && next == 0) {
            best = s;
            tok = eos;
        } else if (alive && !fin && next < k) {
            const Cand q = cand[r * k + next];
            if (q.v >= 0) {
                best = s + (q.z - c);
                tok = q.v;
            }
        }
        double b = tok >= 0 ? best : -INFINITY;
        int bw = tok >= 0 ? w : 64;
        for (int o = 1; o < 64; o <<= 1) {
            const double ob = __shfl_xor(b, o);
            const int ow = __shfl_xor(bw, o);
            if (ow < 64 && (bw == 64 || ob > b || (ob == b && ow < bw))) b = ob, bw = ow;
        }
        const int64_t at = item * k + j;
        if (bw == 64) {
            if (w == 0) {
                scores_out[at] = -INFINITY;
                parents_out[at] = -1;
                tokens_out[at] = -1;
                finished_out[at] = 0;
            }
        } else if (w == bw) {
            scores_out[at] = static_cast<float>(b);
            parents_out[at] = w;
            tokens_out[at] = tok;
            finished_out[at] = fin || tok == eos;
            ++next;
        }
    }
}

}  // namespace

int64_t beam_workspace_bytes(int, int64_t, int64_t n_items, int n_beams, int n_select) {
    const int64_t rows = n_items * n_beams;
    return rows * static_cast<int64_t>(sizeof(double)) + rows * n_select * static_cast<int64_t>(sizeof(Cand));
}

hipError_t launch_beam_select(const BeamArgs& a, void* workspace, hipStream_t stream) {
    const int64_t rows = a.n_items * a.n_beams;
    double* lse = static_cast<double*>(workspace);
    Cand* cand = reinterpret_cast<Cand*>(lse + rows);
    if (a.type == kBF16)
        beam_rows_kernel<uint16_t><<<dim3(static_cast<unsigned>(rows)), kThreads, 0, stream>>>(
            static_cast<const uint16_t*>(a.logits), a.vocab, a.row_stride, a.n_select, a.scores, a.finished, lse, cand);
    else
        beam_rows_kernel<float><<<dim3(static_cast<unsigned>(rows)), kThreads, 0, stream>>>(
            static_cast<const float*>(a.logits), a.vocab, a.row_stride, a.n_select, a.scores, a.finished, lse, cand);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    beam_merge_kernel<<<dim3(static_cast<unsigned>(a.n_items)), 64, 0, stream>>>(
        a.n_beams, a.n_select, a.scores, a.finished, a.eos, lse, cand, a.scores_out, a.parents_out, a.tokens_out,
        a.finished_out);
    return hipGetLastError();
}

}  // namespace kldk
