// Rows rounded to 8-bit integers with a scale each:
//   a = max |x|,  scale = a / 127,  q = 127 x / a to the nearest whole number,
//   ties to even.
//
// q is that of exact arithmetic. 127 x / a is formed in float64 as x (127 / a), off
// by less than 2^-45. A quotient of float32 values near a half-integer either is that
// half-integer or lies at least 2^-35 from it: with x = X 2^i and a = A 2^j of 24-bit
// whole numbers the distance is a whole number over 2 A 2^-s, s = i - j >= -10 where
// |127 x / a| is a quarter or more. Rounded to whole multiples of 2^-36 first, a tie
// becomes exactly one and nothing else does.
//
// A row is read once: each thread keeps its share in registers between the
// maximum and the rounding (kHold units of eight elements; the units of longer rows
// beyond those are read again, out of the cache). Memory bounds it: 32000 x 4096
// bfloat16 (393 MB) 81-87 us, 4.5-4.9 TB/s, a large copy's rate; 8192 x 1001 float32 11.7 us,
// one row of 4096 2.4 us in the kernel. Beside memory the rounding in float64, at half rate,
// takes the most: the product and its first rounding are one fused operation (in two, 30000 x 2048
// took an eighth more).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "kld_answer.h"

namespace kldk {
namespace {

constexpr int kUnit = 8;       // elements per thread and step
constexpr int kThreads = 256;  // per workgroup

struct Unit {
    unsigned int w[8];  // eight float32, or eight bfloat16 in the first four
};

template <class E>
struct In;
template <>
struct In<uint16_t> {
    static __device__ __forceinline__ float get(const Unit& u, int e) {
        const unsigned int w = u.w[e >> 1];
        return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
    }
    static __device__ __forceinline__ void put(Unit& u, int e, uint16_t b) {
        u.w[e >> 1] |= static_cast<unsigned int>(b) << (16 * (e & 1));
    }
};
template <>
struct In<float> {
    static __device__ __forceinline__ float get(const Unit& u, int e) { return __uint_as_float(u.w[e]); }
    static __device__ __forceinline__ void put(Unit& u, int e, float x) { u.w[e] = __float_as_uint(x); }
};

// Elements [at, at + 8) of a row, zero from `dim` on; any alignment.
template <class E>
__device__ __forceinline__ Unit load_unit(const E* row, int64_t at, int64_t dim) {
    Unit u = {};
    if (at + kUnit <= dim) {
        memcpy(u.w, row + at, kUnit * sizeof(E));
    } else if (at < dim) {
        const int64_t last = dim - 1;
#pragma unroll
        for (int e = 0; e < kUnit; ++e) {
            const E x = row[at + e < dim ? at + e : last];
            In<E>::put(u, e, at + e < dim ? x : E{0});
        }
    }
    return u;
}

// Largest bits of |x|: above those of the largest finite value where one is not finite.
template <class E>
__device__ __forceinline__ unsigned int most_of(const Unit& u) {
    unsigned int m = 0;
#pragma unroll
    for (int e = 0; e < kUnit; ++e) m = max(m, __float_as_uint(In<E>::get(u, e)) & 0x7fffffffu);
    return m;
}

template <class E>
__device__ __forceinline__ void store_unit(int8_t* row, int64_t at, int64_t dim, const Unit& u, double per) {
    unsigned int w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < kUnit; ++e) {
        // to whole multiples of 2^-36, then to whole numbers: both by what float64 holds beside a larger value
        const double t = fma(static_cast<double>(In<E>::get(u, e)), per, 0x1.8p16) - 0x1.8p16;
        const unsigned int q = static_cast<unsigned int>(__double2loint(t + 0x1.8p52));
        w[e >> 2] |= (q & 0xffu) << (8 * (e & 3));
    }
    if (at + kUnit <= dim) {
        memcpy(row + at, w, kUnit);
    } else {
#pragma unroll
        for (int e = 0; e < kUnit; ++e)
            if (at + e < dim) row[at + e] = static_cast<int8_t>(w[e >> 2] >> (8 * (e & 3)));
    }
}

// kPer threads per row: a quarter of a wave or a wave (nothing shared with the others of their workgroup) or the
// workgroup.
template <class E, int kPer, int kHold>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const E* __restrict__ x, int64_t dim, int64_t x_stride, int64_t first, int64_t n_rows,
                    int8_t* __restrict__ q, int64_t q_stride, float* __restrict__ scales) {
    static_assert(kPer == 16 || kPer == 64 || kPer == kThreads, "");
    int in_block = threadIdx.x / kPer;
    if (kPer >= 64) in_block = __builtin_amdgcn_readfirstlane(in_block);
    const int64_t r = first + static_cast<int64_t>(blockIdx.x) * (kThreads / kPer) + in_block;
    if (r >= n_rows) return;  // kPer == kThreads: all threads of the workgroup alike
    const int t = threadIdx.x % kPer;
    const E* in = x + r * x_stride;
    Unit held[kHold];
    unsigned int most = 0;
#pragma unroll
    for (int h = 0; h < kHold; ++h) held[h] = load_unit(in, (static_cast<int64_t>(h) * kPer + t) * kUnit, dim);
#pragma unroll
    for (int h = 0; h < kHold; ++h) most = max(most, most_of<E>(held[h]));
    const int64_t behind = static_cast<int64_t>(kHold) * kPer * kUnit;
    for (int64_t at = behind + t * kUnit; at < dim; at += kPer * kUnit) most = max(most, most_of<E>(load_unit(in, at, dim)));
#pragma unroll
    for (int o = std::min(kPer, 64) / 2; o >= 1; o >>= 1)
        most = max(most, static_cast<unsigned int>(__shfl_xor(static_cast<int>(most), o)));
    if constexpr (kPer > 64) {
        __shared__ unsigned int part[kPer / 64];
        if ((t & 63) == 0) part[t >> 6] = most;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPer / 64; ++i) most = max(most, part[i]);
    }
    const bool finite = most < 0x7f800000u;
    const double a = static_cast<double>(__uint_as_float(most));
    // a row of zeros, or one with a NaN or an infinity: zeros
    const double per = finite && most != 0 ? 127.0 / a : 0.0;
    if (t == 0) scales[r] = finite ? static_cast<float>(a / 127.0) : NAN;
    int8_t* out = q + r * q_stride;
    const auto store = [&](int64_t at, Unit u) {
        if (!finite) u = Unit{};
        store_unit<E>(out, at, dim, u, per);
    };
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
        const int64_t at = (static_cast<int64_t>(h) * kPer + t) * kUnit;
        if (at < dim) store(at, held[h]);
    }
    for (int64_t at = behind + t * kUnit; at < dim; at += kPer * kUnit) store(at, load_unit(in, at, dim));
}

template <class E, int kPer, int kHold>
hipError_t launch(const QuantizeArgs& a, hipStream_t stream) {
    constexpr int64_t kRows = kThreads / kPer;
    const int64_t most = max_blocks_per_launch(kThreads);
    for (int64_t first = 0; first < a.n_rows; first += most * kRows) {
        const int64_t blocks = std::min(most, (a.n_rows - first + kRows - 1) / kRows);
        quantize_kernel<E, kPer, kHold><<<dim3(static_cast<unsigned int>(blocks)), dim3(kThreads), 0, stream>>>(
            static_cast<const E*>(a.x), a.dim, a.x_stride, first, a.n_rows, a.q, a.q_stride, a.scales);
    }
    return hipGetLastError();
}

// Threads of a row: as many as it takes to hold it in few units each. Rows of up to 256 take a quarter of
// a wave, the rest of whose lanes would idle (309697 x 116 bfloat16: 47-54 us, with a wave each 129); up to 2048 a
// wave that waits for no other (40000 x 1040: 34-42 us, with the workgroup 58-71; 30000 x 2048: 35-37, 52). Above,
// eight units in a wave leave room for too few waves (32000 x 4096: 140 us, with the workgroup 83; 30000 x 2064: 70,
// 57). Widths between these steps leave lanes idle: 384 moves 3.1 TB/s, 513 2.5, 2064 3.2 and 4112 3.6, where 2048 and
// 4096 move 4.7 to 5.0.
template <class E>
hipError_t launch_type(const QuantizeArgs& a, hipStream_t stream) {
    if (a.dim <= 16 * kUnit) return launch<E, 16, 1>(a, stream);
    if (a.dim <= 16 * kUnit * 2) return launch<E, 16, 2>(a, stream);
    if (a.dim <= 64 * kUnit) return launch<E, 64, 1>(a, stream);
    if (a.dim <= 64 * kUnit * 2) return launch<E, 64, 2>(a, stream);
    if (a.dim <= 64 * kUnit * 3) return launch<E, 64, 3>(a, stream);
    if (a.dim <= 64 * kUnit * 4) return launch<E, 64, 4>(a, stream);
    if (a.dim <= kThreads * kUnit * 2) return launch<E, kThreads, 2>(a, stream);
    return launch<E, kThreads, 4>(a, stream);
}

}  // namespace

hipError_t launch_quantize_int8(const QuantizeArgs& a, hipStream_t stream) {
    return a.type == kF32 ? launch_type<float>(a, stream) : launch_type<uint16_t>(a, stream);
}

}  // namespace kldk
