// Where a logit lies among a row's bins: the arithmetic that drawing tokens places every token
// with, on the GPU, and that tests run on the host as well.
//
// With c = 4 log2 e / T a weight is 2^(c z / 4). A logit's place is its own: the whole number f
// nearest to c z and what is left of it, r = c z - f, both exact but for one rounding of r. What is
// counted from, a row's or a slice's largest logit, only shifts f by a whole number; a logit that
// occurs in several slices lies in one bin.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

namespace kldk {

constexpr int kPerUnit = 4;  // bins per binary unit
constexpr int kBins = 272;   // 64 binary units below the largest weight, and what rounding needs

// Added to a number below 2^51 it leaves the nearest whole number (ties to even), whose last 32 bits are
// the sum's: differences of such sums need no conversion.
constexpr double kWhole = 0x1.8p52;
__host__ __device__ __forceinline__ uint32_t last_bits(double x) { return static_cast<uint32_t>(__builtin_bit_cast(uint64_t, x)); }

// c for a temperature above 0. Taken into these ends, c and its products with logits are finite and c is above
// 0: further out the weights are those of the ends, the largest logit's alone or all the same.
struct Heat {
    double heat, per;  // T, c
};
__host__ __device__ __forceinline__ Heat heat_of(double temperature) {
    const double heat = fmin(fmax(temperature, 0x1p-660), 0x1p1000);
    return Heat{heat, kPerUnit * 1.4426950408889634074 / heat};
}

// What the logits of a row or slice are placed by.
struct Frame {
    double per;  // c
    double top;  // kWhole and the whole number nearest to c m, m the largest logit
    double low;  // some more than kBins bins below m; taken for anything lower
    float most;  // m
};
// Where c |m| passes 2^45 any other logit lies 2^21 bins or more below m. There a c at which it lies 2^20 bins
// below serves as well, and c m does not pass what kWhole holds.
constexpr double kSteep = 0x1p45;
__host__ __device__ __forceinline__ Frame frame_of(float m, Heat h) {
    const double most = m;
    if (fabs(most * h.per) >= kSteep) h = Heat{fabs(most) * (kPerUnit * 1.4426950408889634074 / 0x1p44), 0x1p44 / fabs(most)};
    return Frame{h.per, fma(most, h.per, kWhole), most - h.heat * ((kBins + 8) / (kPerUnit * 1.4426950408889634074)), m};
}

// A weight is 2^((r - bin) / 4) of that of the whole number at the top.
struct Spot {
    int bin;   // kBins or more: none
    double r;  // |r| <= 1/2
};
// Of anything up to the largest logit, of -infinity and of a NaN.
__host__ __device__ __forceinline__ Spot spot_of(float z, const Frame& f) {
    const double x = fmax(static_cast<double>(z), f.low), sum = fma(x, f.per, kWhole);
    return Spot{static_cast<int>(last_bits(f.top) - last_bits(sum)), fma(x, f.per, kWhole - sum)};
}
// The bin, -1 above the largest logit, kBins for none.
__host__ __device__ __forceinline__ int bin_of(float z, const Frame& f) {
    if (z > f.most) return -1;
    const int bin = spot_of(z, f).bin;
    return bin < kBins ? bin : kBins;
}

// 2^(r / kPerUnit), |r| <= 1/2, less kOffset, which is a little below the least of them, plus kRaised, whose last
// place is 2^-kUnit: a polynomial of degree 7 (1 + r
// times one that interpolates at Chebyshev's nodes; relative error 1.4e-15 = 2^-49.4), rounded once to whole units,
// half of one 2^-45.87 of the smallest: within 2^-45.7 in all.
constexpr int kUnit = 45;  // mantissas are whole multiples of 2^-kUnit
constexpr double kRaised = 128.0, kOffset = 0.875;
constexpr uint64_t kOffsetUnits = static_cast<uint64_t>(kOffset * (uint64_t{1} << kUnit));
struct Raise {
    static constexpr int kDegree = 7;
    double c[kDegree + 1] = {kRaised + (1.0 - kOffset),
                             0x1.62e42fefa39efp-3,
                             0x1.ebfbdff83132cp-7,
                             0x1.c6b08d704b8a8p-11,
                             0x1.3b2ab6606b75bp-15,
                             0x1.5d87fe190396ap-20,
                             0x1.431c79fede795p-25,
                             0x1.ffe3e4e78d71cp-31};
    __host__ __device__ __forceinline__ double operator()(double r) const {
        double s = c[kDegree];
#pragma unroll
        for (int i = kDegree - 1; i >= 0; --i) s = fma(s, r, c[i]);
        return s;
    }
};
static_assert(52 - kUnit == 7 && kPerUnit == 4, "2^7, of quarters");
// What Raise gives as a mantissa, and as its units.
__host__ __device__ __forceinline__ double mantissa_of(double raised) { return raised - (kRaised - kOffset); }
__host__ __device__ __forceinline__ uint64_t units_of(double raised) {
    return __builtin_bit_cast(uint64_t, raised) - __builtin_bit_cast(uint64_t, kRaised) + kOffsetUnits;
}
// A bin's tokens are summed by adding what Raise gives them, bits and all, to a 64-bit word: below kWordCount the sum
// of the units that their mantissas have above kOffset, from it on their number times an odd one, kRaised's bits
// there, whose inverse gives the number back. Both fit for kWordTokens tokens. (With a subtraction and an addition of
// 1 for each token instead the scan of 1024 x 151936 bfloat16 takes 134 us, not 130.)
constexpr int kWordCount = 53, kWordTokens = 1024;
constexpr uint64_t kOdd = 0x203, kInverse = 171, kMostCount = (uint64_t{1} << (64 - kWordCount)) - 1;
static_assert(__builtin_bit_cast(uint64_t, kRaised) == kOdd << kWordCount && (kOdd * kInverse & kMostCount) == 1, "");
static_assert(kWordTokens <= kMostCount && kWordTokens * (1.0906 - kOffset) < static_cast<double>(1 << (kWordCount - kUnit)), "");
__host__ __device__ __forceinline__ int count_in(uint64_t word) { return static_cast<int>((word >> kWordCount) * kInverse & kMostCount); }
__host__ __device__ __forceinline__ uint64_t units_in(uint64_t word) {
    return (word & ((uint64_t{1} << kWordCount) - 1)) + static_cast<uint64_t>(count_in(word)) * kOffsetUnits;
}
// 2^(f / kPerUnit) for whole f.
__host__ __device__ __forceinline__ double scale_of(int f) {
    const double half = f & 2 ? 0x1.6a09e667f3bcdp+0 : 1.0;
    return ldexp(f & 1 ? half * 0x1.306fe0a31b715p+0 : half, f >> 2);
}

}  // namespace kldk
