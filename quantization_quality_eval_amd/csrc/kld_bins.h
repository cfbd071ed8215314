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

}  // namespace kldk
