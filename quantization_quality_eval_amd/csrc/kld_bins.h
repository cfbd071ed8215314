// Where a logit lies among a row's bins: the arithmetic that drawing tokens places every token
// with, on the GPU, and that tests run on the host as well.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>

namespace kldk {

constexpr int kPerUnit = 4;  // bins per binary unit
constexpr int kBins = 272;   // 64 binary units below the largest weight, and what rounding and bases need

// The base of a slice whose largest logit is m: one to two bins above c m, a whole number, so that
// bases differ by whole numbers. Where c |m| passes 2^45 any other logit lies 2^21 bins or more below
// m, and the base is c m itself.
constexpr double kSteep = 0x1p45;
__host__ __device__ __forceinline__ double base_of(float m, double per) {
    const double at = static_cast<double>(m) * per;
    return fabs(at) < kSteep ? floor(at) + 2.0 : at;
}
// Bins of a logit above the base (at most -1); far below for one that a steep slice drops.
__host__ __device__ __forceinline__ double position(float z, float m, double per, double base) {
    if (fabs(base) < kSteep) return fma(static_cast<double>(z), per, -base);
    return z >= m ? -1.0 : -0x1p60;
}
constexpr double kLowest = -0.5 - kBins;  // positions from here on have a bin (a NaN, 0 times infinity, has none)

// The bin of a position that has one.
__host__ __device__ __forceinline__ int bin_of(double x) { return -1 - static_cast<int>(rint(x)); }
// The bin of any position's whole part f, kBins if it has none: -infinity, what a small temperature puts
// far below and a NaN are brought to there before the conversion, which is defined for int's range only.
__host__ __device__ __forceinline__ int bin_or_none(double f) { return -1 - static_cast<int>(fmax(f, -1.0 - kBins)); }

}  // namespace kldk
