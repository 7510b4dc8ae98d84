// The linear bins of a float32 row's draw: where an element falls, and which
// floats a bin holds. Host and device code.
#pragma once

#include "float_order.hpp"

namespace vsv {

constexpr int kBins = 4096;
constexpr int kReach = 1536;       // bins below the maximum that count (48 T)
constexpr int kBase = kReach + 2;  // about where the first group's maximum lies
// Beyond this |x| per / T bins are too coarse in float64 to trust.
constexpr double kFarBin = 4194304.0;

// Position of an element among the bins: t = fma(x, s, k) with k = 1.5 2^52
// minus an even integer rounds to the bin's number in the low bits of t
// (even, so that a y halfway between two bins goes to the same one on every
// grid).
constexpr double kMagic = 6755399441055744.0;         // 1.5 * 2^52
constexpr uint32_t kMagicHi = 0x43380000u;
struct Grid {
  double s, k, per;   // s = per / T: bins per T
  // The grid that puts `ref` at bin kBase; far: it lies too far out for bins.
  static __host__ __device__ __forceinline__ Grid around(float ref, double T, double per, bool& far) {
    Grid g{per / T, 0.0, per};
    const double y = static_cast<double>(ref) * g.s;
    far = !(__builtin_fabs(y) < kFarBin);
    g.k = kMagic - (far ? 0.0 : 2.0 * __builtin_rint(0.5 * y)) + static_cast<double>(kBase);
    return g;
  }
  __host__ __device__ __forceinline__ double t(float x) const { return __builtin_fma(static_cast<double>(x), s, k); }
  // bin number, or -1 where the element lies outside the bins
  static __host__ __device__ __forceinline__ int slot(double t) {
    const uint64_t b = __builtin_bit_cast(uint64_t, t);
    const uint32_t lo = static_cast<uint32_t>(b);
    return (static_cast<uint32_t>(b >> 32) == kMagicHi && lo < static_cast<uint32_t>(kBins)) ? static_cast<int>(lo) : -1;
  }
  __host__ __device__ __forceinline__ bool reaches(float x, int b) const { return t(x) >= kMagic + static_cast<double>(b); }
  // the least float whose bin is at least b: a step or two from where its
  // border rounds to
  __host__ __device__ __forceinline__ float least_in(int b) const {
    float x = static_cast<float>((static_cast<double>(b) - 0.5 - (k - kMagic)) / s);
    while (reaches(x, b)) x = next_down(x);
    while (!reaches(x, b)) x = next_up(x);
    return x;
  }
};

}  // namespace vsv
