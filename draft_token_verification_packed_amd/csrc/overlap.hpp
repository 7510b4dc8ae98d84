// Whether two strided sets of byte ranges meet (host code).
#pragma once

#include <stdint.h>

#include <utility>

namespace vsv {

// `count[d]` steps of `stride[d]` bytes (not negative) in each dimension,
// `bytes` at each place.
struct Places {
  const void* base;
  int64_t bytes;
  int64_t stride[3], count[3];
};

// Does the range [s, s + bytes) meet a place of `in`? Its dimensions d .. n - 1
// go from lo[d] to hi[d], the inner ones inside a step of the outer ones and
// `bytes` inside the innermost step: the range meets two steps at most.
inline bool range_meets(int64_t s, int64_t bytes, const Places& in, const int64_t* lo, const int64_t* hi, int d, int n) {
  if (d == n) return s < in.bytes && s + bytes > 0;
  int64_t k = s / in.stride[d];
  if (k * in.stride[d] > s) --k;
  for (int step = 0; step < 2; ++step, ++k)
    if (k >= lo[d] && k <= hi[d] && range_meets(s - k * in.stride[d], bytes, in, lo, hi, d + 1, n)) return true;
  return false;
}

// Do places of `out` (rows and heads of a matrix, as many bytes each as the
// places of `in`, or `in` is one place) and of `in` share memory? Slices of the
// same rows are told apart exactly, in as many steps as they have heads; an
// `in` that overlaps itself counts as all the memory from its first place to
// its last.
inline bool places_meet(const Places& out, Places in) {
  int64_t out_end = out.bytes, in_end = in.bytes;
  for (int d = 0; d < 3; ++d) {
    out_end += (out.count[d] - 1) * out.stride[d];
    in_end += (in.count[d] - 1) * in.stride[d];
  }
  const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(out.base) - reinterpret_cast<uintptr_t>(in.base));
  if (at >= in_end || at + out_end <= 0) return false;
  int n = 0;
  for (int d = 0; d < 3; ++d)
    if (in.count[d] > 1 && in.stride[d] > 0) {
      in.stride[n] = in.stride[d];
      in.count[n++] = in.count[d];
    }
  for (int d = 0; d < n; ++d)
    for (int e = d + 1; e < n; ++e)
      if (in.stride[e] > in.stride[d]) {
        std::swap(in.stride[d], in.stride[e]);
        std::swap(in.count[d], in.count[e]);
      }
  int64_t inner = in.bytes, lo[3], hi[3];
  for (int d = n - 1; d >= 0; --d) {
    if (in.stride[d] < inner) return true;
    inner += (in.count[d] - 1) * in.stride[d];
    lo[d] = 0;
    hi[d] = in.count[d] - 1;
  }
  // a dimension of `out` with the outermost step of `in`: only their difference counts
  int64_t left[3];
  bool taken = n == 0;
  for (int d = 0; d < 3; ++d) {
    left[d] = out.count[d];
    if (taken || left[d] <= 1 || in.stride[0] != out.stride[d]) continue;
    taken = true;
    lo[0] = 1 - left[d];
    left[d] = 1;
  }
  for (int64_t x = 0; x < left[0]; ++x)
    for (int64_t y = 0; y < left[1]; ++y)
      for (int64_t z = 0; z < left[2]; ++z)
        if (range_meets(at + x * out.stride[0] + y * out.stride[1] + z * out.stride[2], out.bytes, in, lo, hi, 0, n)) return true;
  return false;
}

}  // namespace vsv
