// Passing once over a row of logits with one workgroup: 16-byte vectors
// tid, tid + NT, ... of the row's aligned body in groups of U per thread, two
// groups in turn so that one group's loads are in flight while the other is
// used, then the elements before and after the body, one per thread.
#pragma once

#include "device.hpp"
#include "float_order.hpp"
#include "row_stream.hpp"

namespace vsv {

// Elements before the first 16-byte boundary of `row` (at most V).
template <typename E>
__device__ __forceinline__ int row_head(const E* row, int V) {
  const int head = static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / sizeof(E));
  return head > V ? V : head;
}

// Part `part` of P equal shares of a row's 16-byte body, as elements [e0, e1):
// the first part also takes the elements before the body, the last those
// after it.
template <typename E>
__device__ __forceinline__ void row_part(const E* row, int V, int P, int part, int& e0, int& e1) {
  constexpr int N = Elem<E>::kVec;
  const int head = row_head(row, V);
  const int64_t nv = (V - head) / N;
  e0 = part == 0 ? 0 : head + static_cast<int>(nv * part / P) * N;
  e1 = part == P - 1 ? V : head + static_cast<int>(nv * (part + 1) / P) * N;
}

// One 64-bit key in rank order (value desc, index asc): larger is earlier.
__device__ __forceinline__ uint64_t rank_key(float x, int e) {
  return (static_cast<uint64_t>(up_key(x)) << 32) | static_cast<uint32_t>(~e);
}

// Running sum of exp2(x c) kept as s 2^mc, mc an integer (log2 units) at or
// just above the largest x c seen, so every rescale is an exact power of two.
// Terms are summed in float within a group and the groups in float64.
struct ExpSum {
  float mc;   // -FLT_MAX until an x c above it
  double s;   // NaN or +inf if a term was
};

// x c - mc, at most 0 for the x that set mc. One rounding (fma) where mc is
// of an ordinary size; from 2^22 on the rounding of mc itself would show
// against the exact product, so x c is rounded as it was for mc.
constexpr float kFarRef = 4194304.f;
__device__ __forceinline__ float far_arg(float x, float c, float mc) {
#pragma clang fp contract(off)
  const float y = x * c;
  return y - mc;
}
__device__ __forceinline__ float exp_arg(float x, float c, float mc) {
  return fabsf(mc) < kFarRef ? fmaf(x, c, -mc) : far_arg(x, c, mc);
}

// The sum at reference m >= mc.
__device__ __forceinline__ double sum_at(double s, float mc, float m) {
  return ldexp(s, static_cast<int>(fmaxf(mc - m, -2000.f)));
}

__device__ __forceinline__ void raise_ref(ExpSum& p, float xmax, float c) {
  const float y = xmax * c;
  if (y > p.mc && y < FLT_MAX) {
    const float nm = ceilf(y);
    p.s = sum_at(p.s, p.mc, nm);
    p.mc = nm;
  }
}

// Add n terms whose largest x is xmax; f is overwritten.
template <int n>
__device__ __forceinline__ void add_terms(ExpSum& p, float* f, float xmax, float c) {
  raise_ref(p, xmax, c);
  const float mc = p.mc;
  if (fabsf(mc) < kFarRef) {
#pragma unroll
    for (int k = 0; k < n; ++k) f[k] = fast_exp2(fmaf(f[k], c, -mc));
  } else {
#pragma unroll
    for (int k = 0; k < n; ++k) f[k] = fast_exp2(far_arg(f[k], c, mc));
  }
  p.s += static_cast<double>(tree_sum<n>(f));
}
__device__ __forceinline__ void add_term(ExpSum& p, float x, float c) { add_terms<1>(p, &x, x, c); }

// f.template group<kPartial>(w, v, nvec): vectors v, v + NT, .. of one thread
// (kPartial: those at or beyond nvec hold zeros and are to be left out);
// f.one(x, e): element e. `first` sees each thread's first group, w[u] the
// vector tid + u NT where that is below nvec, before any of it is visited;
// every thread calls it, so it may hold barriers.
struct NoFirst {
  __device__ __forceinline__ void operator()(const u32x4*, int) const {}
};
template <typename E, int NT, int U, int kAux, typename F, typename First = NoFirst>
__device__ __forceinline__ void visit_row(const E* __restrict__ row, int V, F& f, First first = First()) {
  constexpr int N = Elem<E>::kVec;
  const int tid = threadIdx.x;
  const int head = row_head(row, V);
  const int nvec = (V - head) / N;
  const int body_end = head + nvec * N;
  constexpr int G = U * NT;
  const int nfull = nvec / G;
  if (nvec > 0) {
    const __amdgpu_buffer_rsrc_t rsrc = vec_rsrc(row + head, nvec);
    u32x4 a[U], b[U];
    load_group_rsrc<NT, U, kAux>(a, rsrc, 0);
    first(a, nvec);
    int g = 0;
    for (; g + 2 <= nfull; g += 2) {
      load_group_rsrc<NT, U, kAux>(b, rsrc, g + 1);
      f.template group<false>(a, g * G + tid, nvec);
      load_group_rsrc<NT, U, kAux>(a, rsrc, g + 2);
      f.template group<false>(b, (g + 1) * G + tid, nvec);
    }
    if (g < nfull) {
      load_group_rsrc<NT, U, kAux>(b, rsrc, g + 1);
      f.template group<false>(a, g * G + tid, nvec);
      f.template group<true>(b, nfull * G + tid, nvec);
    } else {
      f.template group<true>(a, nfull * G + tid, nvec);
    }
  } else {
    u32x4 none[U];
    first(none, 0);
  }
  if (tid < head) f.one(Elem<E>::at(row, tid), tid);
  const int tail = V - body_end;
  if (tid < tail) f.one(Elem<E>::at(row, body_end + tid), body_end + tid);
}

}  // namespace vsv
