// The k first logits of every row in the order (value desc, index asc), with
// the row's log-sum-exp of x / T: what a distillation loss reads of a teacher.
#include "row_visit.hpp"
#include "rows.hpp"

namespace vsv {

namespace {

constexpr int kTopThreads = 512;
constexpr int kTopUnroll = 2;
constexpr int kTopList = 4096;    // elements a row may keep as candidates

// Order-preserving unsigned key of a float (-0 mapped to +0).
__device__ __forceinline__ uint32_t up_key(float x) {
  const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
// One 64-bit key in rank order: larger is earlier.
__device__ __forceinline__ uint64_t rank_key(float x, int e) {
  return (static_cast<uint64_t>(up_key(x)) << 32) | static_cast<uint32_t>(~e);
}

template <int NT> struct TopLds {
  static constexpr int NW = NT / kWave;
  uint64_t list[kTopList];
  uint32_t hist[256];
  int n, digit, below;
  float mc[NW];
  double s[NW];
  int scan[NW];
};

template <typename E, int NT, int U>
struct SumAll {
  ExpSum p;
  float c;
  template <bool kPartial>
  __device__ __forceinline__ void group(const u32x4* w, int v, int nvec) {
    constexpr int N = Elem<E>::kVec;
    float f[U * N];
    float gmax = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Elem<E>::decode(w[u], f + u * N);
      if (kPartial && v + u * NT >= nvec) {
#pragma unroll
        for (int k = 0; k < N; ++k) f[u * N + k] = -INFINITY;
      }
#pragma unroll
      for (int k = 0; k < N; ++k) gmax = fmaxf(gmax, f[u * N + k]);
    }
    add_terms<U * N>(p, f, gmax, c);
  }
  __device__ __forceinline__ void one(float x, int) { add_term(p, x, c); }
};

// Calls f(key) for every element's rank key.
template <typename E, int NT, int U, typename F>
struct EachKey {
  F& f;
  int head;
  template <bool kPartial>
  __device__ __forceinline__ void group(const u32x4* w, int v, int nvec) {
    constexpr int N = Elem<E>::kVec;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kPartial && v + u * NT >= nvec) continue;
      float x[N];
      Elem<E>::decode(w[u], x);
#pragma unroll
      for (int k = 0; k < N; ++k) f(rank_key(x[k], head + (v + u * NT) * N + k));
    }
  }
  __device__ __forceinline__ void one(float x, int e) { f(rank_key(x, e)); }
};
template <typename E, int NT, int U, typename F>
__device__ __forceinline__ void each_key(const E* row, int V, F&& f) {
  EachKey<E, NT, U, F> v{f, row_head(row, V)};
  visit_row<E, NT, U, kLoadNormal>(row, V, v);
}

// The key of the k-th element in rank order (k >= 1), a byte at a time from
// the highest: the row is read once per byte.
template <typename E, int NT, int U>
__device__ uint64_t nth_key(const E* row, int V, int k, TopLds<NT>& L) {
  uint64_t prefix = 0;
  int left = k;
  for (int shift = 56; shift >= 0; shift -= 8) {
    for (int b = threadIdx.x; b < 256; b += NT) L.hist[b] = 0;
    lds_barrier();
    each_key<E, NT, U>(row, V, [&](uint64_t key) {
      if (shift == 56 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&L.hist[(key >> shift) & 255], 1u);
    });
    lds_barrier();
    if (threadIdx.x == 0) {
      int before = 0, d = 255;
      for (; d > 0 && before + static_cast<int>(L.hist[d]) < left; --d) before += static_cast<int>(L.hist[d]);
      L.digit = d;
      L.below = before;
    }
    lds_barrier();
    prefix |= static_cast<uint64_t>(L.digit) << shift;
    left -= L.below;
    lds_barrier();
  }
  return prefix;
}

template <typename E, int NT, int U>
__global__ __launch_bounds__(NT) void top_kernel(TopArgs a) {
  __shared__ TopLds<NT> L;
  constexpr int NW = NT / kWave;
  const int64_t r = blockIdx.x;
  const E* __restrict__ row = static_cast<const E*>(a.x.p) + r * a.x.ld;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  SumAll<E, NT, U> f;
  f.p = ExpSum{-FLT_MAX, 0.0};
  f.c = a.c;
  visit_row<E, NT, U, kLoadNormal>(row, a.x.V, f);
  const float mw = wave_all(f.p.mc, MaxOp());
  if (lane == 0) L.mc[wave] = mw;
  lds_barrier();
  float mc = L.mc[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) mc = fmaxf(mc, L.mc[w]);
  const double sw = wave_sum_f64(sum_at(f.p.s, f.p.mc, mc));
  if (lane == 0) L.s[wave] = sw;
  lds_barrier();
  double total = 0.0;
#pragma unroll
  for (int w = 0; w < NW; ++w) total += L.s[w];

  const uint64_t last = nth_key<E, NT, U>(row, a.x.V, a.k, L);
  if (tid == 0) L.n = 0;
  lds_barrier();
  each_key<E, NT, U>(row, a.x.V, [&](uint64_t key) {
    if (key >= last) {
      const int at = atomicAdd(&L.n, 1);
      if (at < kTopList) L.list[at] = key;
    }
  });
  lds_barrier();
  const int n = min(L.n, kTopList);
  for (int i = tid; i < n; i += NT) {
    const uint64_t key = L.list[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += L.list[j] > key ? 1 : 0;
    if (rank < a.k) {
      a.values[r * a.k + rank] = key_value(static_cast<uint32_t>(key >> 32));
      a.ids[r * a.k + rank] = static_cast<int>(~static_cast<uint32_t>(key));
    }
  }
  if (tid == 0) {
    const bool ok = total > 0.0 && total < INFINITY;
    if (a.lse) a.lse[r] = static_cast<float>(0.69314718055994530942 * (static_cast<double>(mc) + log2(total)));
    if (!ok && a.error_flag) atomicOr(a.error_flag, VSV_FLAG_LOGITS);
  }
}

template <typename E>
hipError_t top_t(const TopArgs& a, hipStream_t s) {
  top_kernel<E, kTopThreads, kTopUnroll><<<dim3(a.x.N), dim3(kTopThreads), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_top(const TopArgs& a, hipStream_t s) {
  return a.x.dtype == VSV_BF16 ? top_t<uint16_t>(a, s) : top_t<float>(a, s);
}

}  // namespace vsv
