// One token per row of logits, drawn with a given random number after
// temperature, top-k, top-p and min-p.
//
// The law is that of sampled verification (sampled_row.hpp): with m the row's
// maximum and w = exp((x - m) / T), tokens ordered by (x desc, index asc), the
// survivors are a prefix of that order (the first top_k; of those the
// shortest prefix whose weight reaches top_p of theirs; of those the tokens
// with (x - m) / T >= ln min_p), and the token is the first whose cumulative
// weight exceeds u times the survivors' total.
//
// Every cut is a comparison of sums over up to the whole row, so the sums
// have to be better than the float sums of a softmax: a relative error of
// 1e-7 decides the wrong token in about one row of a hundred where the law is
// broad. Weights are 64-bit integers, rint(w 2^s) with the largest s whose
// total cannot overflow, so sums are exact in any order and the same on every
// run; a row of 152064 logits has s = 44 and sums within about 1e-11.
#include "row_visit.hpp"
#include "rows.hpp"

namespace vsv {

namespace {

constexpr int kDrawThreads = 512;
constexpr int kDrawUnroll = 2;

__device__ __forceinline__ uint32_t up_key(float x) {
  const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
__device__ __forceinline__ uint64_t rank_key(float x, int e) {
  return (static_cast<uint64_t>(up_key(x)) << 32) | static_cast<uint32_t>(~e);
}

template <int NT> struct DrawLds {
  static constexpr int NW = NT / kWave;
  unsigned long long mass[256];
  uint32_t cnt[256];
  unsigned long long total;
  uint64_t best;
  int digit, bad;
  uint64_t red[NW];
};

template <typename E, int NT, int U, typename F>
struct EachElem {
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
      for (int k = 0; k < N; ++k) f(x[k], head + (v + u * NT) * N + k);
    }
  }
  __device__ __forceinline__ void one(float x, int e) { f(x, e); }
};
template <typename E, int NT, int U, typename F>
__device__ __forceinline__ void each_elem(const E* row, int V, F&& f) {
  EachElem<E, NT, U, F> v{f, row_head(row, V)};
  visit_row<E, NT, U, kLoadNormal>(row, V, v);
}

struct Weigh {
  double m, T, one;   // row maximum, temperature, 2^s
  __device__ __forceinline__ double z(float x) const { return (static_cast<double>(x) - m) / T; }
  __device__ __forceinline__ unsigned long long operator()(float x) const {
    return static_cast<unsigned long long>(rint(exp(z(x)) * one));
  }
};

// The first element in rank order with `count` elements, or a weight of
// `target` (or more than it: strict), through it; `through` receives the
// weight through it. A byte of the rank key at a time, the row read once per
// byte.
template <typename E, int NT, int U>
__device__ uint64_t find_cut(const E* row, int V, const Weigh& w, bool by_count, int count, double target, bool strict,
                             unsigned long long& through, DrawLds<NT>& L) {
  uint64_t prefix = 0;
  unsigned long long mass = 0;
  unsigned long long cnt = 0;
  for (int shift = 56; shift >= 0; shift -= 8) {
    for (int b = threadIdx.x; b < 256; b += NT) {
      L.cnt[b] = 0;
      L.mass[b] = 0;
    }
    lds_barrier();
    each_elem<E, NT, U>(row, V, [&](float x, int e) {
      const uint64_t key = rank_key(x, e);
      if (shift == 56 || (key >> (shift + 8)) == (prefix >> (shift + 8))) {
        const int d = static_cast<int>(key >> shift) & 255;
        atomicAdd(&L.cnt[d], 1u);
        atomicAdd(&L.mass[d], w(x));
      }
    });
    lds_barrier();
    // every thread walks the digits alike; the last one that holds anything
    // is taken if none reaches the target
    int d = 255, hit = -1;
    unsigned long long bm = mass, bc = cnt;
    for (; d >= 0; --d) {
      if (L.cnt[d] == 0) continue;
      hit = d;
      bm = mass;
      bc = cnt;
      const unsigned long long nm = mass + L.mass[d], nc = cnt + L.cnt[d];
      const bool done = by_count ? nc >= static_cast<unsigned long long>(count)
                                 : (strict ? static_cast<double>(nm) > target : static_cast<double>(nm) >= target);
      if (done) break;
      mass = nm;
      cnt = nc;
    }
    through = bm + L.mass[hit < 0 ? 0 : hit];
    mass = bm;
    cnt = bc;
    prefix |= static_cast<uint64_t>(hit < 0 ? 0 : hit) << shift;
    lds_barrier();
  }
  return prefix;
}

// Sum of a 64-bit integer over the workgroup.
template <int NT>
__device__ __forceinline__ unsigned long long block_sum(unsigned long long v, DrawLds<NT>& L) {
  if (threadIdx.x == 0) L.total = 0;
  lds_barrier();
  atomicAdd(&L.total, v);
  lds_barrier();
  const unsigned long long t = L.total;
  lds_barrier();
  return t;
}

template <typename E, int NT, int U>
__global__ __launch_bounds__(NT) void draw_kernel(DrawArgs a) {
  __shared__ DrawLds<NT> L;
  const int64_t r = blockIdx.x;
  const E* __restrict__ row = static_cast<const E*>(a.x.p) + r * a.x.ld;
  const int V = a.x.V;
  const int tid = threadIdx.x;
  float T = a.temperature[r], top_p = a.top_p[r], min_p = a.min_p[r], u = a.uniform[r];
  const int top_k = a.top_k[r];
  int bits = 0;
  if (!(T >= 0.f && T < INFINITY) || !(top_p > 0.f && top_p <= 1.f) || !(min_p >= 0.f && min_p <= 1.f) ||
      !(u >= 0.f && u < 1.f)) {
    bits |= VSV_FLAG_PARAMS;
    T = (T >= 0.f && T < INFINITY) ? T : 0.f;
    top_p = (top_p > 0.f && top_p <= 1.f) ? top_p : 1.f;
    min_p = (min_p >= 0.f && min_p <= 1.f) ? min_p : 0.f;
    u = (u >= 0.f && u < 1.f) ? u : 0.f;
  }
  // the first element of the rank order
  uint64_t best = 0;
  int bad = 0;
  each_elem<E, NT, U>(row, V, [&](float x, int e) {
    bad |= !(x < INFINITY);
    const uint64_t key = rank_key(x, e);
    best = key > best ? key : best;
  });
  best = wave_all(best, MaxOp());
  if ((tid & (kWave - 1)) == 0) L.red[tid / kWave] = best;
  bad = __syncthreads_or(bad);
  for (int w = 0; w < NT / kWave; ++w) best = L.red[w] > best ? L.red[w] : best;
  const float m = key_value(static_cast<uint32_t>(best >> 32));
  if (bad || !(m > -INFINITY)) {
    if (tid == 0) {
      a.token[r] = 0;
      if (a.logprob) a.logprob[r] = 0.f;
      if (a.lse) a.lse[r] = m;
      if (a.error_flag) atomicOr(a.error_flag, bits | VSV_FLAG_LOGITS);
    }
    return;
  }
  const int s = 62 - (32 - __clz(V));
  const Weigh w{static_cast<double>(m), T > 0.f ? static_cast<double>(T) : 1.0, ldexp(1.0, s)};
  unsigned long long mine = 0, above = 0;
  const double zmin = min_p > 0.f ? log(static_cast<double>(min_p)) : -INFINITY;
  each_elem<E, NT, U>(row, V, [&](float x, int) {
    const unsigned long long f = w(x);
    mine += f;
    if (w.z(x) >= zmin) above += f;
  });
  const unsigned long long total = block_sum<NT>(mine, L);
  const unsigned long long kept = block_sum<NT>(above, L);
  const double lse = w.m / w.T + log(static_cast<double>(total) / w.one);
  uint64_t at = best;
  double logprob = 0.0;
  if (T > 0.f) {
    unsigned long long left = total;
    if (top_k > 0 && top_k < V) find_cut<E, NT, U>(row, V, w, true, top_k, 0.0, false, left, L);
    if (top_p < 1.f)
      find_cut<E, NT, U>(row, V, w, false, 0, static_cast<double>(top_p) * static_cast<double>(left), false, left, L);
    left = kept < left ? kept : left;
    unsigned long long through;
    at = find_cut<E, NT, U>(row, V, w, false, 0, static_cast<double>(u) * static_cast<double>(left), true, through, L);
    logprob = w.z(key_value(static_cast<uint32_t>(at >> 32))) - log(static_cast<double>(left) / w.one);
  }
  if (tid == 0) {
    a.token[r] = static_cast<int>(~static_cast<uint32_t>(at));
    if (a.logprob) a.logprob[r] = static_cast<float>(logprob);
    if (a.lse) a.lse[r] = static_cast<float>(lse);
    if (bits && a.error_flag) atomicOr(a.error_flag, bits);
  }
}

template <typename E>
hipError_t draw_t(const DrawArgs& a, hipStream_t s) {
  draw_kernel<E, kDrawThreads, kDrawUnroll><<<dim3(a.x.N), dim3(kDrawThreads), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_draw(const DrawArgs& a, hipStream_t s) {
  return a.x.dtype == VSV_BF16 ? draw_t<uint16_t>(a, s) : draw_t<float>(a, s);
}

}  // namespace vsv
