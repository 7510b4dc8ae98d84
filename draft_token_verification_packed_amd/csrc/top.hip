// The k first logits of every row in the order (value desc, index asc), with
// the row's log-sum-exp of x / T: what a distillation loss reads of a teacher.
//
// One pass over the row. The k-th largest of the threads' own maxima bounds
// the row's k-th largest element from below (k different elements are at
// least that large), and it is close: with 512 threads and k = 64 about 70
// elements of a shuffled row lie above it. So the first group of every thread
// gives a bound, the stream keeps the indices of the elements at or above it
// while it sums the exponentials, and the bound is raised after 4, 16 and 64
// groups; at the end the kept elements above the last bound are ranked
// against each other. Rows whose order defeats this (more kept than the list
// holds, as in a rising row) are read once more with the last bound, and rows
// of too many ties are searched a byte of the rank key at a time.
#include "row_visit.hpp"
#include "rows.hpp"

namespace vsv {

namespace {

// A wave has to see k of the workgroup's maxima: up to kFewTop of them 256
// threads serve, with fewer maxima to search and a list more workgroups can
// hold per CU; beyond it 512. The top 64 of 640 bf16 rows of 152064 take 50
// us with 256 threads against 54, the top 256 of them 73 us with 512 and 2.4
// ms with 256 (the bound is the least maximum there and keeps too much).
// Vectors per group: four, for bf16 rows of 512 threads two (73 us; 77 with
// four, whose registers leave room for fewer workgroups).
constexpr int kFewTop = 64;
constexpr int kTopList = 4096;    // elements a row may keep

constexpr int kTopKeys = 1024;    // of them, those that are ranked

__device__ __forceinline__ void top_lse(const TopArgs& a, int64_t r, float mc, double total) {
  if (a.lse) a.lse[r] = static_cast<float>(0.69314718055994530942 * (static_cast<double>(mc) + log2(total)));
  if (!(total > 0.0 && total < INFINITY) && a.error_flag) atomicOr(a.error_flag, VSV_FLAG_LOGITS);
}

template <int NT> struct TopLds {
  static constexpr int NW = NT / kWave;
  uint32_t list[kTopList];
  uint64_t keys[kTopKeys];
  float most[NT];                 // each thread's maximum
  uint32_t hist[256];
  int n, m, digit, below;
  float mc[NW];
  double s[NW];
};

// A lower bound of the k-th largest of the NT maxima in `most`: their keys'
// leading kBits are searched, by every wave for itself.
template <int NT, int kBits>
__device__ __forceinline__ float kth_bound(const float* most, int k) {
  constexpr int PER = NT / kWave;
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = up_key(most[(threadIdx.x & (kWave - 1)) + i * kWave]);
  // leading bits that all of them share are no question
  uint32_t all = ~0u, any = 0u;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    all &= key[i];
    any |= key[i];
  }
  all = wave_all(all, [](uint32_t x, uint32_t y) { return x & y; });
  any = wave_all(any, [](uint32_t x, uint32_t y) { return x | y; });
  const int same = __clz(all ^ any);   // 32 where all are equal
  uint32_t p = same >= 32 ? any : any & ~(0xFFFFFFFFu >> same);
#pragma unroll 1
  for (int b = 31 - same; b >= 32 - kBits; --b) {
    const uint32_t t = p | 1u << b;
    int n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) n += __popcll(__builtin_amdgcn_ballot_w64(key[i] >= t));
    p = n >= k ? t : p;
  }
  // keys below that of -inf are no values
  return p < 0x00800000u ? -INFINITY : key_value(p);
}

template <typename E, int NT, int U>
struct TopVisit {
  TopLds<NT>& L;
  ExpSum p;
  float c, most, bound;
  int k, head, at;   // at: groups seen

  __device__ __forceinline__ void raise() {
    lds_barrier();
    L.most[threadIdx.x] = most;
    lds_barrier();
    bound = kth_bound<NT, sizeof(E) == 2 ? 16 : 20>(L.most, k);
  }
  __device__ __forceinline__ void keep(uint32_t mask, int v) {
    constexpr int N = Elem<E>::kVec;
    const int c = __popc(mask);
    const int incl = wave_scan_incl(c);
    int to = 0;
    if ((threadIdx.x & (kWave - 1)) == kWave - 1) to = atomicAdd(&L.n, incl);
    to = read_lane(to, kWave - 1) + incl - c;
    while (mask) {
      const int b = __ffs(mask) - 1;
      mask &= mask - 1;
      if (to < kTopList) L.list[to] = static_cast<uint32_t>(head + (v + b / N * NT) * N + b % N);
      ++to;
    }
  }
  template <bool kPartial>
  __device__ __forceinline__ void group(const u32x4* w, int v, int nvec) {
    constexpr int N = Elem<E>::kVec;
    if (at == 4 || at == 16 || at == 64) raise();
    ++at;
    float f[U * N];
    float gmax = -INFINITY;
    uint32_t in = 0;   // the vectors that are there
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Elem<E>::decode(w[u], f + u * N);
      const bool out = kPartial && v + u * NT >= nvec;
      in |= out ? 0u : ((1u << N) - 1) << (u * N);
      if (out) {
#pragma unroll
        for (int q = 0; q < N; ++q) f[u * N + q] = -INFINITY;
      }
#pragma unroll
      for (int q = 0; q < N; ++q) gmax = fmaxf(gmax, f[u * N + q]);
    }
    most = fmaxf(most, gmax);
    if (__builtin_amdgcn_ballot_w64(gmax >= bound) != 0) {
      uint32_t mask = 0;
#pragma unroll
      for (int q = 0; q < U * N; ++q) mask |= f[q] >= bound ? 1u << q : 0u;
      keep(mask & in, v);
    }
    add_terms<U * N>(p, f, gmax, c);
  }
  __device__ __forceinline__ void one(float x, int e) {
    if (x >= bound) {
      const int to = atomicAdd(&L.n, 1);
      if (to < kTopList) L.list[to] = static_cast<uint32_t>(e);
    }
    most = fmaxf(most, x);
    add_term(p, x, c);
  }
};

// Whole rows element by element, for the rare paths.
template <typename E, int NT, typename F>
__device__ __forceinline__ void each_elem(const E* row, int V, F&& f) {
#pragma unroll 1
  for (int e = threadIdx.x; e < V; e += NT) f(Elem<E>::at(row, e), e);
}

// The key of the k-th element in rank order (k >= 1), a byte at a time from
// the highest: the row is read once per byte.
template <typename E, int NT>
__device__ __forceinline__ uint64_t nth_key(const E* row, int V, int k, TopLds<NT>& L) {
  uint64_t prefix = 0;
  int left = k;
#pragma unroll 1
  for (int shift = 56; shift >= 0; shift -= 8) {
    for (int b = threadIdx.x; b < 256; b += NT) L.hist[b] = 0;
    lds_barrier();
    each_elem<E, NT>(row, V, [&](float x, int e) {
      const uint64_t key = rank_key(x, e);
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

// What a part of a row leaves in the scratch: its sum, and behind the heads
// of all parts its first keys in rank order, k words of them (0: no element).
struct TopPart {
  double mc, sum;
};

// A workgroup per row, or (kPart) per part of a row.
template <typename E, int NT, int U, int kWaves, bool kPart>
__global__ __launch_bounds__(NT, kWaves) void top_kernel(TopArgs a) {
  __shared__ TopLds<NT> L;
  constexpr int NW = NT / kWave;
  int64_t r = blockIdx.x;
  int e0 = 0, V = a.x.V;
  if (kPart) {
    r = blockIdx.x / a.parts;
    const E* whole = static_cast<const E*>(a.x.p) + r * a.x.ld;
    const int part = static_cast<int>(blockIdx.x - r * a.parts);
    int e1;
    row_part<E>(whole, V, a.parts, part, e0, e1);
    V = e1 - e0;
  }
  const E* __restrict__ row = static_cast<const E*>(a.x.p) + r * a.x.ld + e0;
  const int k = kPart ? min(a.k, V) : a.k;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  if (tid == 0) L.n = L.m = 0;
  TopVisit<E, NT, U> f{L, ExpSum{-FLT_MAX, 0.0}, a.c, -INFINITY, -INFINITY, k, row_head(row, V), 0};
  visit_row<E, NT, U, kLoadStream>(row, V, f, [&](const u32x4* w, int nvec) {
    float t = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[Elem<E>::kVec];
      if (tid + u * NT < nvec) t = fmaxf(t, vec_max<E>(w[u], x));
    }
    f.most = t;
    f.raise();
  });
  const float mw = wave_all(f.p.mc, MaxOp());
  if (lane == 0) L.mc[wave] = mw;
  f.raise();
  float mc = L.mc[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) mc = fmaxf(mc, L.mc[w]);
  const double sw = wave_sum_f64(sum_at(f.p.s, f.p.mc, mc));
  if (lane == 0) L.s[wave] = sw;

  // ---- the kept elements at or above the last bound
  const int n = L.n;
  auto take = [&](float x, int e) {
    if (x >= f.bound) {
      const int to = atomicAdd(&L.m, 1);
      if (to < kTopKeys) L.keys[to] = rank_key(x, e);
    }
  };
  if (n <= kTopList) {
    for (int i = tid; i < n; i += NT) {
      const int e = static_cast<int>(L.list[i]);
      take(Elem<E>::at(row, e), e);
    }
  } else {
    each_elem<E, NT>(row, V, take);
  }
  lds_barrier();
  int m = L.m;
  if (m > kTopKeys || m < k) {
    // too many ties at the bound (or NaN elements, which no bound keeps)
    const uint64_t last = nth_key<E, NT>(row, V, k, L);
    if (tid == 0) L.m = 0;
    lds_barrier();
    each_elem<E, NT>(row, V, [&](float x, int e) {
      const uint64_t key = rank_key(x, e);
      if (key >= last) {
        const int to = atomicAdd(&L.m, 1);
        if (to < kTopKeys) L.keys[to] = key;
      }
    });
    lds_barrier();
    m = min(L.m, kTopKeys);
  }
  uint64_t* keys = nullptr;
  if (kPart) {
    keys = reinterpret_cast<uint64_t*>(static_cast<TopPart*>(a.part) + static_cast<int64_t>(a.x.N) * a.parts) +
           blockIdx.x * static_cast<int64_t>(a.k);
    for (int i = tid; i < a.k; i += NT)
      if (i >= k) keys[i] = 0;
  }
  for (int i = tid; i < m; i += NT) {
    const uint64_t key = L.keys[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < m; ++j) rank += L.keys[j] > key ? 1 : 0;
    if (rank < k) {
      if (kPart) {
        keys[rank] = key - static_cast<uint32_t>(e0);   // ~(e + e0) = ~e - e0
      } else {
        a.values[r * a.k + rank] = key_value(static_cast<uint32_t>(key >> 32));
        a.ids[r * a.k + rank] = static_cast<int>(~static_cast<uint32_t>(key));
      }
    }
  }
  if (tid == 0) {
    double total = 0.0;
#pragma unroll
    for (int w = 0; w < NW; ++w) total += L.s[w];
    if (kPart) {
      static_cast<TopPart*>(a.part)[blockIdx.x] = TopPart{static_cast<double>(mc), total};
    } else {
      top_lse(a, r, mc, total);
    }
  }
}

// A row's result from its parts': a key's rank is its place in its own part
// and, by bisection, the number of larger keys in each of the others.
constexpr int kMostTopParts = 8;
constexpr int kJoinKeys = 1024;   // keys of all parts of a row
__global__ __launch_bounds__(256) void top_join_kernel(TopArgs a) {
  __shared__ uint64_t key[kJoinKeys];
  const int64_t r = blockIdx.x;
  const int n = a.parts * a.k;
  const TopPart* head = static_cast<const TopPart*>(a.part) + r * a.parts;
  const uint64_t* in = reinterpret_cast<const uint64_t*>(static_cast<const TopPart*>(a.part) +
                                                         static_cast<int64_t>(a.x.N) * a.parts) + r * n;
  const int lane = threadIdx.x & (kWave - 1);
  const TopPart mine = lane < a.parts ? head[lane] : TopPart{-FLT_MAX, 0.0};
  for (int i = threadIdx.x; i < n; i += 256) key[i] = in[i];
  lds_barrier();
  for (int i = threadIdx.x; i < n; i += 256) {
    const uint64_t x = key[i];
    if (x == 0) continue;
    const int own = i / a.k;
    int rank = i - own * a.k;
    for (int p = 0; p < a.parts; ++p) {
      if (p == own) continue;
      int lo = 0, hi = a.k;   // keys [0, lo) of part p are larger
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (key[p * a.k + mid] > x) lo = mid + 1;
        else hi = mid;
      }
      rank += lo;
    }
    if (rank < a.k) {
      a.values[r * a.k + rank] = key_value(static_cast<uint32_t>(x >> 32));
      a.ids[r * a.k + rank] = static_cast<int>(~static_cast<uint32_t>(x));
    }
  }
  if (threadIdx.x < kWave) {
    const float mc = static_cast<float>(mine.mc);
    const float all = wave_all(mc, MaxOp());
    const double total = wave_sum_f64(sum_at(mine.sum, mc, all));
    if (lane == 0) top_lse(a, r, all, total);
  }
}

template <typename E, bool kPart>
void top_rows(const TopArgs& a, hipStream_t s) {
  constexpr bool kTwo = sizeof(E) == 2;
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.x.N) * (kPart ? a.parts : 1)));
  if (a.k <= kFewTop) {
    top_kernel<E, 256, 4, 4, kPart><<<grid, dim3(256), 0, s>>>(a);
  } else {
    top_kernel<E, 512, kTwo ? 2 : 4, kTwo ? 6 : 4, kPart><<<grid, dim3(512), 0, s>>>(a);
  }
}

template <typename E>
hipError_t top_t(const TopArgs& a, hipStream_t s) {
  if (a.parts > 1) {
    top_rows<E, true>(a, s);
    top_join_kernel<<<dim3(a.x.N), dim3(256), 0, s>>>(a);
  } else {
    top_rows<E, false>(a, s);
  }
  return hipGetLastError();
}

}  // namespace

int32_t top_parts(int32_t num_rows, int32_t vocab, int32_t dtype, int32_t k) {
  const int64_t bytes = static_cast<int64_t>(vocab) * (dtype == VSV_BF16 ? 2 : 4);
  if (bytes < 131072) return 1;
  int64_t p = 512 / (num_rows > 0 ? num_rows : 1);
  const int64_t most = bytes / 32768;
  if (p > most) p = most;
  if (p > kMostTopParts) p = kMostTopParts;
  if (p * k > kJoinKeys) p = kJoinKeys / k;
  return p < 2 ? 1 : static_cast<int32_t>(p);
}
size_t top_part_bytes(int32_t k) { return sizeof(TopPart) + sizeof(uint64_t) * static_cast<size_t>(k); }

hipError_t launch_top(const TopArgs& a, hipStream_t s) {
  return a.x.dtype == VSV_BF16 ? top_t<uint16_t>(a, s) : top_t<float>(a, s);
}

}  // namespace vsv
