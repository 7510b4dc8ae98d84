// One token per row of logits, drawn with a given random number after
// temperature, top-k, top-p and min-p.
//
// The law is that of sampled verification (sampled_row.hpp): with m the row's
// maximum and w = exp((x - m) / T), tokens ordered by (x desc, index asc), the
// survivors are a prefix of that order (the first top_k; of those the
// shortest prefix whose weight reaches top_p of theirs; of those the tokens
// with (x - m) / T >= ln min_p), and the token is the first whose cumulative
// weight exceeds u times the survivors' total. T = 0 is the first token.
//
// Every cut is a comparison of sums over up to the whole row, so the sums
// have to be better than the float sums of a softmax: a relative error of
// 1e-7 decides the wrong token in about one row of a hundred where the law is
// broad. So weights are summed as 64-bit integers, exact in any order:
//
// float32: the row is streamed once. With y = per x / T, an element falls into
// bin rint(y), and its weight relative to the bin's centre, exp((y - rint(y))
// / per) by a polynomial in float64, is added to the bin as an integer (2^44
// to one for a vocabulary up to 2^18) by one LDS atomic. With per = 32 (64 for
// flat rows) bins reach from 48 T below the first group's maximum to 80 T above
// it; lower elements weigh less than e^-48 and move no cut. A scan over the
// bins below the maximum turns them into cumulative weights, and each cut and
// the draw are known to within a bin or two (a cut inside a bin leaves the
// total of what follows it known to within that bin). One more pass gathers
// the elements of those bins, and the exact order among them decides. The
// float64 work (18 issue slots an element) and the atomics (16 us a row of
// 152064 and CU, 28 with the counts of a top-k row) bound the stream beside
// the HBM share of 26 us: 128 rows with every filter take 54 us. Per-element
// LDS sums in float would be as many atomics and 1e-7; moments per bin more.
//
// bfloat16: a count per 16-bit code, see CodeLds: 512 rows of 152064 with
// top-p take 58 us, of which the counting is 26 and the search for the drawn
// element, which reads the row again, 13.
//
// Rows neither can serve (too many equal elements at a cut for the list,
// values too large for bins) are searched a byte of the rank key at a time.
#include "draw_grid.hpp"
#include "row_visit.hpp"
#include "rows.hpp"

namespace vsv {

namespace {

constexpr int kDrawThreads = 512;
constexpr int kDrawUnroll = 2;
constexpr int kGatherUnroll = 4;   // the second readings, which do less per vector
constexpr double kPerT = 32.0;     // bins per T
constexpr double kFinePerT = 64.0; // of rows whose bulk spans little
constexpr int kList = 4096;        // elements the gathered list holds
constexpr int kMostParts = 8;
constexpr int kFew = 128;          // lists decided by direct comparison
// Sums hold to about 1e-13 of the row's weight (in the bins a weight's integer
// is off by up to half a unit, 2^-45 of it for a vocabulary up to 2^18 and
// more for a larger one as its units grow; the polynomial by 2e-14), so two that differ by less than this share are taken as equal:
// where weights are equal and a border falls exactly between tokens, it is
// decided as exact sums would.
constexpr double kEqual = 1.0 / 4398046511104.0;   // 2^-42

typedef unsigned long long ull;
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ bool any_lane(bool v) { return __builtin_amdgcn_ballot_w64(v) != 0; }

__device__ __forceinline__ float key_x(uint64_t k) { return key_value(static_cast<uint32_t>(k >> 32)); }

template <int NT> struct DrawLds {
  static constexpr int NW = NT / kWave;
  ull bin[kBins];              // weights; then, as doubles, cumulative weights
  union {
    uint32_t cnt[kBins];       // counts (top-k rows), until the cuts are located
    uint64_t list[kList];      // rank keys of the gathered elements
  } u;
  ull mass[256], mass_lo[256]; // radix search
  uint32_t num[256];
  double w[kFew];
  int at[kFew];
  ull red_u[NW], red_v[NW];
  double red_d[NW];
  float red_f[NW];
  int red_i[NW];
  ull key[2];
  ull kept;
  double cut;
  int n, before, j[8], digit[2];
  uint32_t parts;
  double ptop[kMostParts];
};

// ---------------------------------------------------------------- bins

template <typename E, int NT, int U, bool kCount>
struct BinVisit {
  Grid g;
  ull* bin;
  uint32_t* cnt;
  double c[6];   // the polynomial's coefficients, in weight units
  float top;     // IEEE maximum: a NaN stays
  float cut;     // an element outside the bins, but above this, is missed
  int* missed;

  __device__ __forceinline__ void put(float x) {
    const double t = g.t(x);
    const uint64_t b = __builtin_bit_cast(uint64_t, t);
    const uint32_t lo = static_cast<uint32_t>(b);
    if (static_cast<uint32_t>(b >> 32) == kMagicHi && lo < static_cast<uint32_t>(kBins)) {
      // r in [-1/2, 1/2]; exp(r / per) in weight units, the integer in the low
      // bits of a double between 2^52 and 2^53
      const double r = fma(static_cast<double>(x), g.s, -(t - g.k));
      double h = fma(r, c[5], c[4]);
      h = fma(r, h, c[3]);
      h = fma(r, h, c[2]);
      h = fma(r, h, c[1]);
      h = fma(r, h, c[0]);
      atomicAdd(&bin[lo], __builtin_bit_cast(uint64_t, h) - 0x4330000000000000ull);
      if (kCount) atomicAdd(&cnt[lo], 1u);
    } else if (x > cut) {
      *missed = 1;
    }
  }
  template <bool kPartial>
  __device__ __forceinline__ void group(const u32x4* w, int v, int nvec) {
    constexpr int N = Elem<E>::kVec;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kPartial && v + u * NT >= nvec) continue;
      float f[N];
      top = __builtin_elementwise_maximum(top, vec_max<E, true>(w[u], f));
#pragma unroll
      for (int k = 0; k < N; ++k) put(f[k]);
    }
  }
  __device__ __forceinline__ void one(float x, int) {
    top = __builtin_elementwise_maximum(top, x);
    put(x);
  }
};

// ---------------------------------------------------------------- gathering

// The wanted elements of a range of the row: want(w, mask) sets a bit per
// wanted element of a vector, want.one(x) decides one element, and
// put(position, element) stores it. Positions come from one LDS atomic per
// wave and group.
template <typename E, int NT, int U, typename Want, typename Put>
struct GatherVisit {
  Want& want;
  Put& put;
  int* n;
  int head;
  template <bool kPartial>
  __device__ __forceinline__ void group(const u32x4* w, int v, int nvec) {
    constexpr int N = Elem<E>::kVec;
    uint32_t mask = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t m = want(w[u]);
      mask |= (kPartial && v + u * NT >= nvec) ? 0u : m << (u * N);
    }
    if (any_lane(mask != 0)) {
      const int c = __popc(mask);
      const int incl = wave_scan_incl(c);
      int at = 0;
      if ((threadIdx.x & (kWave - 1)) == kWave - 1) at = atomicAdd(n, incl);
      at = read_lane(at, kWave - 1) + incl - c;
      while (mask) {
        const int b = __ffs(mask) - 1;
        mask &= mask - 1;
        put(at++, head + (v + b / N * NT) * N + b % N);
      }
    }
  }
  __device__ __forceinline__ void one(float x, int e) {
    if (want.one(x)) put(atomicAdd(n, 1), e);
  }
};

// Up to four ranges of bins, as positions downwards from the maximum's.
struct Ranges {
  int n = 0, a[4], b[4];
  __device__ __forceinline__ void add(int x, int y) {
    bool known = x > y;
#pragma unroll
    for (int i = 0; i < 4; ++i) known = known || (i < n && x >= a[i] && y <= b[i]);
    if (known) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i == n) {
        a[i] = x;
        b[i] = y;
      }
    }
    ++n;
  }
};

// Elements within any of up to four closed intervals.
template <typename E> struct WantBetween {
  int n;
  float least;            // the lowest of the bounds
  float low[4], high[4];
  __device__ __forceinline__ bool one(float x) const {
    bool r = __builtin_amdgcn_fmed3f(x, low[0], high[0]) == x;
#pragma unroll
    for (int i = 1; i < 4; ++i)
      if (i < n) r = r || __builtin_amdgcn_fmed3f(x, low[i], high[i]) == x;
    return r;
  }
  __device__ __forceinline__ uint32_t operator()(const u32x4& w) const {
    constexpr int N = Elem<E>::kVec;
    float x[N];
    uint32_t m = 0;
    // most vectors lie wholly below where the cuts are
    if (vec_max<E, true>(w, x) < least) return m;
#pragma unroll
    for (int k = 0; k < N; ++k) m |= __builtin_amdgcn_fmed3f(x[k], low[0], high[0]) == x[k] ? 1u << k : 0u;
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      if (i >= n) break;
#pragma unroll
      for (int k = 0; k < N; ++k) m |= __builtin_amdgcn_fmed3f(x[k], low[i], high[i]) == x[k] ? 1u << k : 0u;
    }
    return m;
  }
};

// bfloat16 elements with one bit pattern.
struct WantCode {
  uint32_t code;   // in both halves
  __device__ __forceinline__ bool one(float x) const { return __float_as_uint(x) >> 16 == (code & 0xFFFFu); }
  __device__ __forceinline__ uint32_t operator()(const u32x4& w) const {
    const uint32_t d[4] = {w.x ^ code, w.y ^ code, w.z ^ code, w.w ^ code};
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) m |= ((d[k] & 0xFFFFu) == 0 ? 1u << (2 * k) : 0u) | (d[k] < 0x10000u ? 2u << (2 * k) : 0u);
    return m;
  }
};

// ---------------------------------------------------------------- radix search

// A weight relative to the row's maximum as two integers, in units of one over
// `one` and 2^-32 of that: sums are exact in any order, and thousands of equal
// elements far below the maximum, whose roundings all point one way, still
// hold to 2^-77 of the total each (with the first word alone 150000 of them
// at z = -15 were off by 2e-9 of it, a hundredth of a token's share).
struct Mass {
  ull hi = 0, lo = 0;
  __device__ __forceinline__ Mass& operator+=(const Mass& o) {
    hi += o.hi;
    lo += o.lo;
    return *this;
  }
};

struct Weigh {
  double m, T, one;   // row maximum, temperature, 2^s
  __device__ __forceinline__ double z(float x) const { return (static_cast<double>(x) - m) / T; }
  __device__ __forceinline__ double exact(float x) const { return exp(z(x)); }
  __device__ __forceinline__ Mass operator()(float x) const {
    const double v = exact(x) * one, whole = floor(v);
    Mass w;
    w.hi = static_cast<ull>(whole);
    w.lo = static_cast<ull>(rint((v - whole) * 4294967296.0));   // below 2^62 for 2^30 of them
    return w;
  }
  __device__ __forceinline__ double value(const Mass& s) const {
    return (static_cast<double>(s.hi) + static_cast<double>(s.lo) * (1.0 / 4294967296.0)) / one;
  }
};

// A cumulative weight reaches t / exceeds t exactly where it is at least /
// more than these.
__device__ __forceinline__ double reach(double t) { return t - t * kEqual; }
__device__ __forceinline__ double exceed(double t) { return t + t * kEqual; }

// Log-probability of a token at z among survivors of weight `left`; a lone
// survivor's is 0, which the sums' last bits would not always say.
__device__ __forceinline__ float log_share(double z, double left) {
  const double p = z - log(left);
  return fabs(p) < kEqual ? 0.f : static_cast<float>(p);
}

// A cut: the first element in rank order with `count` elements through it
// (count > 0), or a cumulative weight of `target` (strict: more than it).
struct Cut {
  int count;
  bool strict;
  double target;
};

// The cut's element among those that each(f) visits with f(x, e), all of them
// behind elements of weight w0 and number n0; `through` receives the weight
// through it. A byte of the rank key at a time, one visit of the elements per
// byte; the last element is taken if none reaches the target.
template <int NT, typename Each>
__device__ __forceinline__ uint64_t find_cut(const Each& each, const Weigh& w, const Cut& c, double w0, int n0,
                                             double& through, DrawLds<NT>& L) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  constexpr int kDigits = 256, DW = kDigits / kWave;
  static_assert(NT >= kDigits, "one digit per thread");
  // bytes that all keys share need no search
  ull all = ~0ull, any = 0ull;
  each([&](float x, int e) {
    const ull key = rank_key(x, e);
    all &= key;
    any |= key;
  });
  all = wave_all(all, [](ull p, ull q) { return p & q; });
  any = wave_all(any, [](ull p, ull q) { return p | q; });
  lds_barrier();
  if (tid == 0) {
    L.mass[0] = ~0ull;
    L.mass[1] = 0ull;
  }
  lds_barrier();
  if (lane == 0) {
    atomicAnd(&L.mass[0], all);
    atomicOr(&L.mass[1], any);
  }
  lds_barrier();
  any = L.mass[1];
  const ull differ = L.mass[0] ^ any;
  uint64_t prefix = 0;
  Mass mass;
  int num = n0;
#pragma unroll 1
  for (int shift = 56; shift >= 0; shift -= 8) {
    if (shift > 0 && (differ >> shift & 255) == 0) {
      prefix |= static_cast<uint64_t>(any >> shift & 255) << shift;
      continue;
    }
    lds_barrier();
    if (tid < kDigits) {
      L.num[tid] = 0;
      L.mass[tid] = 0;
      L.mass_lo[tid] = 0;
    }
    if (tid == 0) {
      L.digit[0] = kDigits;
      L.digit[1] = -1;
    }
    lds_barrier();
    each([&](float x, int e) {
      const uint64_t key = rank_key(x, e);
      if (shift == 56 || (key >> (shift + 8)) == (prefix >> (shift + 8))) {
        const int d = static_cast<int>(key >> shift) & 255;
        atomicAdd(&L.num[d], 1u);
        const Mass m = w(x);
        atomicAdd(&L.mass[d], m.hi);
        atomicAdd(&L.mass_lo[d], m.lo);
      }
    });
    lds_barrier();
    // thread t holds digit 255 - t; the first that reaches the cut is taken
    Mass dm, im;
    int dn = 0, in = 0;
    if (wave < DW) {
      dm.hi = L.mass[kDigits - 1 - tid];
      dm.lo = L.mass_lo[kDigits - 1 - tid];
      dn = static_cast<int>(L.num[kDigits - 1 - tid]);
      im.hi = wave_scan_incl(dm.hi);
      im.lo = wave_scan_incl(dm.lo);
      in = wave_scan_incl(dn);
      if (lane == kWave - 1) {
        L.red_u[wave] = im.hi;
        L.red_v[wave] = im.lo;
        L.red_i[wave] = in;
      }
    }
    lds_barrier();
    if (wave < DW) {
#pragma unroll
      for (int k = 0; k < DW; ++k) {
        im.hi += k < wave ? L.red_u[k] : 0ull;
        im.lo += k < wave ? L.red_v[k] : 0ull;
        in += k < wave ? L.red_i[k] : 0;
      }
      im += mass;
      in += num;
      const double cum = w0 + w.value(im);
      const bool done = dn > 0 && (c.count > 0 ? in >= c.count : (c.strict ? cum > c.target : cum >= c.target));
      if (done) atomicMin(&L.digit[0], tid);
      if (dn > 0) atomicMax(&L.digit[1], tid);
    }
    lds_barrier();
    const int hit = L.digit[0] < kDigits ? L.digit[0] : L.digit[1];
    if (hit < 0) return 0;   // nothing to search (every thread returns)
    if (tid == hit) {
      L.red_u[0] = im.hi;
      L.red_v[0] = im.lo;
      L.red_u[1] = im.hi - dm.hi;
      L.red_v[1] = im.lo - dm.lo;
      L.red_i[0] = in - dn;
      L.red_i[1] = dn;
    }
    lds_barrier();
    Mass to;
    to.hi = L.red_u[0];
    to.lo = L.red_v[0];
    through = w0 + w.value(to);
    mass.hi = L.red_u[1];
    mass.lo = L.red_v[1];
    num = L.red_i[0];
    prefix |= static_cast<uint64_t>(kDigits - 1 - hit) << shift;
    if (shift > 0 && L.red_i[1] == 1) {
      // one element left: its key needs no more digits
      each([&](float x, int e) {
        const uint64_t key = rank_key(x, e);
        if (key >> shift == prefix >> shift) L.key[0] = key;
      });
      lds_barrier();
      return L.key[0];
    }
  }
  lds_barrier();
  return prefix;
}

struct Draw {
  float T, top_p, min_p, u;
  int top_k;
};

template <int NT>
__device__ __forceinline__ Mass block_sum(const Mass& v, DrawLds<NT>& L) {
  const ull hi = wave_all(v.hi, SumOp()), lo = wave_all(v.lo, SumOp());
  lds_barrier();
  if ((threadIdx.x & (kWave - 1)) == 0) {
    L.red_u[threadIdx.x / kWave] = hi;
    L.red_v[threadIdx.x / kWave] = lo;
  }
  lds_barrier();
  Mass t;
#pragma unroll
  for (int w = 0; w < NT / kWave; ++w) {
    t.hi += L.red_u[w];
    t.lo += L.red_v[w];
  }
  return t;
}

// A row's parameters; those outside their ranges are flagged and replaced.
__device__ __forceinline__ Draw load_draw(const DrawArgs& a, int64_t r, int& bits, bool& greedy) {
  Draw d{a.temperature[r], a.top_p[r], a.min_p[r], a.uniform[r], a.top_k[r]};
  if (!(d.T >= 0.f && d.T < INFINITY) || !(d.top_p > 0.f && d.top_p <= 1.f) || !(d.min_p >= 0.f && d.min_p <= 1.f) ||
      !(d.u >= 0.f && d.u < 1.f)) {
    bits |= VSV_FLAG_PARAMS;
    d.T = (d.T >= 0.f && d.T < INFINITY) ? d.T : 0.f;
    d.top_p = (d.top_p > 0.f && d.top_p <= 1.f) ? d.top_p : 1.f;
    d.min_p = (d.min_p >= 0.f && d.min_p <= 1.f) ? d.min_p : 0.f;
    d.u = (d.u >= 0.f && d.u < 1.f) ? d.u : 0.f;
  }
  // the arg-max is the first token of the order at any temperature
  greedy = d.T == 0.f;
  if (greedy) d = Draw{1.f, 1.f, 0.f, 0.f, 0};
  return d;
}
// Weights are integers in units of one over this: V of them stay below 2^63,
// and one below 2^52.
__device__ __forceinline__ double weight_units(int V) { return ldexp(1.0, min(50, 62 - (32 - __clz(V)))); }

// ---------------------------------------------------------------- rows and parts

// The bins of a range of a row: where they lie, its IEEE maximum (finite or
// the bins mean nothing), and whether it lies too far out for bins.
struct Binned {
  Grid g;
  float m;
  bool far;
};

// Elements [0, V) at `row` into L.bin (and L.u.cnt), by the whole workgroup.
// The grid goes by the first group of `sample` (the row, of `sampled`
// elements, that the range belongs to): its maximum, and how far its other
// elements lie below. A row that spans less than 7 T there gets twice the
// bins per T, so that a bin of its bulk holds half as many; a row the finer
// grid then misses something of goes again on the wider one. (Finer still
// would leave no room for a rise of 12 T above the sample's maximum.)
template <typename E, int NT, int U>
__device__ __forceinline__ Binned row_bins(const E* __restrict__ row, int V, const E* __restrict__ sample, int sampled,
                                           double T, double one, bool count, DrawLds<NT>& L) {
  constexpr int NW = NT / kWave;
  constexpr int N = Elem<E>::kVec;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  Grid g{kPerT / T, 0.0, kPerT};
  float m = -INFINITY;
  bool far = false, missed = false, known = false;
  double per = kPerT;
  auto bins = [&](auto& f) {
    f.bin = L.bin;
    f.cnt = L.u.cnt;
    f.top = -INFINITY;
    f.missed = &L.n;
    for (int b = tid; b < kBins; b += NT) L.bin[b] = 0;
    if (count)
      for (int b = tid; b < kBins; b += NT) L.u.cnt[b] = 0;
    if (tid == 0) L.n = 0;
    visit_row<E, NT, U, kLoadNormal>(row, V, f, [&](const u32x4* w, int nvec) {
      float ref = m;
      if (!known) {
        // the sample's vectors, and its elements before and after its body
        const int head = row_head(sample, sampled);
        const int sv = (sampled - head) / N, tail = sampled - head - sv * N;
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = tid + u * NT;
          if (V != sampled && i < sv) v[u] = reinterpret_cast<const u32x4*>(sample + head)[i];
          else v[u] = w[u];
        }
        float hx = tid < head ? Elem<E>::at(sample, tid) : -INFINITY;
        float tx = tid < tail ? Elem<E>::at(sample, sampled - 1 - tid) : -INFINITY;
        float t = fmaxf(hx, tx);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float x[N];
          if (tid + u * NT < sv) t = fmaxf(t, vec_max<E>(v[u], x));
        }
        t = wave_all(t, MaxOp());
        if (lane == 0) L.red_f[wave] = t;
        lds_barrier();
        ref = L.red_f[0];
#pragma unroll
        for (int k = 1; k < NW; ++k) ref = fmaxf(ref, L.red_f[k]);
        const float cut = static_cast<float>(static_cast<double>(ref) - 48.0 * T);
        auto lower = [&](float lo, float x) { return x > cut ? fminf(lo, x) : lo; };
        float lo = lower(lower(ref, hx), tx);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float x[N];
          Elem<E>::decode(v[u], x);
          if (tid + u * NT < sv) {
#pragma unroll
            for (int k = 0; k < N; ++k) lo = lower(lo, x[k]);
          }
        }
        lo = wave_all(lo, MinOp());
        if (lane == 0) L.red_d[wave] = static_cast<double>(lo);
        lds_barrier();
        double least = L.red_d[0];
#pragma unroll
        for (int k = 1; k < NW; ++k) least = fmin(least, L.red_d[k]);
        // half as much again as the sample spans, and 12 T of rise above it,
        // in kReach bins
        const double span = (static_cast<double>(ref) - least) / T * 1.5 + 12.0;
        if (kFinePerT * span <= kReach - 100) per = kFinePerT;
      } else {
        lds_barrier();
      }
      f.cut = per > kPerT ? static_cast<float>(static_cast<double>(ref) - 48.0 * T) : INFINITY;
      f.g = Grid::around(ref, T, per, far);
      f.c[0] = one;
#pragma unroll
      for (int k = 1; k < 6; ++k) f.c[k] = f.c[k - 1] * (1.0 / (per * k));
      f.c[0] += 4503599627370496.0;
    });
    g = f.g;
    const float t = wave_all(f.top, [](float p, float q) { return __builtin_elementwise_maximum(p, q); });
    lds_barrier();
    if (lane == 0) L.red_f[wave] = t;
    lds_barrier();
    m = L.red_f[0];
#pragma unroll
    for (int k = 1; k < NW; ++k) m = __builtin_elementwise_maximum(m, L.red_f[k]);
    // bins further below the maximum than will be looked at have to be empty,
    // unless the grid is the wider, where they weigh nothing
    missed = L.n != 0;
    if (per > kPerT && m > -INFINITY && m < INFINITY && !far) {
      const int top = Grid::slot(g.t(m));
      int held = 0;
      for (int b = tid; b <= top - kReach; b += NT) held |= L.bin[b] != 0;
      held = wave_all(held, MaxOp());
      if (lane == 0 && held) atomicOr(&L.n, 1);
      lds_barrier();
      missed = L.n != 0;
    }
  };
  for (;;) {
    if (count) {
      BinVisit<E, NT, U, true> f;
      bins(f);
    } else {
      BinVisit<E, NT, U, false> f;
      bins(f);
    }
    if (!(m > -INFINITY && m < INFINITY)) break;
    const bool above = !far && g.t(m) >= kMagic + static_cast<double>(kBins);
    if (known && far) break;
    if (!known && above) {
      // from the true maximum
    } else if ((!known && far) || (missed && per > kPerT)) {
      per = kPerT;
    } else {
      break;
    }
    known = true;
    lds_barrier();
  }
  lds_barrier();
  return Binned{g, m, far};
}

// A row cut into parts, one workgroup each: what a part leaves in the scratch.
struct BinPart {
  double m, top, far;       // maximum, its bin's absolute number, 1 if too far out
  double per;               // bins per T
  int low, pad;             // the lowest bin below that holds weight
  ull bin[kReach];          // downwards from the part's own top bin
  uint32_t cnt[kReach];
};
template <int NT>
__device__ __forceinline__ void leave_bins(const Binned& b, bool count, BinPart* out, DrawLds<NT>& L) {
  const bool fine = b.m > -INFINITY && b.m < INFINITY;
  // (a part may lie wholly below the row's bins)
  const int top = fine && !b.far ? Grid::slot(b.g.t(b.m)) : -1;
  int low = 0;
  if (top >= 0) {
    for (int j = threadIdx.x; j < kReach; j += NT) {
      const ull w = j <= top ? L.bin[top - j] : 0ull;
      out->bin[j] = w;
      if (count) out->cnt[j] = j <= top ? L.u.cnt[top - j] : 0u;
      low = w != 0 ? j : low;
    }
    low = wave_all(low, MaxOp());
    if ((threadIdx.x & (kWave - 1)) == 0) L.red_i[threadIdx.x / kWave] = low;
    lds_barrier();
  }
  if (threadIdx.x == 0) {
    if (top >= 0) {
#pragma unroll
      for (int k = 0; k < NT / kWave; ++k) low = max(low, L.red_i[k]);
    }
    out->m = static_cast<double>(b.m);
    out->top = top < 0 ? -INFINITY : static_cast<double>(top) - (b.g.k - kMagic);
    out->far = fine && b.far ? 1.0 : 0.0;
    out->per = b.g.per;
    out->low = low;
  }
}

// The bins of the whole row from its parts'. What other workgroups have just
// written is far away (a microsecond a load), so every load of a step is
// issued before any is used: one lane per part reads the heads, and the
// parts' bins are read for all parts at once.
template <int NT>
__device__ __forceinline__ Binned join_bins(const BinPart* in, int P, double T, bool count, DrawLds<NT>& L) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  Binned b{Grid{kPerT / T, 0.0, kPerT}, -INFINITY, false};
  const BinPart& mine = in[lane < P ? lane : 0];
  const float pm = static_cast<float>(mine.m);
  const bool fine = pm > -INFINITY;
  const double ptop = fine ? mine.top : -INFINITY;   // -inf: the part holds nothing
  const int pfar = fine && mine.far != 0.0 ? 1 : 0;
  if (tid < kMostParts) L.ptop[tid] = tid < P ? ptop : -INFINITY;
  b.m = wave_all(pm, [](float p, float q) { return __builtin_elementwise_maximum(p, q); });
  // parts that went by different grids cannot be added
  const double pper = ptop > -INFINITY ? mine.per : 0.0;
  const double per = wave_all(pper, MaxOp());
  b.far = wave_all(pfar | (ptop > -INFINITY && pper != per ? 1 : 0), MaxOp()) != 0;
  b.g.per = per;
  b.g.s = per / T;
  const double top = wave_all(ptop, MaxOp());
  b.far = b.far || !(top > -INFINITY);
  // The finer grid's bins reach less far down than weight counts. A part makes
  // sure that they hold what lies within reach of its own maximum, which may
  // be far below the row's: such a row goes again as one.
  const int lost = per > kPerT && ptop > -INFINITY && top - ptop + static_cast<double>(mine.low) >= static_cast<double>(kReach);
  b.far = b.far || wave_all(lost, MaxOp()) != 0;
  if (!(b.m > -INFINITY && b.m < INFINITY) || b.far) return b;
  lds_barrier();
  const double even = 2.0 * floor(0.5 * top);
  b.g.k = kMagic - even + static_cast<double>(kBase);
  const int at = kBase + static_cast<int>(top - even);   // the maximum's bin
  int shift[kMostParts];   // bins between the row's top and the part's
#pragma unroll
  for (int p = 0; p < kMostParts; ++p) shift[p] = top - L.ptop[p] < kReach ? static_cast<int>(top - L.ptop[p]) : kReach;
  for (int j = tid; j < kReach; j += NT) {
    ull s[kMostParts];
    uint32_t n[kMostParts];
#pragma unroll
    for (int p = 0; p < kMostParts; ++p) {
      const int q = max(0, j - shift[p]);
      const BinPart& part = in[p < P ? p : 0];
      s[p] = part.bin[q];
      n[p] = count ? part.cnt[q] : 0u;
    }
    ull sum = 0;
    uint32_t num = 0;
#pragma unroll
    for (int p = 0; p < kMostParts; ++p) {
      sum += j >= shift[p] ? s[p] : 0ull;
      num += j >= shift[p] ? n[p] : 0u;
    }
    L.bin[at - j] = sum;
    if (count) L.u.cnt[at - j] = num;
  }
  lds_barrier();
  return b;
}

// Row r by linear bins, by the whole workgroup; kJoin: from its parts' bins.
template <typename E, int NT, int U, bool kJoin>
__device__ __forceinline__ void draw_row(const DrawArgs& a, int64_t r, DrawLds<NT>& L) {
  constexpr int NW = NT / kWave;
  constexpr int PER = kReach / NT;
  static_assert(kReach % NT == 0 && kFew <= NT, "bins per thread");
  const E* __restrict__ row = static_cast<const E*>(a.x.p) + r * a.x.ld;
  const int V = a.x.V;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  int bits = 0;
  bool greedy;
  const Draw d = load_draw(a, r, bits, greedy);
  const bool count = d.top_k > 0 && d.top_k < V;
  const double T = static_cast<double>(d.T);
  const double one = weight_units(V);
  const BinPart* parts = kJoin ? reinterpret_cast<const BinPart*>(a.part) + r * a.parts : nullptr;
  int P = 1;   // parts the gathering goes by
  Binned binned{Grid{0.0, 0.0, 0.0}, -INFINITY, true};
  if constexpr (kJoin) {
    binned = join_bins<NT>(parts, a.parts, T, count, L);
    P = a.parts;
  }
  if (!kJoin || binned.far) {
    // (parts that went by different grids: the row again, as one)
    lds_barrier();
    binned = row_bins<E, NT, U>(row, V, row, V, T, one, count, L);
    P = 1;
  }
  const Grid g = binned.g;
  const float m = binned.m;
  const bool far = binned.far;
  if (!(m > -INFINITY && m < INFINITY)) {
    if (tid == 0) {
      a.token[r] = 0;
      if (a.logprob) a.logprob[r] = 0.f;
      if (a.lse) a.lse[r] = m;
      if (a.error_flag) atomicOr(a.error_flag, bits | VSV_FLAG_LOGITS);
    }
    return;
  }
  const Weigh w{static_cast<double>(m), T, one};
  const double top_p = static_cast<double>(d.top_p), u = static_cast<double>(d.u);
  const double zmin = d.min_p > 0.f ? log(static_cast<double>(d.min_p)) : -INFINITY;
  uint64_t key = 0;                  // rank key of the token
  double total = 0.0, left = 0.0;    // weight of the row, of the survivors

  // what the search below goes by: the gathered list (bins), or the row
  int n = V, top_k = 0, jk = -1, jm = -1, top = 0;
  const double* cum = nullptr;
  double through[PER];
  int seen[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    through[k] = 0.0;
    seen[k] = 0;
  }
  // weight through the j-th bin downwards
  auto upto = [&](int j) { return j < 0 ? 0.0 : cum[-j]; };
  auto bin_of = [&](float x) {
    const int b = Grid::slot(g.t(x));
    return b < 0 ? -1 : top - b;
  };
  // the first bin whose k-th slot of its thread satisfies pred, into L.j[q]
  // (the last one if none does)
  auto first_bin = [&](int q, auto pred) {
    int mine = kReach;
#pragma unroll
    for (int k = PER - 1; k >= 0; --k) mine = pred(k) ? tid * PER + k : mine;
    mine = wave_all(mine, MinOp());
    if (lane == 0 && mine < kReach) atomicMin(&L.j[q], mine);
  };
  auto at_least = [&](int q, double t) { first_bin(q, [&](int k) { return through[k] >= t; }); };
  auto more_than = [&](int q, double t) { first_bin(q, [&](int k) { return through[k] > t; }); };

  // the elements of the ranges' bins into the list
  auto collect = [&](const Ranges& rs) {
    WantBetween<E> want;
    want.n = rs.n;
    want.least = INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      want.low[i] = INFINITY;
      want.high[i] = -INFINITY;
      if (i < rs.n) {
        want.low[i] = g.least_in(top - rs.b[i]);
        want.high[i] = rs.a[i] > 0 ? next_down(g.least_in(top - rs.a[i] + 1)) : m;
        // (bins narrower than the floats may hold none)
        if (want.high[i] < want.low[i]) want.low[i] = want.high[i] = INFINITY;
        want.least = fminf(want.least, want.low[i]);
      }
    }
    int e0 = 0, e1 = V;
    auto put = [&](int at, int e) {
      if (at < kList) L.u.list[at] = static_cast<uint64_t>(e0 + e);
    };
    if (kJoin && P > 1) {
      // only the parts that hold something in those bins
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q >= rs.n) break;
        for (int i = tid; i < P * (rs.b[q] - rs.a[q] + 1); i += NT) {
          const int p = i % P, j = rs.a[q] + i / P;
          const double at = static_cast<double>(j) - (static_cast<double>(top) - (g.k - kMagic) - L.ptop[p]);
          if (at >= 0.0 && parts[p].bin[static_cast<int>(at)] != 0) atomicOr(&L.parts, 1u << p);
        }
      }
      lds_barrier();
    }
    const uint32_t take = P > 1 ? L.parts : 1u;
#pragma unroll 1
    for (int p = 0; p < P; ++p) {
      if (!(take >> p & 1u)) continue;
      if (P > 1) row_part<E>(row, V, P, p, e0, e1);
      GatherVisit<E, NT, kGatherUnroll, WantBetween<E>, decltype(put)> v{want, put, &L.n, row_head(row + e0, e1 - e0)};
      visit_row<E, NT, kGatherUnroll, kLoadNormal>(row + e0, e1 - e0, v);
    }
    // the values are read again at the end, all at once: a load per element
    // as it is found would hold its wave up each time
    lds_barrier();
    const int got = min(L.n, kList);
    for (int i = tid; i < got; i += NT) {
      const int e = static_cast<int>(L.u.list[i]);
      L.u.list[i] = rank_key(Elem<E>::at(row, e), e);
    }
  };

  bool two = false;   // the cuts' bins first, the draw's after them
  if (!far) {
    // ---- cumulative weights, downwards from the maximum's bin
    top = Grid::slot(g.t(m));
    const double mpos = fma(static_cast<double>(m), g.s, g.k - kMagic);   // the maximum among the bins' numbers
    double sum = 0.0;
    int num = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int b = top - (tid * PER + k);
      sum += static_cast<double>(L.bin[b]) / one * exp((static_cast<double>(b) - mpos) / g.per);
      through[k] = sum;
      num += count ? static_cast<int>(L.u.cnt[b]) : 0;
      seen[k] = num;
    }
    double wb = wave_scan_incl(sum);
    int nb = wave_scan_incl(num);
    if (lane == kWave - 1) {
      L.red_d[wave] = wb;
      L.red_i[wave] = nb;
    }
    if (tid < 8) L.j[tid] = kReach - 1;
    if (tid == 0) {
      L.n = 0;
      L.before = 0;
      L.parts = 0;
    }
    lds_barrier();
    wb -= sum;
    nb -= num;
    int number = 0;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      wb += k < wave ? L.red_d[k] : 0.0;
      nb += k < wave ? L.red_i[k] : 0;
      total += L.red_d[k];
      number += L.red_i[k];
    }
    double* out = reinterpret_cast<double*>(L.bin) + top;
    cum = out;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      through[k] += wb;
      seen[k] += nb;
      out[-(tid * PER + k)] = through[k];
    }

    // ---- where each cut lies: a range of bins, and bounds of the weight
    // it leaves
    top_k = (count && number >= d.top_k) ? d.top_k : 0;
    lds_barrier();
    double lo = total, hi = total;
    if (top_k) {
      first_bin(0, [&](int k) { return seen[k] >= top_k; });
      lds_barrier();
      jk = L.j[0];
      lo = upto(jk - 1);
      hi = upto(jk);
#pragma unroll
      for (int k = 0; k < PER; ++k)
        if (tid * PER + k == jk) L.before = k ? seen[k - 1] : nb;
    }
    int p0 = kReach, p1 = -1;
    if (d.top_p < 1.f) {
      at_least(1, reach(top_p * lo));
      at_least(2, reach(top_p * hi));
      lds_barrier();
      p0 = L.j[1];
      p1 = L.j[2];
      lo = fmin(lo, upto(p0 - 1));
      hi = fmin(hi, upto(p1));
    }
    if (d.min_p > 0.f) {
      const double jz = static_cast<double>(top) - rint(mpos + g.per * zmin);
      if (jz < static_cast<double>(kReach)) {
        jm = jz > 0.0 ? static_cast<int>(jz) : 0;
        lo = fmin(lo, upto(jm - 1));
        hi = fmin(hi, upto(jm));
      }
    }
    more_than(3, exceed(u * lo));
    more_than(4, exceed(u * hi));
    lds_barrier();
    const int d0 = L.j[3], d1 = L.j[4];
    auto is_cut = [&](int j) { return j == jk || j == jm || (j >= p0 && j <= p1); };
    auto is_draw = [&](int j) { return j >= d0 && j <= d1; };
    // how many elements they hold, from their weights
    double held = 0.0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int j = tid * PER + k;
      if (is_cut(j) || is_draw(j))
        held += (through[k] - (k ? through[k > 0 ? k - 1 : 0] : wb)) * exp((mpos - static_cast<double>(top - j)) / g.per);
    }
    held = wave_all(held, SumOp());
    if (lane == 0) L.red_d[wave] = held;
    lds_barrier();
    held = 0.0;
#pragma unroll
    for (int k = 0; k < NW; ++k) held += L.red_d[k];
    two = held > static_cast<double>(kList - kList / 16);
    Ranges rs;
    if (jk >= 0) rs.add(jk, jk);
    rs.add(p0, p1);
    if (jm >= 0) rs.add(jm, jm);
    if (!two) rs.add(d0, d1);

    // ---- the elements of those bins
    if (rs.n) collect(rs);
    lds_barrier();
    n = L.n;
    left = total;
    if (n <= kFew && !two) {
      // ---- few: each element's cumulative weight from the others of its bin
      uint64_t mine = 0;
      int j = -1;
      if (tid < n) {
        mine = L.u.list[tid];
        j = bin_of(key_x(mine));
        L.w[tid] = w.exact(key_x(mine));
        L.at[tid] = j;
      }
      if (tid < 2) L.key[tid] = 0;
      if (tid == 0) L.kept = __builtin_bit_cast(ull, upto(jm - 1));
      lds_barrier();
      double c = 0.0;
      if (tid < n) {
        int before = 0;
        for (int i = 0; i < n; ++i) {
          const bool in = L.at[i] == j && L.u.list[i] >= mine;
          c += in ? L.w[i] : 0.0;
          before += in ? 1 : 0;
        }
        c += upto(j - 1);
        if (j == jk && L.before + before == top_k) L.cut = c;
      }
      if (top_k) {
        lds_barrier();
        left = L.cut;
      }
      // the first in rank order, whatever rounding does to light tokens' sums
      if (tid < n) {
        if (d.top_p < 1.f && c >= reach(top_p * left)) atomicMax(&L.key[0], static_cast<ull>(mine));
        // (positive doubles order like their bits)
        if (jm >= 0 && w.z(key_x(mine)) >= zmin) atomicMax(&L.kept, __builtin_bit_cast(ull, c));
      }
      lds_barrier();
      if (d.top_p < 1.f) {
        if (mine != 0 && mine == L.key[0]) L.cut = c;
        lds_barrier();
        if (L.key[0] != 0) left = fmin(left, L.cut);
      }
      if (jm >= 0) left = fmin(left, __builtin_bit_cast(double, L.kept));
      if (tid < n && c > exceed(u * left)) atomicMax(&L.key[1], static_cast<ull>(mine));
      lds_barrier();
      key = L.key[1];
    }
  }
  if (key == 0) {
    // ---- more: each cut by a radix search, over its own bin's elements or,
    // where the bins hold too many or cannot place them (or rounding hides a
    // border from the list), over the row
    bool list = !far && (n > kFew || two) && n <= kList;
    int j = -1;
    auto each = [&](auto&& f) {
      if (list) {
        for (int i = tid; i < n; i += NT) {
          const uint64_t k = L.u.list[i];
          if (bin_of(key_x(k)) == j) f(key_x(k), static_cast<int>(~static_cast<uint32_t>(k)));
        }
      } else {
        for (int e = tid; e < V; e += NT) f(Elem<E>::at(row, e), e);
      }
    };
#pragma unroll 1
    for (;; list = false) {
      if (!list) {
        top_k = count ? d.top_k : 0;
        Mass mine;
        each([&](float x, int) { mine += w(x); });
        total = w.value(block_sum<NT>(mine, L));
        left = total;
      }
#pragma unroll 1
      for (int c = 0; c < 3; ++c) {
        if (c == 2 && d.min_p > 0.f && (!list || jm >= 0)) {
          j = jm;
          Mass kept;
          each([&](float x, int) {
            if (w.z(x) >= zmin) kept += w(x);
          });
          left = fmin(left, (list ? upto(jm - 1) : 0.0) + w.value(block_sum<NT>(kept, L)));
        }
        if ((c == 0 && !top_k) || (c == 1 && !(d.top_p < 1.f))) continue;
        const double t = c == 1 ? reach(top_p * left) : exceed(u * left);
        if (list) {
          if (c == 0) {
            j = jk;
          } else {
            if (c == 1) at_least(5, t);
            else more_than(6, t);
            lds_barrier();
            j = L.j[4 + c];
          }
          if (c == 2 && two) {
            if (tid == 0) {
              L.n = 0;
              L.parts = 0;
            }
            lds_barrier();
            Ranges rs;
            rs.add(j, j);
            collect(rs);
            lds_barrier();
            n = L.n;
            if (n > kList) {
              key = 0;
              break;
            }
          }
        }
        double to;
        key = find_cut<NT>(each, w, Cut{c == 0 ? top_k : 0, c == 2, t}, list ? upto(j - 1) : 0.0, list ? L.before : 0, to, L);
        if (c < 2) left = to;
      }
      if (key != 0 || !list) break;
    }
  }
  if (tid == 0) {
    const float x = key_x(key);
    a.token[r] = static_cast<int>(~static_cast<uint32_t>(key));
    if (a.logprob) a.logprob[r] = greedy ? 0.f : log_share(w.z(x), left);
    if (a.lse) a.lse[r] = static_cast<float>(w.m / T + log(total));
    if (bits && a.error_flag) atomicOr(a.error_flag, bits);
  }
}

// ---------------------------------------------------------------- bfloat16 codes

// A bfloat16 row holds few distinct values: a count per 16-bit code says all
// of its weights exactly, so its stream needs no exponentials, and a cut
// inside a code is arithmetic. The table covers 2^-16 <= |x| < 2^8, 24
// binades of 128 codes of either sign; smaller |x| (zeros among them) are one
// cell between the signs, with their weight, and rows with other values that
// matter are left to draw_row.
constexpr uint32_t kCodeLow = 0x3780u;     // 2^-16
constexpr int kCodes = 0xC00;              // codes of a sign
constexpr int kTab = 8192;                 // sign << 12 | code - kCodeLow
constexpr int kCells = 2 * kCodes + 1;     // in rank order: positive, tiny, negative
constexpr int kCodeList = 4096;
constexpr double kTinyT = 1.0 / 1024.0;    // below this T the tiny cell is no point

template <int NT> struct CodeLds {
  static constexpr int NW = NT / kWave;
  uint32_t tab[kTab];
  uint32_t list[kCodeList];
  uint32_t hist[256];
  ull tiny;          // weight of the tiny cell relative to x = 0
  uint32_t tiny_n;
  int bad;           // a value of 2^8 or more, or a NaN
  uint32_t low;      // key of the largest finite value at or below -2^8
  int n, j[6];
  double red_d[NW];
  int red_i[NW];
  double cut_w;
  int cut_j, cut_r, cut_n, digit, before;
  int token;
};

template <int NT, int U>
struct CodeVisit {
  CodeLds<NT>& L;
  double inv_t, units;

  __device__ __forceinline__ void rare(uint32_t h) {
    const uint32_t mag = h & 0x7FFFu;
    const uint32_t q = mag - kCodeLow;
    if (q < static_cast<uint32_t>(kCodes)) {
      atomicAdd(&L.tab[(h >> 15 << 12) | q], 1u);
    } else if (mag < kCodeLow) {
      const float x = __uint_as_float(h << 16);
      atomicAdd(&L.tiny, static_cast<ull>(rint(exp(static_cast<double>(x) * inv_t) * units)));
      atomicAdd(&L.tiny_n, 1u);
    } else if (h == 0xFF80u) {
      // -inf weighs nothing
    } else if ((h & 0x8000u) && mag < 0x7F80u) {
      atomicMax(&L.low, up_key(__uint_as_float(h << 16)));
    } else {
      L.bad = 1;
    }
  }
  template <bool kPartial>
  __device__ __forceinline__ void group(const u32x4* w, int v, int nvec) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kPartial && v + u * NT >= nvec) continue;
      const uint32_t d[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
      u16x2 q[4], m = {0, 0};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const u16x2 base = {static_cast<uint16_t>(kCodeLow), static_cast<uint16_t>(kCodeLow)};
        q[k] = __builtin_bit_cast(u16x2, d[k] & 0x7FFF7FFFu) - base;
        m = __builtin_elementwise_max(m, q[k]);
      }
      if (m.x < kCodes && m.y < kCodes) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a = __builtin_bit_cast(uint32_t, q[k]) | (d[k] >> 3 & 0x10001000u);
          atomicAdd(&L.tab[a & 0xFFFFu], 1u);
          atomicAdd(&L.tab[a >> 16], 1u);
        }
      } else {
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          const uint32_t h = k == 0 ? w[u].x : k == 1 ? w[u].y : k == 2 ? w[u].z : w[u].w;
          rare(h & 0xFFFFu);
          rare(h >> 16);
        }
      }
    }
  }
  __device__ __forceinline__ void one(float x, int) { rare(__float_as_uint(x) >> 16); }
};

// The r-th (1, 2, ..) element of [e0, e1) that holds `code`, by index, or -1
// where there are more than the list holds.
template <int NT>
__device__ __forceinline__ int nth_code(const uint16_t* row, int e0, int e1, uint32_t code, int r, CodeLds<NT>& L) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  if (tid == 0) L.n = 0;
  lds_barrier();
  WantCode want{code | code << 16};
  auto put = [&](int at, int e) {
    if (at < kCodeList) L.list[at] = static_cast<uint32_t>(e);
  };
  GatherVisit<uint16_t, NT, kGatherUnroll, WantCode, decltype(put)> v{want, put, &L.n, row_head(row + e0, e1 - e0)};
  visit_row<uint16_t, NT, kGatherUnroll, kLoadNormal>(row + e0, e1 - e0, v);
  lds_barrier();
  const int n = L.n;
  if (n > kCodeList || r > n) return -1;
  if (n <= NT) {
    if (tid < n) {
      const uint32_t mine = L.list[tid];
      int before = 0;
      for (int i = 0; i < n; ++i) before += L.list[i] < mine ? 1 : 0;
      if (before == r - 1) L.token = static_cast<int>(mine);
    }
    lds_barrier();
    return e0 + L.token;
  }
  // a byte of the index at a time
  uint32_t prefix = 0;
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (shift > 0 && (static_cast<uint32_t>(e1 - e0) >> shift) == 0) continue;
    lds_barrier();
    for (int b = tid; b < 256; b += NT) L.hist[b] = 0;
    lds_barrier();
    for (int i = tid; i < n; i += NT) {
      const uint32_t e = L.list[i];
      if (shift == 24 || (e >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&L.hist[e >> shift & 255], 1u);
    }
    lds_barrier();
    if (tid < kWave) {
      // four digits a lane, upwards
      int c[4], sum = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) sum += c[k] = static_cast<int>(L.hist[lane * 4 + k]);
      int at = wave_scan_incl(sum) - sum;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (at < r && r <= at + c[k]) {
          L.digit = lane * 4 + k;
          L.before = at;
        }
        at += c[k];
      }
    }
    lds_barrier();
    prefix |= static_cast<uint32_t>(L.digit) << shift;
    r -= L.before;
  }
  lds_barrier();
  return e0 + static_cast<int>(prefix);
}

__device__ __forceinline__ uint32_t cell_code(int j) {
  return j < kCodes ? kCodeLow + static_cast<uint32_t>(kCodes - 1 - j) : (0x8000u | kCodeLow) + static_cast<uint32_t>(j - kCodes - 1);
}

template <int NT>
__device__ __forceinline__ void clear_codes(CodeLds<NT>& L) {
  for (int b = threadIdx.x; b < kTab; b += NT) L.tab[b] = 0;
  if (threadIdx.x == 0) {
    L.tiny = 0;
    L.tiny_n = 0;
    L.bad = 0;
    L.low = 0;
  }
  lds_barrier();
}

// The draw from a row's counts: L's tiny cell and flags, and cnt[k], the
// count of cell PER * thread + k. nth(code, r) finds the r-th element that
// holds a code. False where the row is left to draw_row (nothing is written).
template <int NT, int PER, typename Nth>
__device__ __forceinline__ bool draw_codes(const DrawArgs& a, int64_t r, const Draw& d, bool greedy, int bits,
                                           const int (&cnt)[PER], CodeLds<NT>& L, Nth nth) {
  constexpr int NW = NT / kWave;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const double T = static_cast<double>(d.T);
  if (tid < 6) L.j[tid] = kCells;
  lds_barrier();
  auto first_cell = [&](int q, auto pred) {
    int mine = kCells;
#pragma unroll
    for (int k = PER - 1; k >= 0; --k) mine = (cnt[k] > 0 && pred(k)) ? tid * PER + k : mine;
    mine = wave_all(mine, MinOp());
    if (lane == 0 && mine < kCells) atomicMin(&L.j[q], mine);
  };
  first_cell(0, [](int) { return true; });
  lds_barrier();
  const int jmax = L.j[0];
  if (L.bad || jmax >= kCells || jmax == kCodes || !(T >= kTinyT)) return false;
  const Weigh w{static_cast<double>(__uint_as_float(cell_code(jmax) << 16)), T, weight_units(a.x.V)};
  // a value below the table within reach of the maximum
  if (L.low != 0 && static_cast<double>(key_value(L.low)) > w.m - 48.0 * T) return false;

  // ---- cumulative weights and counts
  auto z_of = [&](int j) { return j == kCodes ? -w.m / T : w.z(__uint_as_float(cell_code(j) << 16)); };
  double through[PER], sum = 0.0;
  int seen[PER], num = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int j = tid * PER + k;
    if (cnt[k] > 0) {
      const double z = z_of(j);
      if (z > -48.0) sum += exp(z) * (j == kCodes ? static_cast<double>(L.tiny) / w.one : static_cast<double>(cnt[k]));
    }
    through[k] = sum;
    num += cnt[k];
    seen[k] = num;
  }
  double wb = wave_scan_incl(sum);
  int nb = wave_scan_incl(num);
  if (lane == kWave - 1) {
    L.red_d[wave] = wb;
    L.red_i[wave] = nb;
  }
  lds_barrier();
  wb -= sum;
  nb -= num;
  double total = 0.0;
#pragma unroll
  for (int k = 0; k < NW; ++k) {
    wb += k < wave ? L.red_d[k] : 0.0;
    nb += k < wave ? L.red_i[k] : 0;
    total += L.red_d[k];
  }
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    through[k] += wb;
    seen[k] += nb;
  }
  // ---- cuts: the cell, and how many of its tokens are through
  enum { kByCount, kReach_, kExceed };
  auto cut = [&](int q, int how, int count, double t) {
    if (how == kByCount) first_cell(q, [&](int k) { return seen[k] >= count; });
    if (how == kReach_) first_cell(q, [&](int k) { return through[k] >= t; });
    if (how == kExceed) first_cell(q, [&](int k) { return through[k] > t; });
    lds_barrier();
    const int j = L.j[q];
    if (j >= kCells || j == kCodes) return false;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      if (tid * PER + k == j) {
        const double before = k ? through[k > 0 ? k - 1 : 0] : wb;
        const double one = exp(z_of(j));
        int c;
        if (how == kByCount) {
          c = count - (k ? seen[k > 0 ? k - 1 : 0] : nb);
        } else {
          // the least c with before + c one at least (more than) t
          const double f = one > 0.0 ? fmin((t - before) / one, static_cast<double>(cnt[k])) : 1.0;
          c = how == kReach_ ? static_cast<int>(ceil(f)) : static_cast<int>(floor(f)) + 1;
          c = max(1, min(c, cnt[k]));
          auto past = [&](int q2) {
            const double s = before + static_cast<double>(q2) * one;
            return how == kReach_ ? s >= t : s > t;
          };
          if (c > 1 && past(c - 1)) --c;
          else if (c < cnt[k] && !past(c)) ++c;
        }
        L.cut_w = before + static_cast<double>(c) * one;
        L.cut_r = c;
      }
    }
    lds_barrier();
    return true;
  };
  double left = total;
  if (d.top_k > 0 && d.top_k < a.x.V) {
    // (-inf tokens are in no cell: a cut among them leaves everything)
    first_cell(1, [&](int k) { return seen[k] >= d.top_k; });
    lds_barrier();
    if (L.j[1] < kCells) {
      if (!cut(1, kByCount, d.top_k, 0.0)) return false;
      left = L.cut_w;
    }
  }
  if (d.top_p < 1.f) {
    if (!cut(2, kReach_, 0, reach(static_cast<double>(d.top_p) * left))) return false;
    left = fmin(left, L.cut_w);
  }
  if (d.min_p > 0.f) {
    const double zmin = log(static_cast<double>(d.min_p));
    // the tiny cell spans a few 2^-16 / T of z
    if (fabs(zmin + w.m / T) * T < 1.0 / 16384.0) return false;
    first_cell(3, [&](int k) { return z_of(tid * PER + k) < zmin; });
    lds_barrier();
    const int j = L.j[3];
    if (j < kCells) {
#pragma unroll
      for (int k = 0; k < PER; ++k)
        if (tid * PER + k == j) L.cut_w = k ? through[k > 0 ? k - 1 : 0] : wb;
      lds_barrier();
      left = fmin(left, L.cut_w);
    }
  }
  if (!cut(4, kExceed, 0, exceed(static_cast<double>(d.u) * left))) return false;
  const int j = L.j[4];
  const int token = nth(cell_code(j), L.cut_r);
  if (token < 0) return false;
  if (tid == 0) {
    a.token[r] = token;
    if (a.logprob) a.logprob[r] = greedy ? 0.f : log_share(z_of(j), left);
    if (a.lse) a.lse[r] = static_cast<float>(w.m / T + log(total));
    if (bits && a.error_flag) atomicOr(a.error_flag, bits);
  }
  return true;
}

template <int NT> constexpr int cells_per() { return (kCells + NT - 1) / NT; }

// The count of a cell of the table.
template <int NT>
__device__ __forceinline__ int cell_count(const CodeLds<NT>& L, int j) {
  if (j < kCodes) return static_cast<int>(L.tab[kCodes - 1 - j]);
  if (j == kCodes) return static_cast<int>(L.tiny_n);
  return j < kCells ? static_cast<int>(L.tab[4096 + j - kCodes - 1]) : 0;
}

// What a part of a bfloat16 row leaves: its cells' counts (a part has fewer
// than 2^16 elements), two to a word, and the rest of its table.
constexpr int kCellWords = (kCells + 1) / 2;
struct CodePart {
  uint32_t cells[kCellWords];
  uint32_t low;
  ull tiny;
  uint32_t bad, pad;
};

template <int NT>
__device__ __forceinline__ void leave_codes(CodePart* out, const CodeLds<NT>& L) {
  for (int i = threadIdx.x; i < kCellWords; i += NT)
    out->cells[i] = static_cast<uint32_t>(cell_count(L, 2 * i)) | static_cast<uint32_t>(cell_count(L, 2 * i + 1)) << 16;
  if (threadIdx.x == 0) {
    out->low = L.low;
    out->tiny = L.tiny;
    out->bad = static_cast<uint32_t>(L.bad);
  }
}
__device__ __forceinline__ int part_count(const CodePart& in, int j) { return static_cast<int>(in.cells[j >> 1] >> (j & 1) * 16 & 0xFFFFu); }

template <typename E, int NT, int U>
__global__ __launch_bounds__(NT, 4) void draw_part_kernel(DrawArgs a) {
  const int64_t r = blockIdx.x / a.parts;
  const int part = static_cast<int>(blockIdx.x - r * a.parts);
  const E* __restrict__ row = static_cast<const E*>(a.x.p) + r * a.x.ld;
  int e0, e1;
  row_part<E>(row, a.x.V, a.parts, part, e0, e1);
  int bits = 0;
  bool greedy;
  const Draw d = load_draw(a, r, bits, greedy);
  if constexpr (sizeof(E) == 2) {
    __shared__ CodeLds<NT> L;
    clear_codes(L);
    CodeVisit<NT, U> f{L, 1.0 / static_cast<double>(d.T), weight_units(a.x.V)};
    visit_row<E, NT, U, kLoadNormal>(row + e0, e1 - e0, f);
    lds_barrier();
    leave_codes(reinterpret_cast<CodePart*>(a.part) + blockIdx.x, L);
  } else {
    __shared__ DrawLds<NT> L;
    const bool count = d.top_k > 0 && d.top_k < a.x.V;
    const Binned b = row_bins<E, NT, U>(row + e0, e1 - e0, row, a.x.V, static_cast<double>(d.T), weight_units(a.x.V), count, L);
    leave_bins<NT>(b, count, reinterpret_cast<BinPart*>(a.part) + blockIdx.x, L);
  }
}

template <typename E, int NT, int U>
__global__ __launch_bounds__(NT, 4) void draw_join_kernel(DrawArgs a) {
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  if constexpr (sizeof(E) == 2) {
    __shared__ union {
      DrawLds<NT> row;
      CodeLds<NT> code;
    } L;
    constexpr int PER = cells_per<NT>();
    int bits = 0;
    bool greedy;
    const Draw d = load_draw(a, r, bits, greedy);
    const E* __restrict__ row = static_cast<const E*>(a.x.p) + r * a.x.ld;
    const CodePart* in = reinterpret_cast<const CodePart*>(a.part) + r * a.parts;
    // the cells' sums in rank order, through LDS; every load of a step is
    // issued before any is used (see join_bins)
    if (tid == 0) {
      L.code.bad = 0;
      L.code.low = 0;
      L.code.tiny = 0;
    }
    const CodePart& head = in[tid < a.parts ? tid : 0];
    const uint32_t bad = head.bad, low = head.low;
    const ull tiny = head.tiny;
    lds_barrier();
    if (tid < a.parts) {
      atomicOr(&L.code.bad, static_cast<int>(bad));
      atomicMax(&L.code.low, low);
      atomicAdd(&L.code.tiny, tiny);
    }
#pragma unroll 2
    for (int i = tid; i < kCellWords; i += NT) {
      uint32_t c[kMostParts];
#pragma unroll
      for (int p = 0; p < kMostParts; ++p) c[p] = in[p < a.parts ? p : 0].cells[i];
      uint32_t lo = 0, hi = 0;
#pragma unroll
      for (int p = 0; p < kMostParts; ++p) {
        lo += p < a.parts ? c[p] & 0xFFFFu : 0u;
        hi += p < a.parts ? c[p] >> 16 : 0u;
      }
      L.code.tab[2 * i] = lo;
      L.code.tab[2 * i + 1] = hi;
    }
    lds_barrier();
    int cnt[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int j = tid * PER + k;
      cnt[k] = j < kCells ? static_cast<int>(L.code.tab[j]) : 0;
    }
    const bool done = draw_codes<NT, PER>(a, r, d, greedy, bits, cnt, L.code, [&](uint32_t code, int q) {
      // the part that holds the q-th, and there the rest of the way
      const int j = (code & 0x8000u) ? kCodes + 1 + static_cast<int>(code - (0x8000u | kCodeLow))
                                     : kCodes - 1 - static_cast<int>(code - kCodeLow);
      const int lane = tid & (kWave - 1);
      const int held = part_count(in[lane < a.parts ? lane : 0], j);
      int p = 0;
      for (; p < a.parts - 1; ++p) {
        const int n = read_lane(held, p);
        if (q <= n) break;
        q -= n;
      }
      int e0, e1;
      row_part<E>(row, a.x.V, a.parts, p, e0, e1);
      return nth_code<NT>(row, e0, e1, code, q, L.code);
    });
    if (done) return;
    lds_barrier();
    draw_row<E, NT, U, false>(a, r, L.row);
  } else {
    __shared__ DrawLds<NT> L;
    draw_row<E, NT, U, true>(a, r, L);
  }
}

template <typename E, int NT, int U>
__global__ __launch_bounds__(NT, 4) void draw_kernel(DrawArgs a) {
  const int64_t r = blockIdx.x;
  if constexpr (sizeof(E) == 2) {
    __shared__ union {
      DrawLds<NT> row;
      CodeLds<NT> code;
    } L;
    constexpr int PER = cells_per<NT>();
    int bits = 0;
    bool greedy;
    const Draw d = load_draw(a, r, bits, greedy);
    const E* __restrict__ row = static_cast<const E*>(a.x.p) + r * a.x.ld;
    clear_codes(L.code);
    CodeVisit<NT, U> f{L.code, 1.0 / static_cast<double>(d.T), weight_units(a.x.V)};
    visit_row<E, NT, U, kLoadNormal>(row, a.x.V, f);
    lds_barrier();
    int cnt[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) cnt[k] = cell_count(L.code, static_cast<int>(threadIdx.x) * PER + k);
    const bool done = draw_codes<NT, PER>(a, r, d, greedy, bits, cnt, L.code, [&](uint32_t code, int q) {
      return nth_code<NT>(row, 0, a.x.V, code, q, L.code);
    });
    if (done) return;
    lds_barrier();
    draw_row<E, NT, U, false>(a, r, L.row);
  } else {
    __shared__ DrawLds<NT> L;
    draw_row<E, NT, U, false>(a, r, L);
  }
}

template <typename E>
hipError_t draw_t(const DrawArgs& a, hipStream_t s) {
  if (a.parts > 1) {
    draw_part_kernel<E, kDrawThreads, kDrawUnroll>
        <<<dim3(static_cast<unsigned>(a.x.N * a.parts)), dim3(kDrawThreads), 0, s>>>(a);
    draw_join_kernel<E, kDrawThreads, kDrawUnroll><<<dim3(a.x.N), dim3(kDrawThreads), 0, s>>>(a);
  } else {
    draw_kernel<E, kDrawThreads, kDrawUnroll><<<dim3(a.x.N), dim3(kDrawThreads), 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

int32_t draw_parts(int32_t num_rows, int32_t vocab, int32_t dtype) {
  const int64_t bytes = static_cast<int64_t>(vocab) * (dtype == VSV_BF16 ? 2 : 4);
  if (bytes < 131072) return 1;
  int64_t p = 512 / (num_rows > 0 ? num_rows : 1);
  const int64_t most = bytes / 32768;
  if (p > most) p = most;
  if (p > kMostParts) p = kMostParts;
  // a part's counts are 16 bits wide
  if (p < 2 || vocab / p >= 65000) return 1;
  return static_cast<int32_t>(p);
}

size_t draw_part_bytes(int32_t dtype) { return dtype == VSV_BF16 ? sizeof(CodePart) : sizeof(BinPart); }

hipError_t launch_draw(const DrawArgs& a, hipStream_t s) {
  return a.x.dtype == VSV_BF16 ? draw_t<uint16_t>(a, s) : draw_t<float>(a, s);
}

}  // namespace vsv
