// Distillation of a student's rows of logits from a teacher's top logits:
// the loss of every row and its gradient.
//
// With y a student row, q = softmax(y / T), and a row's used entries (an id
// and the teacher's logit z there):
//   without the teacher's log-sum-exp: t = softmax(z / T) over the entries,
//     loss = sum_k t_k (ln t_k - ln q_k);
//   with it (L): t_k = exp(z_k / T - L), what they leave of one,
//     t_r = max(0, 1 - sum t), is the mass of the rest, set against the
//     student's mass outside the named ids, q_r:
//     loss = sum_k t_k (ln t_k - ln q_k) + t_r (ln t_r - ln q_r)
//     (t_r counts as 0 where it is the rounding of L and q_r is nothing).
// With M = sum t + t_r the gradient of a row's loss is
//   (q_i M - sum of the t that name i) / T   at a named id,
//   q_i (M - t_r / q_r) / T                  elsewhere,
// so the pass over the row only multiplies a softmax by one number and the
// named ids are put right afterwards.
//
// q_r is summed over the elements outside the ids, not taken from 1 - q(ids):
// once the student agrees with the teacher the ids hold nearly everything
// and the difference would keep few digits. A bit per element in LDS, read a
// vector at a time, says which elements are named. That sum has an exponent
// reference of its own, and the unnamed elements' gradient is taken relative
// to it, exp2(x c - reference) times M / (sum of the row) - t_r / (sum of the
// rest): with the row's reference both factors of q_i t_r / q_r would leave
// the float range once the named logits lie 88 T above the rest.
//
// HBM bounds all of it: the losses of 640 bf16 rows of 152064 take 38 us (5.1
// TB/s), the gradient of 2048 from their state 245 us (5.1 TB/s read and
// written, as a large copy), loss and gradient in one launch 290 us, 240 being
// one read and one write at a copy's rate.
#include "row_visit.hpp"
#include "rows.hpp"

namespace vsv {

namespace {

// Vectors per thread and group: two in the forward pass (22.7 us for 300
// bf16 rows of 152064, 25.8 with three; the same for 640 and 2048), three
// where the gradient follows in the same launch (2048 rows: 290 us, 298 with
// two), four for the gradient's own pass (2048 rows: 245 us, 247 with two).
constexpr int kDistThreads = 512;
constexpr int kSumUnroll = 2;
constexpr int kBothUnroll = 3;
constexpr int kGradUnroll = 4;
constexpr int kEntries = VSV_MAX_TOP / kWave;   // entries per lane of the wave that handles them
// Vectors whose named elements one LDS map holds, a byte per vector (and two
// for the elements before and after them). Longer rows go in pieces.
constexpr int kMapSlots = 20480;
constexpr int kMapWords = kMapSlots / 4;

// The map's byte of an element: 0 before the aligned body, then one per
// vector, the last after the body.
template <typename E>
__device__ __forceinline__ int map_slot(int e, int head, int& bit) {
  constexpr int N = Elem<E>::kVec;
  const int q = e + N - head;
  bit = q % N;
  return q / N;
}

template <typename E, int NT, int U, bool kRest>
struct SumVisit {
  ExpSum p;
  float c, most;   // most: the largest element seen
  const uint8_t* map;
  int head;

  template <bool kPartial>
  __device__ __forceinline__ void group(const u32x4* w, int v, int nvec) {
    constexpr int N = Elem<E>::kVec;
    float f[U * N];
    float gmax = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool out = kPartial && v + u * NT >= nvec;
      Elem<E>::decode(w[u], f + u * N);
      const int named = (kRest && !out) ? map[v + u * NT + 1] : 0;
      if (out || named) {
#pragma unroll
        for (int k = 0; k < N; ++k) f[u * N + k] = (out || (named >> k & 1)) ? -INFINITY : f[u * N + k];
      }
#pragma unroll
      for (int k = 0; k < N; ++k) gmax = fmaxf(gmax, f[u * N + k]);
    }
    if (kRest) most = fmaxf(most, gmax);
    add_terms<U * N>(p, f, gmax, c);
  }
  __device__ __forceinline__ void one(float x, int e) {
    if (kRest) {
      int bit;
      const int slot = map_slot<E>(e, head, bit);
      if (map[slot] >> bit & 1) return;
    }
    if (kRest) most = fmaxf(most, x);
    add_term(p, x, c);
  }
};

// A range's sums outside and over the named ids, each relative to its own
// exponent reference, and the largest elements there. Without a rest
// everything counts as outside.
struct Sums {
  double rest = 0.0, named = 0.0;
  float mr = -FLT_MAX, xr = -INFINITY, mn = -FLT_MAX, xn = -INFINITY;
};
static_assert(sizeof(Sums) == kPartDoubles * sizeof(double), "a part's scratch");

template <int NT> struct DistillLds {
  static constexpr int NW = NT / kWave;
  uint32_t map[kMapWords];
  float mr[NW], xr[NW];
  double rest[NW];
  double row[kStateWords];
  int any;
};

// A row's entries, lane + 64 j of one wave: id (-1: unused), the teacher's
// logit, the student's logit there and whether the id appears for the first
// time.
struct Entries {
  int id[kEntries];
  float z[kEntries], y[kEntries];
  bool first[kEntries];
};

template <typename E>
__device__ __forceinline__ void load_entries(const DistillArgs& a, int64_t r, const E* row, Entries& t, int& bits) {
  const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
  for (int j = 0; j < kEntries; ++j) {
    const int k = lane + j * kWave;
    t.id[j] = -1;
    t.z[j] = t.y[j] = 0.f;
    t.first[j] = false;
    if (k < a.K) {
      int id = a.ids[r * a.K + k];
      if (id >= a.x.V) {
        bits |= VSV_FLAG_TOKEN;
        id = -1;
      }
      if (id >= 0) {
        t.id[j] = id;
        t.z[j] = a.top[r * a.K + k];
        t.y[j] = Elem<E>::at(row, id);
      }
    }
  }
}

// Whether any of a wave's entries is used.
__device__ __forceinline__ bool any_used(const Entries& t) {
  bool used = false;
#pragma unroll
  for (int j = 0; j < kEntries; ++j) used |= t.id[j] >= 0;
  return __builtin_amdgcn_ballot_w64(used) != 0;
}

// The sums of elements [e0, e1) of a row over the whole workgroup. With
// kRest the named elements' weights are kept apart, each id counted once; the
// wave that handles the entries receives those.
template <typename E, int NT, int U, bool kRest, int kAux>
__device__ __forceinline__ Sums range_sums(const DistillArgs& a, const E* __restrict__ row, int e0, int e1, Entries& t,
                                           DistillLds<NT>& L) {
  constexpr int N = Elem<E>::kVec;
  constexpr int NW = NT / kWave;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  SumVisit<E, NT, U, kRest> f;
  f.p = ExpSum{-FLT_MAX, 0.0};
  f.c = a.c;
  f.most = -INFINITY;
  f.map = reinterpret_cast<const uint8_t*>(L.map);
  // pieces end at 16-byte boundaries of the row, so only the first has
  // elements before its body and only the last some after it
  constexpr int kPiece = (kMapSlots - 2) * N;
  for (int p0 = e0; p0 < e1;) {
    f.head = row_head(row + p0, e1 - p0);
    const int p1 = (kRest && e1 - p0 > kPiece) ? p0 + f.head + (kMapSlots - 3) * N : e1;
    if (kRest) {
      const int words = min(kMapWords, ((p1 - p0) / N + 2) / 4 + 1);
      for (int w = tid; w < words; w += NT) L.map[w] = 0u;
      lds_barrier();
      if (wave == 0) {
#pragma unroll
        for (int j = 0; j < kEntries; ++j) {
          if (t.id[j] >= p0 && t.id[j] < p1) {
            int bit;
            const int slot = map_slot<E>(t.id[j] - p0, f.head, bit);
            const uint32_t m = 1u << ((slot & 3) * 8 + bit);
            t.first[j] = (atomicOr(&L.map[slot >> 2], m) & m) == 0u;
          }
        }
      }
      lds_barrier();
    }
    visit_row<E, NT, U, kAux>(row + p0, p1 - p0, f);
    p0 = p1;
    if (kRest && p0 < e1) lds_barrier();
  }
  const float mw = wave_all(f.p.mc, MaxOp()), xw = wave_all(f.most, MaxOp());
  if (lane == 0) {
    L.mr[wave] = mw;
    L.xr[wave] = xw;
  }
  lds_barrier();
  Sums o;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    o.mr = fmaxf(o.mr, L.mr[w]);
    o.xr = fmaxf(o.xr, L.xr[w]);
  }
  const double sr = wave_sum_f64(sum_at(f.p.s, f.p.mc, o.mr));
  if (lane == 0) L.rest[wave] = sr;
  lds_barrier();
#pragma unroll
  for (int w = 0; w < NW; ++w) o.rest += L.rest[w];
  if (kRest && wave == 0) {
#pragma unroll
    for (int j = 0; j < kEntries; ++j)
      if (t.first[j]) o.xn = fmaxf(o.xn, t.y[j]);
    o.xn = wave_all(o.xn, MaxOp());
    ExpSum n{-FLT_MAX, 0.0};
    raise_ref(n, o.xn, a.c);
    o.mn = n.mc;
    double named = 0.0;
#pragma unroll
    for (int j = 0; j < kEntries; ++j)
      if (t.first[j]) named += static_cast<double>(fast_exp2(exp_arg(t.y[j], a.c, o.mn)));
    o.named = wave_sum_f64(named);
  }
  return o;
}

// The exponent references of a row's unnamed elements and of its whole, one
// word of its state. (Put together as an integer: the cast of a struct of two
// floats goes through memory, which the compiler moves to LDS by way of the
// dispatch packet, and the kernels took up to 7 us more.)
__device__ __forceinline__ double pack_refs(float rest, float row) {
  return __builtin_bit_cast(double, static_cast<uint64_t>(__float_as_uint(row)) << 32 | __float_as_uint(rest));
}
__device__ __forceinline__ float rest_ref(double s) { return __uint_as_float(static_cast<uint32_t>(__builtin_bit_cast(uint64_t, s))); }
__device__ __forceinline__ float row_ref(double s) { return __uint_as_float(static_cast<uint32_t>(__builtin_bit_cast(uint64_t, s) >> 32)); }

// A rest of the teacher counts as none where the student's is below 2^-126
// (ln of it) and it is no more than the float32 log-sum-exp, of float32
// exponentials, may be off by: those and the terms' arguments are within
// 2^-22 (1 + |x| / T) together, the result is rounded by 2^-24 of itself, and
// |x| / T is |lse| but for the few T over which weight spreads. Where the
// student's rest is larger, such a t_r adds less than 1e-4 and is kept.
constexpr double kNoRest = -87.33654475055310;
constexpr double kLseRounding = 1.0 / 1048576.0;   // 2^-20

constexpr double kLn2 = 0.69314718055994530942;

// x c as the terms took it, above their reference m.
__device__ __forceinline__ double above_ref(float x, float c, float m) {
  return fabsf(m) < kFarRef ? static_cast<double>(x) * static_cast<double>(c) - static_cast<double>(m)
                            : static_cast<double>(far_arg(x, c, m));
}

// The row's loss and state from its sums, by one whole wave: `st` receives
// what the backward pass needs.
template <bool kRest>
__device__ __forceinline__ void finish_distill(const DistillArgs& a, int64_t r, const Sums& s, const Entries& t, int bits,
                                               double* st) {
  const int lane = threadIdx.x & (kWave - 1);
  const float mc = fmaxf(s.mr, s.mn);
  const double total = sum_at(s.rest, s.mr, mc) + sum_at(s.named, s.mn, mc);
  const double lg = log2(total);
  // log t_k = z_k / T - lt
  double lt;
  if (kRest) {
    lt = static_cast<double>(a.tlse[r]);
  } else {
    double zm = -INFINITY, es = 0.0;
#pragma unroll
    for (int j = 0; j < kEntries; ++j)
      if (t.id[j] >= 0) zm = fmax(zm, static_cast<double>(t.z[j]) * a.inv_t);
    zm = wave_all(zm, MaxOp());
#pragma unroll
    for (int j = 0; j < kEntries; ++j)
      if (t.id[j] >= 0 && zm > -INFINITY) es += exp(static_cast<double>(t.z[j]) * a.inv_t - zm);
    // entries of weight 0 alone name nothing: every t_k is 0 then
    lt = zm > -INFINITY ? zm + log(wave_sum_f64(es)) : 0.0;
  }
  double mass = 0.0, loss = 0.0;
#pragma unroll
  for (int j = 0; j < kEntries; ++j) {
    if (t.id[j] >= 0) {
      const double lk = static_cast<double>(t.z[j]) * a.inv_t - lt;
      const double tk = exp(lk);
      if (!(tk == 0.0)) {
        mass += tk;
        // ln q_k; the exponent is exact where its float would not be
        const double at = above_ref(t.y[j], a.c, mc);
        loss += tk * (lk - kLn2 * (at - lg));
      }
    }
  }
  mass = wave_sum_f64(mass);
  loss = wave_sum_f64(loss);
  double every = mass, off = 0.0;   // off: what t_r takes off the unnamed tokens' factor
  if (kRest) {
    const double tr = 1.0 - mass;
    if (tr > 0.0) {
      const float xm = fmaxf(s.xr, s.xn);
      // ln q_r by way of the two largest elements, whose difference may be
      // most of it: in float64, where x c is rounded
      const double log_qr = s.rest == 0.0 ? -INFINITY
                                          : (static_cast<double>(s.xr) - static_cast<double>(xm)) * a.inv_t +
                                                kLn2 * ((log2(s.rest) - above_ref(s.xr, a.c, s.mr)) -
                                                        (lg - above_ref(xm, a.c, mc)));
      // of a teacher whose entries hold all of its mass, as where a vocabulary
      // mask leaves no others, its float32 log-sum-exp leaves a rounding
      if (!(log_qr < kNoRest && tr <= kLseRounding * (1.0 + fabs(lt)))) {
        every += tr;
        loss += tr * (log(tr) - log_qr);
        off = s.rest == 0.0 ? 0.0 : tr / s.rest;
      }
    }
  }
  if (!(total > 0.0 && total < INFINITY) || !(mass < INFINITY)) bits |= VSV_FLAG_LOGITS;
  bits = wave_all(bits, [](int p, int q) { return p | q; });
  if (lane == 0) {
    const double norm = 1.0 / total;
    st[0] = pack_refs(s.mr, mc);
    st[1] = norm;
    st[2] = sum_at(every, s.mr, mc) * norm - off;
    st[3] = every;
    st[4] = lt;
    if (a.loss) a.loss[r] = static_cast<float>(loss);
    if (bits && a.error_flag) atomicOr(a.error_flag, bits);
  }
}

// A row without a used entry: loss and gradient are 0 whatever it holds.
__device__ __forceinline__ void finish_unused(const DistillArgs& a, int64_t r, int bits, double* st) {
  if ((threadIdx.x & (kWave - 1)) == 0) {
#pragma unroll
    for (int k = 0; k < kStateWords; ++k) st[k] = 0.0;
    if (a.loss) a.loss[r] = 0.f;
  }
  bits = wave_all(bits, [](int p, int q) { return p | q; });
  if (bits && a.error_flag && (threadIdx.x & (kWave - 1)) == 0) atomicOr(a.error_flag, bits);
}

// Statistics of row r by the whole workgroup, up to its state in L.row; false
// if the row has no used entry.
template <typename E, int NT, int U, bool kRest, int kAux>
__device__ __forceinline__ bool row_state(const DistillArgs& a, int64_t r, DistillLds<NT>& L) {
  const E* __restrict__ row = static_cast<const E*>(a.x.p) + r * a.x.ld;
  const int wave = threadIdx.x / kWave;
  Entries t;
  int bits = 0;
  if (wave == 0) {
    load_entries<E>(a, r, row, t, bits);
    const bool any = any_used(t);
    if (threadIdx.x == 0) L.any = any;
    if (!any) finish_unused(a, r, bits, L.row);
  } else {
#pragma unroll
    for (int j = 0; j < kEntries; ++j) {
      t.id[j] = -1;
      t.first[j] = false;
    }
  }
  lds_barrier();
  if (!L.any) return false;
  const Sums s = range_sums<E, NT, U, kRest, kAux>(a, row, 0, a.x.V, t, L);
  if (wave == 0) finish_distill<kRest>(a, r, s, t, bits, L.row);
  lds_barrier();
  return true;
}

template <typename E, int NT, int U, bool kRest>
__global__ __launch_bounds__(NT) void distill_forward_kernel(DistillArgs a) {
  __shared__ DistillLds<NT> L;
  const int64_t r = blockIdx.x;
  row_state<E, NT, U, kRest, kLoadStream>(a, r, L);
  if (a.state && threadIdx.x < kStateWords) a.state[r * kStateWords + threadIdx.x] = L.row[threadIdx.x];
}

// Few rows: a workgroup per part of a row leaves the part's sums, and one
// wave per row joins them.
template <typename E, int NT, int U, bool kRest>
__global__ __launch_bounds__(NT) void distill_part_kernel(DistillArgs a) {
  __shared__ DistillLds<NT> L;
  const int64_t r = blockIdx.x / a.parts;
  const int part = static_cast<int>(blockIdx.x - r * a.parts);
  const E* __restrict__ row = static_cast<const E*>(a.x.p) + r * a.x.ld;
  int e0, e1;
  row_part<E>(row, a.x.V, a.parts, part, e0, e1);
  Entries t;
  int bits = 0;
  if (threadIdx.x < kWave) {
    load_entries<E>(a, r, row, t, bits);
    const bool any = any_used(t);
    if (threadIdx.x == 0) L.any = any;
  } else {
#pragma unroll
    for (int j = 0; j < kEntries; ++j) {
      t.id[j] = -1;
      t.first[j] = false;
    }
  }
  lds_barrier();
  if (!L.any) return;   // the join finds the same and reads no sums
  const Sums s = range_sums<E, NT, U, kRest, kLoadStream>(a, row, e0, e1, t, L);
  if (threadIdx.x == 0) {
    reinterpret_cast<Sums*>(a.part)[blockIdx.x] = s;
  }
}

template <typename E, bool kRest>
__global__ __launch_bounds__(kWave) void distill_join_kernel(DistillArgs a) {
  __shared__ double st[kStateWords];
  const int64_t r = blockIdx.x;
  const E* __restrict__ row = static_cast<const E*>(a.x.p) + r * a.x.ld;
  const int lane = threadIdx.x;
  Entries t;
  int bits = 0;
  load_entries<E>(a, r, row, t, bits);
  if (!any_used(t)) {
    finish_unused(a, r, bits, st);
  } else {
    Sums mine;
    if (lane < a.parts) mine = reinterpret_cast<const Sums*>(a.part)[r * a.parts + lane];
    Sums s;
    s.mr = wave_all(mine.mr, MaxOp());
    s.xr = wave_all(mine.xr, MaxOp());
    s.mn = wave_all(mine.mn, MaxOp());
    s.xn = wave_all(mine.xn, MaxOp());
    s.rest = wave_sum_f64(sum_at(mine.rest, mine.mr, s.mr));
    s.named = wave_sum_f64(sum_at(mine.named, mine.mn, s.mn));
    finish_distill<kRest>(a, r, s, t, bits, st);
  }
  lds_barrier();
  if (a.state && lane < kStateWords) a.state[r * kStateWords + lane] = st[lane];
}

// ---------------------------------------------------------------- gradient

// 16 bytes at an address that is a multiple of the element size only: the
// gradient's rows are stored aligned, and the student's rows may lie
// otherwise.
template <typename E> struct Loose;
template <> struct Loose<uint16_t> {
  typedef u32x4 type __attribute__((aligned(2)));
};
template <> struct Loose<float> {
  typedef u32x4 type __attribute__((aligned(4)));
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Rounded to nearest even once, from float.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}
template <typename E> __device__ __forceinline__ u32x4 encode(const float* f);
template <> __device__ __forceinline__ u32x4 encode<float>(const float* f) {
  return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
}
template <> __device__ __forceinline__ u32x4 encode<uint16_t>(const float* f) {
  return u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16(v, 0.f)); }

// out[e] = exp2(x[e] c - mc) f over [e0, e1).
template <typename E, int NT, int U>
__device__ __forceinline__ void scaled_softmax(const E* row, E* out, int e0, int e1, float c, float mc, float f) {
  constexpr int N = Elem<E>::kVec;
  const int tid = threadIdx.x;
  const E* x = row + e0;
  E* g = out + e0;
  const int n = e1 - e0;
  const int head = row_head(g, n);
  const int nvec = (n - head) / N;
  const typename Loose<E>::type* xv = reinterpret_cast<const typename Loose<E>::type*>(x + head);
  u32x4* gv = reinterpret_cast<u32x4*>(g + head);
  const bool near = fabsf(mc) < kFarRef;
  auto value = [&](float v) { return fast_exp2(near ? fmaf(v, c, -mc) : far_arg(v, c, mc)) * f; };
  auto vec = [&](const u32x4& w) {
    float v[N];
    Elem<E>::decode(w, v);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = value(v[k]);
    return encode<E>(v);
  };
  int i = tid;
  for (; i + (U - 1) * NT < nvec; i += U * NT) {
    u32x4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = xv[i + u * NT];
#pragma unroll
    for (int u = 0; u < U; ++u) __builtin_nontemporal_store(vec(w[u]), gv + i + u * NT);
  }
  for (; i < nvec; i += NT) {
    const u32x4 w = xv[i];
    __builtin_nontemporal_store(vec(w), gv + i);
  }
  if (tid < head) put(g + tid, value(Elem<E>::at(x, tid)));
  const int end = head + nvec * N;
  if (tid < n - end) put(g + end + tid, value(Elem<E>::at(x, end + tid)));
}

template <typename E, int NT>
__device__ __forceinline__ void fill_zero(E* out, int e0, int e1) {
  constexpr int N = Elem<E>::kVec;
  const int tid = threadIdx.x;
  E* g = out + e0;
  const int n = e1 - e0;
  const int head = row_head(g, n);
  const int nvec = (n - head) / N;
  u32x4* gv = reinterpret_cast<u32x4*>(g + head);
  for (int i = tid; i < nvec; i += NT) __builtin_nontemporal_store(u32x4{0u, 0u, 0u, 0u}, gv + i);
  if (tid < head) put(g + tid, 0.f);
  const int end = head + nvec * N;
  if (tid < n - end) put(g + end + tid, 0.f);
}

// The gradient of elements [e0, e1) of row r, given its state.
template <typename E, int NT, int U>
__device__ __forceinline__ void grad_range(const DistillArgs& a, int64_t r, int e0, int e1, const double* st, int* ids,
                                           float* teach) {
  const E* row = static_cast<const E*>(a.x.p) + r * a.x.ld;
  E* out = static_cast<E*>(a.grad) + r * a.grad_ld;
  const int tid = threadIdx.x;
  const float mr = rest_ref(st[0]), mc = row_ref(st[0]);
  const double norm = st[1], factor = st[2], every = st[3], lt = st[4];
  const double g = (a.weight ? static_cast<double>(a.weight[r]) : 1.0) * a.inv_t;
  if (every == 0.0 || g == 0.0) {
    fill_zero<E, NT>(out, e0, e1);
    return;
  }
  // thread k holds entry k: the student's logit is read before anything is
  // written, its teacher mass joins that of the same id's other entries
  int id = -1;
  float y = 0.f;
  if (tid < a.K) {
    id = a.ids[r * a.K + tid];
    float t = 0.f;
    if (id >= a.x.V || id < 0) {
      id = -1;
    } else {
      t = static_cast<float>(exp(static_cast<double>(a.top[r * a.K + tid]) * a.inv_t - lt));
      y = Elem<E>::at(row, id);
    }
    ids[tid] = id;
    teach[tid] = t;
  }
  lds_barrier();
  // (what this leaves at the named ids, which may lie far above the rest, is
  // written over)
  scaled_softmax<E, NT, U>(row, out, e0, e1, a.c, mr, static_cast<float>(factor * g));
  __syncthreads();   // the pass's stores come before the named ids' own
  if (id >= e0 && id < e1) {
    double t = 0.0;
    bool first = true;
    for (int k = 0; k < a.K; ++k) {
      if (ids[k] == id) {
        t += static_cast<double>(teach[k]);
        first = first && k >= tid;
      }
    }
    const double q = static_cast<double>(fast_exp2(exp_arg(y, a.c, mc))) * norm;
    if (first) put(out + id, static_cast<float>((q * every - t) * g));
  }
}

template <typename E, int NT, int U>
__global__ __launch_bounds__(NT) void distill_backward_kernel(DistillArgs a) {
  __shared__ int ids[VSV_MAX_TOP];
  __shared__ float teach[VSV_MAX_TOP];
  const int64_t r = blockIdx.x / a.parts;
  const int part = static_cast<int>(blockIdx.x - r * a.parts);
  int e0, e1;
  row_part<E>(static_cast<const E*>(a.grad) + r * a.grad_ld, a.x.V, a.parts, part, e0, e1);
  grad_range<E, NT, U>(a, r, e0, e1, a.state + r * kStateWords, ids, teach);
}

// Loss and gradient in one launch: a row's second reading follows its first
// at once, so it comes from the caches, and the row crosses HBM once each
// way.
template <typename E, int NT, int U, bool kRest>
__global__ __launch_bounds__(NT) void distill_grad_kernel(DistillArgs a) {
  __shared__ DistillLds<NT> L;
  __shared__ int ids[VSV_MAX_TOP];
  __shared__ float teach[VSV_MAX_TOP];
  const int64_t r = blockIdx.x;
  row_state<E, NT, U, kRest, kLoadNormal>(a, r, L);
  grad_range<E, NT, kGradUnroll>(a, r, 0, a.x.V, L.row, ids, teach);
}

template <typename E>
hipError_t forward_t(const DistillArgs& a, hipStream_t s) {
  const bool rest = a.tlse != nullptr;
  if (a.parts > 1) {
    const int64_t grid = static_cast<int64_t>(a.x.N) * a.parts;
    auto part = rest ? distill_part_kernel<E, kDistThreads, kSumUnroll, true>
                     : distill_part_kernel<E, kDistThreads, kSumUnroll, false>;
    part<<<dim3(static_cast<unsigned>(grid)), dim3(kDistThreads), 0, s>>>(a);
    auto join = rest ? distill_join_kernel<E, true> : distill_join_kernel<E, false>;
    join<<<dim3(a.x.N), dim3(kWave), 0, s>>>(a);
  } else {
    auto k = rest ? distill_forward_kernel<E, kDistThreads, kSumUnroll, true>
                  : distill_forward_kernel<E, kDistThreads, kSumUnroll, false>;
    k<<<dim3(a.x.N), dim3(kDistThreads), 0, s>>>(a);
  }
  return hipGetLastError();
}

template <typename E>
hipError_t backward_t(const DistillArgs& a, hipStream_t s) {
  const int64_t grid = static_cast<int64_t>(a.x.N) * a.parts;
  distill_backward_kernel<E, kDistThreads, kGradUnroll>
      <<<dim3(static_cast<unsigned>(grid)), dim3(kDistThreads), 0, s>>>(a);
  return hipGetLastError();
}

template <typename E>
hipError_t grad_t(const DistillArgs& a, hipStream_t s) {
  auto k = a.tlse ? distill_grad_kernel<E, kDistThreads, kBothUnroll, true>
                  : distill_grad_kernel<E, kDistThreads, kBothUnroll, false>;
  k<<<dim3(a.x.N), dim3(kDistThreads), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

int32_t distill_parts(int32_t num_rows, int32_t vocab, int32_t dtype) {
  const int64_t bytes = static_cast<int64_t>(vocab) * (dtype == VSV_BF16 ? 2 : 4);
  const int64_t n = num_rows > 0 ? num_rows : 1;
  // Rows are cut while whole rows would leave CUs idle, up to 96 of them: 64
  // bf16 rows of 152064 take 28 us with the gradient in three parts, 31 whole
  // (calls back to back). From 97 rows on a workgroup per row is the better
  // use, since it needs no second launch and its gradient follows the sums in
  // the same one: 112 bf16 rows take 17.1 us forward and 33.5 with the
  // gradient, against 15.9 and 36.2 in two parts. (fp32 rows, twice as long,
  // would still gain from two: 26 and 62 us against 20 and 54.) Short rows
  // are not worth the second launch: 128 fp32 rows of 32768 take 8.8 us whole
  // and 10.7 in two parts. The gradient's own pass takes the forward's parts,
  // though for itself it could take more: those 128 rows leave half of the
  // CUs without any, 13 us of which 6.5 are the bytes.
  if (bytes < 196608) return 1;
  int64_t p = 192 / n;
  const int64_t most = bytes / 49152;
  if (p > most) p = most;
  if (p > kWave) p = kWave;
  return p < 1 ? 1 : static_cast<int32_t>(p);
}

hipError_t launch_distill_forward(const DistillArgs& a, hipStream_t s) {
  return a.x.dtype == VSV_BF16 ? forward_t<uint16_t>(a, s) : forward_t<float>(a, s);
}
hipError_t launch_distill_backward(const DistillArgs& a, hipStream_t s) {
  return a.x.dtype == VSV_BF16 ? backward_t<uint16_t>(a, s) : backward_t<float>(a, s);
}
hipError_t launch_distill_grad(const DistillArgs& a, hipStream_t s) {
  if (a.parts > 1) {
    const hipError_t e = launch_distill_forward(a, s);
    return e != hipSuccess ? e : launch_distill_backward(a, s);
  }
  return a.x.dtype == VSV_BF16 ? grad_t<uint16_t>(a, s) : grad_t<float>(a, s);
}

}  // namespace vsv
