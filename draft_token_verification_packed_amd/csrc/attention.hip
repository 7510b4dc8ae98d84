// Attention of packed draft rows over a paged cache (gfx950, MFMA).
//
// Row r of request i (a node of its tree of drafts) sees the request's
// length[i] cached tokens, the rows on its path from the root, and itself:
//   o[r, h] = sum_t p_t v_t,  p = softmax over the seen t of scale q[r, h] . k_t
// The rows' own keys and values come packed beside q, not from the cache:
// which of them belong into the cache is known only once the drafts are
// verified, so no rejected draft ever takes a slot there.
//
// The M = rows * G queries that share a key head (G = H / KV) are one matrix,
// so a key head's tokens are read once for all of them. Scores are computed
// transposed, S^T = K Q^T: a lane then holds one query (column) and 4 tokens
// (rows) per 16 x 16 tile, which is how O^T = V^T P^T takes P^T as its second
// factor, so P never leaves the registers, and the running maximum, the sum
// and the rescaling of O^T are per-lane scalars. The order of the tokens
// inside a product is free: lane group g's 8 tokens are 4 g .. 4 g + 3 of
// each half of a 32-token slice, and V^T is read from LDS in the same order
// (bfloat16 through the transposing LDS read).
//
// Work: a tile is WK slices of tokens of one (request, key head, block of MT
// queries), an item the tiles of one such triple. The tiles of the whole
// batch form one list, cut into equal spans, one per workgroup, whatever the
// requests' lengths: each workgroup finds its span with a scan over the requests.
// An item inside one span is finished there; the pieces of an item that
// spans several go to scratch (reference, weight, sum) and a second kernel
// joins them. (Pieces handed over inside the launch, the worker of an item's
// first tiles waiting for the others, took 27 instead of 17 us for one
// request of 1024 tokens and 169 instead of 112 us for two long ones: three
// trips between XCDs one after another, and one workgroup to join 32
// pieces.) WQ waves share a slice and split the queries; the WK slices of a tile go
// to different waves, joined through LDS at the end of an item. With few
// queries (WQ = 1) waves share nothing and meet no barrier in the loop.
//
// Few queries are bound by HBM, many by waiting: waves that share a slice
// meet at every tile, some with two blocks of 16 queries and some with one
// (trees: a wave waits 44 % of its time and waits to issue another 26 %;
// matrix units are busy 53,000 of about 250,000 cycles, vector instructions
// take 74,000). On one MI355X, key heads of 128 columns, bfloat16:
//   128 requests x 5 rows, 200-1019 tokens, 40 / 8 heads   98 us  3.4 TB/s
//     (the loads alone 69; joining and storing 1024 items about 25)
//   2 requests x 3-8 rows, 49-65 thousand tokens, 64 / 8  108 us  4.3 TB/s
//   16 trees of 20-50 rows, 1-8 thousand tokens, 40 / 8   134 us  390 TFLOP/s
//     (the loads alone 63)
#include <type_traits>
#include <utility>

#include "attention.hpp"
#include "tree.hpp"
#include "vspec_verify.h"

namespace vsv {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kSlice = 32;     // tokens a wave takes at a time
// Spans move to an item's border within a kSnap-th of their length: 128
// requests of 200 to 1019 tokens take 100 us so, 108 with even cuts, 98 with
// a third, which costs 16 long trees 150 instead of 141.
constexpr int kSnap = 5;
constexpr int kPages = 1024;   // pages looked up at a time

// One 16 x 16 product over 32 of the inner dimension: lane l holds 8 inner
// elements of row (column) l % 16, the same 8 in both factors.
template <typename E> struct Frag;
template <> struct Frag<uint16_t> {
  using T = bf16x8;
  __device__ static __forceinline__ f32x4 mma(T a, T b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  __device__ static __forceinline__ T zero() { return T{}; }
  __device__ static __forceinline__ T load(const uint16_t* p) { return *reinterpret_cast<const T*>(p); }
  // P is rounded to bfloat16 for the product with V, as the matrix unit takes
  // both factors in one type: each weight is off by half a step, 2^-8 of it at
  // most, at random, about what the result's own rounding costs. The weights'
  // sum is taken before the rounding.
  __device__ static __forceinline__ T pack(const float* p) {
    T r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = static_cast<__bf16>(p[e]);
    return r;
  }
};
template <> struct Frag<float> {
  using T = f32x8;
  // eight products over 4: product e takes element e of every lane group
  __device__ static __forceinline__ f32x4 mma(T a, T b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
  __device__ static __forceinline__ T zero() { return T{}; }
  __device__ static __forceinline__ T load(const float* p) {
    const f32x4 lo = reinterpret_cast<const f32x4*>(p)[0], hi = reinterpret_cast<const f32x4*>(p)[1];
    return T{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  }
  __device__ static __forceinline__ T pack(const float* p) {
    return T{p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7]};
  }
};

// Shape of an instantiation.
template <typename E, int D, int QT, int WQ, int WK>
struct Shape {
  static constexpr int kThreads = WQ * WK * kWave;
  static constexpr int kMT = 16 * QT * WQ;           // queries of an item
  // Steps of a slice: fewer barriers where waves share it (256 queries: four
  // took 135 us on 16 trees, two 142, one 157).
  static constexpr int kSub = WQ == 8 && D * static_cast<int>(sizeof(E)) <= 256 ? 4 : WK == 1 ? 2 : 1;
  static constexpr int kTokens = kSlice * kSub;      // tokens of a slice
  static constexpr int kTile = WK * kTokens;         // tokens of a tile
  static constexpr int kRowBytes = D * static_cast<int>(sizeof(E));
  static constexpr int kChunks = kRowBytes / 16;     // 16-byte chunks of a token's row
  static constexpr int kSliceBytes = kTokens * kRowBytes;
  static constexpr int kLoads = kSliceBytes / 16 / (kWave * WQ);   // chunks a lane brings of K (and of V)
  // Two workgroups of four waves share a CU where the LDS holds both, which
  // hides what each does between its items. Waves that share nothing keep one
  // buffer and refill its halves as they are read; the others keep a ring.
  static constexpr int kGroups = kThreads == 256 && WK * kSliceBytes * (WQ == 1 ? 1 : 2) <= 32 * 1024 ? 2 : 1;
  static constexpr int kWaves = kGroups * kThreads / 256;   // a SIMD's waves
  static constexpr int kFit = 128 * 1024 / (kGroups * WK * kSliceBytes * 2);
  static constexpr int kStages = WQ == 1 ? 1 : kFit > 4 ? 4 : kFit;
  static_assert(WQ == 1 || kStages >= 2, "shared slices are brought ahead");
  static_assert(kLoads <= (kChunks == 8 ? 8 : 16), "a lane of 16 for every load");
  // The row of the slice whose place lane (grp, col) of wave wq works out.
  __device__ static __forceinline__ int owned_row(int wq, int grp, int col) {
    return kChunks == 8    ? wq * 8 + 2 * grp + (col & 1) + (col >> 1) * 8 * WQ
           : kChunks == 16 ? wq * 4 + grp + col * 4 * WQ
                           : wq * 2 + (grp >> 1) + col * 2 * WQ;
  }
  static constexpr int kOutStride = D + 4;           // of a joined row of O, off the banks' period
};

struct Request {
  int r0, n, len, tiles, blocks;   // rows, context, tiles of an item, blocks of queries
};

template <typename E, int D, int QT, int WQ, int WK>
struct alignas(16) AttnScratch {
  using S = Shape<E, D, QT, WQ, WK>;
  union {
    struct {
      uint32_t k[S::kSliceBytes / 4];
      uint32_t v[S::kSliceBytes / 4];
    } tile[S::kStages][WK];
    float join[WK][S::kMT][S::kOutStride];
  };
  int page[kPages];   // the pages of the tiles at hand
  float ml[WK][S::kMT][2];
  float fin[S::kMT][2];
  int64_t out_at[S::kMT];  // where a query's result goes
  int lse_at[S::kMT];
  uint64_t path[VSV_MAX_TREE_ROWS];
  int64_t scan[S::kThreads / kWave];
  int64_t base;
  int64_t cut[2];
  int request;
  Request first;
  int odd;   // a value among the rows' own is not finite
};

// Where chunk c of token row r lies in its slice. Rows are 128 bytes or more
// apart, so lanes that read one column of many rows would meet in the same
// banks: the chunks of a row are permuted by an exclusive or. Keys are read
// 16 rows at a time, a chunk each; values 8 rows of two chunks (bfloat16,
// transposed) or 4 rows, four apart, of four chunks (float32).
template <int C>
__device__ __forceinline__ int swizzle_k(int r) {
  return C == 8 ? (r >> 1) & 7 : r & 15;
}
template <typename E, int C>
__device__ __forceinline__ int swizzle_v(int r) {
  if (sizeof(E) == 4) return 4 * ((r >> 2) & 3);
  return C == 8 ? 2 * ((r >> 1) & 3) : 2 * (r & 7);
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  int2 h = __builtin_bit_cast(int2, v);
  h.x = __builtin_amdgcn_readfirstlane(h.x);
  h.y = __builtin_amdgcn_readfirstlane(h.y);
  return __builtin_bit_cast(int64_t, h);
}

template <int NT>
__device__ __forceinline__ int64_t block_scan64(int64_t v, int64_t* scratch, int64_t& total) {
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const int64_t incl = wave_scan_incl(v);
  lds_barrier();
  if (lane == kWave - 1) scratch[w] = incl;
  lds_barrier();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int k = 0; k < NT / kWave; ++k) {
    const int64_t s = scratch[k];
    before += k < w ? s : 0;
    total += s;
  }
  return before + incl - v;
}

template <typename S>
__device__ __forceinline__ Request request_of(const AttentionArgs& a, int i, bool& bad) {
  // (inputs no kernel writes: uniform ones come through the scalar cache)
  typedef const __attribute__((address_space(4))) int32_t* Constant;
  const int r0 = ((Constant)a.offsets)[i], r1 = ((Constant)a.offsets)[i + 1], len = ((Constant)a.length)[i];
  const int64_t room = static_cast<int64_t>(a.table_width) << a.page_shift;
  bad = r0 < 0 || r1 < r0 || r1 > a.R || r1 - r0 > VSV_MAX_TREE_ROWS || len < 0 || len > room;
  Request q{r0, r1 - r0, len, 0, 0};
  if (bad) q.n = 0;
  if (q.n > 0) {
    q.tiles = static_cast<int>((static_cast<int64_t>(len) + q.n + S::kTile - 1) / S::kTile);
    q.blocks = (q.n * a.G + S::kMT - 1) / S::kMT;
  }
  return q;
}

// Start of a worker's span in a list of `units`; no more workers than units,
// so that every span holds something.
__device__ __forceinline__ int64_t span_start(int64_t units, int w, int workers) {
  return units * w / workers;
}

__device__ __forceinline__ bool not_finite(uint32_t two, std::integral_constant<int, 2>) {
  return (two & 0x7F80u) == 0x7F80u || (two & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ bool not_finite(uint32_t one, std::integral_constant<int, 4>) {
  return (one & 0x7F800000u) == 0x7F800000u;
}

// A load of 16 bytes a lane straight into LDS, at `to` + 16 * lane. The
// compiler makes every later LDS read wait for its own form of this load, the
// reads of the other buffer included; here the wait is wait_loads() alone.
// (m0 is reserved: the compiler keeps no value in it, so it is not named among
// what is written, and it writes m0 nowhere else in these kernels.)
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)p));
}
__device__ __forceinline__ void load_to_lds(int64_t from, uint32_t to) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "s"(to), "v"(from)
      : "memory");
}
// Wait until at most N of the wave's loads are under way (they end in order),
// and for the LDS accesses it issued.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
// The same for all of them in a form that the compiler counts: its own loads
// (the queries) are then known to have ended, and it puts no wait of its own,
// which would be one for the tiles under way, before their uses in the loop.
__device__ __forceinline__ void drain() {
  __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0)
  wait_loads<0>();
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <int... K, typename F>
__device__ __forceinline__ void for_each_index(std::integer_sequence<int, K...>, F&& f) {
  (f(std::integral_constant<int, K>()), ...);
}

// The value of lane K of the lane's group of 16; for rows of 8 chunks, of
// lane 2 K for the group's lower half and of 2 K + 1 for its upper one.
template <int K, int C>
__device__ __forceinline__ int64_t group_broadcast(int64_t v) {
  constexpr int kBroadcast = 0x150;   // DPP row_newbcast of lane 0
  int2 h = __builtin_bit_cast(int2, v), o;
  if constexpr (C == 8) {
    o.x = __builtin_amdgcn_update_dpp(0, h.x, kBroadcast + 2 * K, 0xF, 0x3, false);
    o.y = __builtin_amdgcn_update_dpp(0, h.y, kBroadcast + 2 * K, 0xF, 0x3, false);
    o.x = __builtin_amdgcn_update_dpp(o.x, h.x, kBroadcast + 2 * K + 1, 0xF, 0xC, false);
    o.y = __builtin_amdgcn_update_dpp(o.y, h.y, kBroadcast + 2 * K + 1, 0xF, 0xC, false);
  } else {
    o.x = __builtin_amdgcn_update_dpp(0, h.x, kBroadcast + K, 0xF, 0xF, false);
    o.y = __builtin_amdgcn_update_dpp(0, h.y, kBroadcast + K, 0xF, 0xF, false);
  }
  return __builtin_bit_cast(int64_t, o);
}

// Weight of sums taken relative to m where the common reference is `top`
// (sums without a reference are 0).
__device__ __forceinline__ float weight_of(float m, float top) { return m == -INFINITY ? 1.f : fast_exp2(m - top); }

__device__ __forceinline__ void store_out(uint16_t* p, f32x4 o) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<bf16x4*>(p) = bf16x4{static_cast<__bf16>(o[0]), static_cast<__bf16>(o[1]), static_cast<__bf16>(o[2]),
                                         static_cast<__bf16>(o[3])};
}
__device__ __forceinline__ void store_out(float* p, f32x4 o) { *reinterpret_cast<f32x4*>(p) = o; }

// LDS written by this wave and read by its other lanes.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <typename E, int D, int QT, int WQ, int WK>
__global__ __launch_bounds__((Shape<E, D, QT, WQ, WK>::kThreads), (Shape<E, D, QT, WQ, WK>::kWaves))
void attention_kernel(AttentionArgs a) {
  using S = Shape<E, D, QT, WQ, WK>;
  using F = Frag<E>;
  constexpr int kThreads = S::kThreads;
  constexpr int C = S::kChunks;
  constexpr int KC = D / 32;    // inner steps of K Q^T
  constexpr int DT = D / 16;    // row blocks of O^T
  __shared__ AttnScratch<E, D, QT, WQ, WK> s;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int wq = wave % WQ, wk = wave / WQ;
  const int col = lane & 15, grp = lane >> 4;
  const int w = blockIdx.x;
  int bits = 0;

  // ---- this worker's span: the sum over the requests, then the request that
  // holds the span's start (in the same pass where each has a thread)
  int64_t units = 0, before = 0, size0 = 0;
  Request mine0{};
  for (int base = 0; base < a.B; base += kThreads) {
    const int i = base + tid;
    size0 = 0;
    if (i < a.B) {
      bool bad;
      mine0 = request_of<S>(a, i, bad);
      if (bad) bits |= VSV_FLAG_LAYOUT;
      size0 = static_cast<int64_t>(a.KV) * mine0.blocks * mine0.tiles;
    }
    int64_t total;
    before = units + block_scan64<kThreads>(size0, s.scan, total);
    units += total;
  }
  if (w == 0 && bits && a.error_flag) atomicOr(a.error_flag, bits);
  bits = 0;
  if (tid == 0) a.piece[w].x = -1;
  const int workers = static_cast<int>(min(static_cast<int64_t>(a.workers), units));
  if (w >= workers) return;
  units = uniform64(units);
  // where the even cut falls close to an item's start or end, the item stays whole
  const int64_t slack = units / workers / kSnap;
  const int64_t even[2] = {span_start(units, w, workers), w + 1 < workers ? span_start(units, w + 1, workers) : units - 1};
  auto locate = [&](int i, int64_t before, int64_t size, const Request& q) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (before <= even[k] && even[k] < before + size) {
        const int64_t in_item = (even[k] - before) % q.tiles;
        int64_t at = even[k];
        if (in_item <= slack)
          at -= in_item;
        else if (q.tiles - in_item <= slack)
          at += q.tiles - in_item;
        s.cut[k] = w + 1 < workers || k == 0 ? at : units;
        if (k == 0) {
          s.request = i;
          s.base = before;
          s.first = q;
        }
      }
    }
  };
  if (a.B > kThreads) {
    int64_t seen = 0;
    for (int base = 0; base < a.B && seen <= even[1]; base += kThreads) {
      const int i = base + tid;
      size0 = 0;
      if (i < a.B) {
        bool bad;
        mine0 = request_of<S>(a, i, bad);
        size0 = static_cast<int64_t>(a.KV) * mine0.blocks * mine0.tiles;
      }
      int64_t total;
      before = seen + block_scan64<kThreads>(size0, s.scan, total);
      seen += total;
      locate(i, before, size0, mine0);
    }
  } else {
    locate(tid, before, size0, mine0);
  }
  lds_barrier();
  const int64_t u0 = uniform64(s.cut[0]), u1 = uniform64(s.cut[1]);
  if (u0 >= u1) return;
  int i = __builtin_amdgcn_readfirstlane(s.request);
  int64_t base = uniform64(s.base);
  Request rq = s.first;
  rq.r0 = __builtin_amdgcn_readfirstlane(rq.r0);
  rq.n = __builtin_amdgcn_readfirstlane(rq.n);
  rq.len = __builtin_amdgcn_readfirstlane(rq.len);
  rq.tiles = __builtin_amdgcn_readfirstlane(rq.tiles);
  rq.blocks = __builtin_amdgcn_readfirstlane(rq.blocks);

  // ---- the items of the span
  for (int64_t u = u0; u < u1;) {
    const int64_t size = static_cast<int64_t>(a.KV) * rq.blocks * rq.tiles;
    if (u >= base + size) {
      base += size;
      ++i;
      bool bad;
      rq = request_of<S>(a, i, bad);
      continue;
    }
    const uint32_t rel = static_cast<uint32_t>(u - base);
    const int item = static_cast<int>(rel / static_cast<uint32_t>(rq.tiles));
    const int t0 = static_cast<int>(rel) - item * rq.tiles;
    const int h = item / rq.blocks, mt = item - h * rq.blocks;
    const int t1 = static_cast<int>(min(static_cast<int64_t>(rq.tiles), t0 + (u1 - u)));
    u += t1 - t0;

    const int r0 = rq.r0, n = rq.n, len = rq.len, end = len + n;
    const int M = min(n * a.G - mt * S::kMT, S::kMT);   // queries of this block

    // ---- staging: chunk c of the slice is chunk c % C of its token c / C,
    // brought by lane c % (64 WQ) of the waves that share it. Loads go to LDS
    // without a register: a wave instruction fills 64 chunks in a row, so the
    // permutation of a token's chunks is one of the addresses it reads.
    const char* kc_base = static_cast<const char*>(a.k_cache) + h * a.c_head * static_cast<int64_t>(sizeof(E));
    const char* vc_base = static_cast<const char*>(a.v_cache) + h * a.c_head * static_cast<int64_t>(sizeof(E));
    const char* kr_base = static_cast<const char*>(a.k) + (r0 * a.k_row + h * a.k_head) * static_cast<int64_t>(sizeof(E));
    const char* vr_base = static_cast<const char*>(a.v) + (r0 * a.v_row + h * a.v_head) * static_cast<int64_t>(sizeof(E));
    const int32_t* row_table = a.table + static_cast<int64_t>(i) * a.table_ld;
    const int page_mask = (1 << a.page_shift) - 1;
    const int slot0 = wq * kWave + lane;   // this lane's first chunk
    // Each lane knows the place of one token: the one that load k brings to
    // the lane's group of 16 (the half group, for rows of 8 chunks) is that
    // of the group's lane k (2 k, 2 k + 1), and a broadcast inside the group
    // hands it on.
    const int my_row = min(S::owned_row(wq, grp, col), S::kTokens - 1);
    // The pages of tiles tc .. te - 1, by the whole workgroup.
    auto look_up = [&](int tc, int te) {
      const int p0 = tc * S::kTile >> a.page_shift;
      const int count = ((min(te * S::kTile, len) - 1) >> a.page_shift) + 1 - p0;
      for (int p = tid; p < count; p += kThreads) {
        int id = row_table[p0 + p];
        if (id < 0 || id >= a.num_pages) {
          bits |= VSV_FLAG_PAGES;
          id = 0;
        }
        s.page[p] = id;
      }
    };
    // The place of this lane's token of tile t (keys, values).
    auto place = [&](int t, int p0, int64_t& kp, int64_t& vp) {
      const int x = t * S::kTile + wk * S::kTokens + my_row;
      const int own = min(max(x - len, 0), n - 1);   // behind the last token: any row that exists
      kp = reinterpret_cast<int64_t>(kr_base) + own * a.k_row * static_cast<int64_t>(sizeof(E));
      vp = reinterpret_cast<int64_t>(vr_base) + own * a.v_row * static_cast<int64_t>(sizeof(E));
      const int id = s.page[x < len ? (x >> a.page_shift) - p0 : 0];
      const int64_t cached = (id * a.c_page + (x & page_mask) * a.c_token) * static_cast<int64_t>(sizeof(E));
      kp = x < len ? reinterpret_cast<int64_t>(kc_base) + cached : kp;
      vp = x < len ? reinterpret_cast<int64_t>(vc_base) + cached : vp;
    };
    auto fetch_k = [&](int t, int64_t kp) {
      const uint32_t kd = __builtin_amdgcn_readfirstlane(lds_address(s.tile[t % S::kStages][wk].k) + wq * kWave * 16);
      for_each_index(std::make_integer_sequence<int, S::kLoads>(), [&](auto index) {
        constexpr int k = decltype(index)::value;
        const int c = slot0 + k * kWave * WQ;
        load_to_lds(group_broadcast<k, C>(kp) + (c % C ^ swizzle_k<C>(c / C)) * 16, kd + k * kWave * WQ * 16);
      });
    };
    auto fetch_v = [&](int t, int64_t vp) {
      const uint32_t vd = __builtin_amdgcn_readfirstlane(lds_address(s.tile[t % S::kStages][wk].v) + wq * kWave * 16);
      for_each_index(std::make_integer_sequence<int, S::kLoads>(), [&](auto index) {
        constexpr int k = decltype(index)::value;
        const int c = slot0 + k * kWave * WQ;
        load_to_lds(group_broadcast<k, C>(vp) + (c % C ^ swizzle_v<E, C>(c / C)) * 16, vd + k * kWave * WQ * 16);
      });
    };
    // Values of the rows' own that are not finite would reach rows that do not see
    // them through a weight of 0, and so would what lies behind the last
    // token: both are 0 in the tile (the former are added at the end).
    auto clean = [&](int t) {
      u32x4* vl = reinterpret_cast<u32x4*>(s.tile[t % S::kStages][wk].v);
#pragma unroll 1
      for (int k = 0; k < S::kLoads; ++k) {
        const int c = slot0 + k * kWave * WQ;
        const int x = t * S::kTile + wk * S::kTokens + c / C;
        if (x < len) continue;
        u32x4 v = vl[c];
        bool odd = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) odd |= not_finite(v[e], std::integral_constant<int, sizeof(E)>());
        if (!odd && x < end) continue;
        if (x < end) s.odd = 1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (sizeof(E) == 2) {
            if ((v[e] & 0x7F80u) == 0x7F80u) v[e] &= 0xFFFF0000u;
            if ((v[e] & 0x7F800000u) == 0x7F800000u) v[e] &= 0xFFFFu;
          } else if ((v[e] & 0x7F800000u) == 0x7F800000u) {
            v[e] = 0;
          }
          if (x >= end) v[e] = 0;
        }
        vl[c] = v;
      }
    };

    // first loads: pages, parents, queries
    const int tiles_per_look = ((kPages - 1) << min(a.page_shift, 16)) / S::kTile;   // one page may be cut at its start
    int te = min(t1, t0 + tiles_per_look);
    look_up(t0, te);
    const int up = wave == 0 && a.parents && lane < n ? a.parents[r0 + lane] : 0;
    // ---- queries
    typename F::T qf[QT][KC];
    int row[QT];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
      const int m = (qt * WQ + wq) * 16 + col;
      const bool live = m < M;
      const int at = mt * S::kMT + (live ? m : 0);
      const int j = at / a.G, hq = h * a.G + (at - j * a.G);
      const E* p = static_cast<const E*>(a.q) + (r0 + j) * a.q_row + hq * a.q_head + grp * 8;
#pragma unroll
      for (int kc = 0; kc < KC; ++kc) qf[qt][kc] = live ? F::load(p + kc * 32) : F::zero();
      row[qt] = live ? j : -1;
    }

    for (int q = tid; q < M; q += kThreads) {
      const int at = mt * S::kMT + q, j = at / a.G, hq = h * a.G + (at - j * a.G);
      s.out_at[q] = (r0 + j) * a.o_row + hq * a.o_head;
      s.lse_at[q] = (r0 + j) * a.H + hq;
    }
    if (wave == 0) {
      bool off_tree;
      s.path[lane] = tree_paths(lane, n, up, a.parents == nullptr, off_tree);
      if (off_tree) bits |= VSV_FLAG_LAYOUT;
      if (lane == 0) s.odd = 0;
    }
    lds_barrier();
    uint64_t path[QT];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) path[qt] = row[qt] >= 0 ? s.path[row[qt]] : 0;

    f32x4 acc[DT][QT];
    float mref[QT], mc[QT], l[QT];   // reference, times the scale (0 while there is none), weights so far
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
      mref[qt] = -INFINITY;
      mc[qt] = 0.f;
      l[qt] = 0.f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) acc[dt][qt] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // One tile of this wave's slice, for its first NQ blocks of 16 queries.
    // `between` runs when the keys have been read, before the values are.
    // Where waves share slices, and so meet in step at every tile, what a
    // step reads from LDS is read a phase ahead (its values before the
    // softmax, the next step's keys before the product with the values): 135
    // instead of 139 us on 16 trees.
    constexpr bool kAhead = WQ > 1 && sizeof(E) == 2 && D <= 128;
    auto compute = [&](auto live, int t, auto between) {
      constexpr int NQ = decltype(live)::value;
      const int x0 = t * S::kTile + wk * S::kTokens;
      const char* kl = reinterpret_cast<const char*>(s.tile[t % S::kStages][wk].k);
      const char* vl = reinterpret_cast<const char*>(s.tile[t % S::kStages][wk].v);
      auto key = [&](int sub, int hf, int kc) -> typename F::T {
        const int row = sub * kSlice + hf * 16 + col, z = swizzle_k<C>(row);
        if constexpr (sizeof(E) == 2) {
          return *reinterpret_cast<const bf16x8*>(kl + (row * C + ((kc * 4 + grp) ^ z)) * 16);
        } else {
          const int c0 = kc * 8 + grp * 2;
          const f32x4 lo = *reinterpret_cast<const f32x4*>(kl + (row * C + (c0 ^ z)) * 16);
          const f32x4 hi = *reinterpret_cast<const f32x4*>(kl + (row * C + ((c0 + 1) ^ z)) * 16);
          return f32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        }
      };
      auto value = [&](int sub, int dt) -> typename F::T {
        typename F::T v;
        if constexpr (sizeof(E) == 2) {
          s16x4 half[2];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int row = sub * kSlice + hf * 16 + grp * 4 + (col >> 2);
            const int chunk = dt * 2 + ((col & 3) >> 1);
            const char* p = vl + (row * C + (chunk ^ swizzle_v<E, C>(row))) * 16 + (col & 1) * 8;
            half[hf] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)(const_cast<char*>(p)));
          }
          v = __builtin_bit_cast(bf16x8, s16x8{half[0][0], half[0][1], half[0][2], half[0][3], half[1][0], half[1][1],
                                               half[1][2], half[1][3]});
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int row = sub * kSlice + (e >> 2) * 16 + grp * 4 + (e & 3);
            const int chunk = dt * 4 + (col >> 2);
            v[e] = *reinterpret_cast<const float*>(vl + (row * C + (chunk ^ swizzle_v<E, C>(row))) * 16 + (col & 3) * 4);
          }
        }
        return v;
      };
      typename F::T kf[kAhead ? 2 : 1][kAhead ? KC : 1], vf[kAhead ? DT : 1];
      auto keys_ahead = [&](int sub) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int kc = 0; kc < KC; ++kc) kf[hf][kc] = key(sub, hf, kc);
      };
      if constexpr (kAhead) keys_ahead(0);
#pragma unroll
      for (int sub = 0; sub < S::kSub; ++sub) {
        // S^T of two halves of 16 tokens
        f32x4 sc[2][NQ];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
          for (int qt = 0; qt < NQ; ++qt) sc[hf][qt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int kc = 0; kc < KC; ++kc) {
            typename F::T k;
            if constexpr (kAhead)
              k = kf[hf][kc];
            else
              k = key(sub, hf, kc);
#pragma unroll
            for (int qt = 0; qt < NQ; ++qt) sc[hf][qt] = F::mma(k, qf[qt][kc], sc[hf][qt]);
          }
        }
        if constexpr (kAhead) {
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) vf[dt] = value(sub, dt);
        }
        // tokens from the tree on: only the row's path is seen
        const int xs = x0 + sub * kSlice;
        if (xs + kSlice > len) {
#pragma unroll
          for (int qt = 0; qt < NQ; ++qt) {
            // bit k: the lane's query sees token k of the step
            const int first = xs - len;   // of the rows' own
            const uint32_t seen = first >= 0 ? (first < 64 ? static_cast<uint32_t>(path[qt] >> first) : 0u)
                                             : (static_cast<uint32_t>(path[qt]) << -first) | ((1u << -first) - 1u);
            const uint32_t mine = seen >> (grp * 4);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[hf][qt][e] = mine & (1u << (hf * 16 + e)) ? sc[hf][qt][e] : -INFINITY;
          }
        }
        // The reference moves only where a score passes it by more than kSlack
        // in log2: weights stay below 2^kSlack, and most tiles skip the
        // reduction across lanes and the rescaling.
        constexpr float kSlack = 8.f;
        typename F::T pf[NQ];
        bool move = false;
        float top[NQ];
#pragma unroll
        for (int qt = 0; qt < NQ; ++qt) {
          float b = sc[0][qt][0];
#pragma unroll
          for (int e = 1; e < 8; ++e) b = fmaxf(b, sc[e >> 2][qt][e & 3]);
          top[qt] = b;
          move |= b * a.scale > mref[qt] * a.scale + kSlack;   // false while both are -inf
        }
        if (__builtin_amdgcn_ballot_w64(move)) {
#pragma unroll
          for (int qt = 0; qt < NQ; ++qt) {
            float b = fmaxf(top[qt], mref[qt]);
            b = fmaxf(b, __shfl_xor(b, 16));
            b = fmaxf(b, __shfl_xor(b, 32));
            const float f = b == mref[qt] ? 1.f : fast_exp2((mref[qt] - b) * a.scale);
            mref[qt] = b;
            mc[qt] = b == -INFINITY ? 0.f : b * a.scale;
            l[qt] *= f;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) acc[dt][qt] *= f;
          }
        }
#pragma unroll
        for (int qt = 0; qt < NQ; ++qt) {
          float p[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            p[e] = fast_exp2(fmaf(sc[e >> 2][qt][e & 3], a.scale, -mc[qt]));
            l[qt] += p[e];
          }
          pf[qt] = F::pack(p);
        }
        between();
        if constexpr (kAhead) {
          if (sub + 1 < S::kSub) keys_ahead(sub + 1);
        }
        // O^T += V^T P^T
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          typename F::T v;
          if constexpr (kAhead)
            v = vf[dt];
          else
            v = value(sub, dt);
#pragma unroll
          for (int qt = 0; qt < NQ; ++qt) acc[dt][qt] = F::mma(v, pf[qt], acc[dt][qt]);
        }
      }
    };
    const int blocks = (M + 15) / 16;   // of 16 queries, dealt to the waves in turn
    const int mine = blocks > wq ? (blocks - wq + WQ - 1) / WQ : 0;

    for (int tc = t0; tc < t1;) {
      if (tc > t0) {
        lds_barrier();   // the pages before have been read
        te = min(t1, tc + tiles_per_look);
        look_up(tc, te);
        lds_barrier();
      }
      const int p0 = tc * S::kTile >> a.page_shift;
      int64_t kp, vp;
      if constexpr (WQ == 1) {
        // one buffer: the next keys are under way as soon as these have been
        // read, the next values behind the product with these
        place(tc, p0, kp, vp);
        drain();
        fetch_k(tc, kp);
        fetch_v(tc, vp);
        for (int t = tc; t < te; ++t) {
          const int x0 = t * S::kTile + wk * S::kTokens;
          const bool more = t + 1 < te;
          wait_loads<S::kLoads>();
          if (more) place(t + 1, p0, kp, vp);
          auto between = [&]() {
            if (more) {
              wait_lds();
              fetch_k(t + 1, kp);
              wait_loads<S::kLoads>();
            } else {
              wait_loads<0>();
            }
            if (x0 + S::kTokens > len) clean(t);
            wave_sync();
          };
          if (x0 < end)
            compute(std::integral_constant<int, QT>(), t, between);
          else
            between();   // the slice lies behind the last token
          if (more) {
            wait_lds();
            fetch_v(t + 1, vp);
          }
        }
      } else {
        // a ring of kStages tiles, of which kStages - 1 are under way
        constexpr int L = 2 * S::kLoads, N = S::kStages;
        drain();
        for (int t = tc; t < min(te, tc + N - 1); ++t) {
          place(t, p0, kp, vp);
          fetch_k(t, kp);
          fetch_v(t, vp);
        }
        for (int t = tc; t < te; ++t) {
          const int behind = min(te - 1 - t, N - 2);   // tiles under way behind this one
          if (N > 3 && behind == 2)
            wait_loads<2 * L>();
          else if (N > 2 && behind == 1)
            wait_loads<L>();
          else
            wait_loads<0>();
          const int x0 = t * S::kTile + wk * S::kTokens;
          if (x0 + S::kTokens > len) clean(t);
          lds_barrier();
          if (t + N - 1 < te) {
            // into the buffer of tile t - 1, which every wave has read
            place(t + N - 1, p0, kp, vp);
            fetch_k(t + N - 1, kp);
            fetch_v(t + N - 1, vp);
          }
          if (x0 >= end || mine == 0) continue;   // a slice behind the last token, or no query
          if (QT == 2 && mine == 1)
            compute(std::integral_constant<int, 1>(), t, [] {});
          else
            compute(std::integral_constant<int, QT>(), t, [] {});
        }
      }
      tc = te;
      if (tc < t1 && WQ > 1) lds_barrier();   // the ring starts anew
    }

    // ---- join the slices of the workgroup
    const bool first = t0 == 0, last = t1 == rq.tiles;
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
      l[qt] += __shfl_xor(l[qt], 16);
      l[qt] += __shfl_xor(l[qt], 32);
      if (grp == 0) {
        const int q = (qt * WQ + wq) * 16 + col;
        s.ml[wk][q][0] = mref[qt];
        s.ml[wk][q][1] = l[qt];
      }
    }
    lds_barrier();   // (and the tiles have been read)
    const bool odd = s.odd != 0;
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
      const int q = (qt * WQ + wq) * 16 + col;
      float m = -INFINITY;
#pragma unroll
      for (int k = 0; k < WK; ++k) m = fmaxf(m, s.ml[k][q][0]);
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        const float mk = s.ml[k][q][0];
        sum += mk == -INFINITY ? s.ml[k][q][1] : s.ml[k][q][1] * fast_exp2((mk - m) * a.scale);
      }
      const float f = mref[qt] == -INFINITY ? 1.f : fast_exp2((mref[qt] - m) * a.scale);
      if (grp == 0 && wk == 0) {
        s.fin[q][0] = m * a.scale;
        s.fin[q][1] = sum;
      }
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) *reinterpret_cast<f32x4*>(&s.join[wk][q][dt * 16 + grp * 4]) = acc[dt][qt] * f;
    }
    lds_barrier();
    constexpr int kQuads = D / 4;
    // this workgroup's part of 4 columns of a query
    auto part = [&](int q, int d) {
      f32x4 o = *reinterpret_cast<const f32x4*>(&s.join[0][q][d]);
#pragma unroll
      for (int k = 1; k < WK; ++k) o += *reinterpret_cast<const f32x4*>(&s.join[k][q][d]);
      if (odd) {
        // values that are not finite, for the rows that see them
        const uint64_t seen_rows = s.path[(mt * S::kMT + q) / a.G];
        for (int x = max(t0 * S::kTile, len); x < min(t1 * S::kTile, end); ++x) {
          if (!(seen_rows >> (x - len) & 1)) continue;
          const E* p = static_cast<const E*>(a.v) + static_cast<int64_t>(r0 + x - len) * a.v_row + h * a.v_head;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float f = Elem<E>::at(p, d + e);
            if (!(fabsf(f) < INFINITY)) o[e] += f;
          }
        }
      }
      return o;
    };
    const int64_t at = static_cast<int64_t>(first ? 2 * w + 1 : 2 * w) * S::kMT;   // of a piece
    for (int c = tid; c < M * kQuads; c += kThreads) {
      const int q = c / kQuads, d = c % kQuads * 4;
      const f32x4 o = part(q, d);
      if (first && last) {
        const float m = s.fin[q][0], sum = s.fin[q][1];
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);   // a NaN stays one
        store_out(static_cast<E*>(a.out) + s.out_at[q] + d, o * inv);
        if (d == 0 && a.lse) a.lse[s.lse_at[q]] = 0.69314718f * (m + __log2f(sum));
      } else {
        *reinterpret_cast<f32x4*>(a.part + (at + q) * D + d) = o;
        if (d == 0) a.part_ml[at + q] = make_float2(s.fin[q][0], s.fin[q][1]);
      }
    }
    if (first && !last && tid == 0) {
      // the worker whose span holds the item's last tile: the last one whose
      // span starts before the item's end, and not so close that it starts there
      const int64_t end_unit = u + (rq.tiles - t1) - 1 - slack;
      int x = static_cast<int>(((end_unit + 1) * workers - 1) / units);
      while (x + 1 < workers && span_start(units, x + 1, workers) <= end_unit) ++x;
      while (span_start(units, x, workers) > end_unit) --x;
      a.piece[w] = make_int4(r0, h, mt, x * 512 + M);
    }
    lds_barrier();   // paths and joined columns are free again
  }
  if (bits && a.error_flag) atomicOr(a.error_flag, bits);
}

// Joins the pieces of the items that no worker finished: a wave per query,
// D / 4 lanes for 4 columns each and the pieces dealt to 256 / D groups of
// them. Every workgroup lists the items that were cut, wherever they are, so
// that few long items and many short ones keep the whole grid busy alike.
constexpr int kJoinThreads = 256;
constexpr int kMaxWorkers = 1024;
constexpr int kJoinGroups = 2048;

template <typename E, int D, int MT>
__global__ __launch_bounds__(kJoinThreads) void attention_join_kernel(AttentionArgs a) {
  constexpr int kLanes = D / 4;             // lanes of a piece
  constexpr int kSets = kWave / kLanes;     // pieces side by side
  constexpr int kAhead = 4;                 // rounds of pieces loaded at a time
  __shared__ int4 cut[kMaxWorkers];   // first row, key head, block, worker * 2^20 + last worker * 2^9 + queries
  __shared__ int scan[kJoinThreads / kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  int count = 0;
  for (int base = 0; base < a.workers; base += kJoinThreads) {
    const int w = base + tid;
    int4 p = make_int4(-1, 0, 0, 0);
    if (w < a.workers) p = a.piece[w];
    const bool here = p.x >= 0;
    int found;
    const int at = count + block_exclusive_scan<kJoinThreads>(here ? 1 : 0, scan, found);
    if (here) cut[at] = make_int4(p.x, p.y, p.z, (w << 20) + p.w);
    count += found;
  }
  lds_barrier();
  const int set = lane / kLanes, d = lane % kLanes * 4;
  constexpr int kWaves = kJoinThreads / kWave;
  const int tasks = count * MT;
  for (int task = static_cast<int>(blockIdx.x) * kWaves + tid / kWave; task < tasks;
       task += static_cast<int>(gridDim.x) * kWaves) {
    // queries of one item go to workgroups far apart, items side by side
    const int q = task / count;
    const int4 p = cut[task - q * count];
    const int w = p.w >> 20, w1 = p.w >> 9 & 2047, M = p.w & 511, r0 = p.x, h = p.y, mt = p.z;
    if (q >= M) continue;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, sum = 0.f;
    for (int x0 = w; x0 <= w1; x0 += kAhead * kSets) {
      float mk[kAhead], lk[kAhead];
      f32x4 ok[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        // the item's start lies in the second slot of worker w, the rest in
        // the first slots of w + 1 .. w1
        const int x = x0 + e * kSets + set;
        mk[e] = -INFINITY;
        lk[e] = 0.f;
        ok[e] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (x <= w1) {
          const int64_t at = static_cast<int64_t>(x == w ? 2 * w + 1 : 2 * x) * MT + q;
          const float2 ml = a.part_ml[at];
          mk[e] = ml.x;
          lk[e] = ml.y;
          ok[e] = *reinterpret_cast<const f32x4*>(a.part + at * D + d);
        }
      }
      float top = m;
#pragma unroll
      for (int e = 0; e < kAhead; ++e) top = fmaxf(top, mk[e]);
      const float old = weight_of(m, top);
      o *= old;
      sum *= old;
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const float f = weight_of(mk[e], top);
        o += f * ok[e];
        sum += f * lk[e];
      }
      m = top;
    }
#pragma unroll
    for (int step = kLanes; step < kWave; step *= 2) {
      const float mo = __shfl_xor(m, step), so = __shfl_xor(sum, step);
      f32x4 oo;
#pragma unroll
      for (int e = 0; e < 4; ++e) oo[e] = __shfl_xor(o[e], step);
      const float top = fmaxf(m, mo);
      const float f = weight_of(m, top), fo = weight_of(mo, top);
      o = f * o + fo * oo;
      sum = f * sum + fo * so;
      m = top;
    }
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    const int at = mt * MT + q, j = at / a.G, hq = h * a.G + (at - j * a.G);
    if (set == 0) store_out(static_cast<E*>(a.out) + (r0 + j) * a.o_row + hq * a.o_head + d, o * inv);
    if (a.lse && lane == 0) a.lse[static_cast<int64_t>(r0 + j) * a.H + hq] = 0.69314718f * (m + __log2f(sum));
  }
}

// ---- launch

// Blocks of queries: the smallest one that holds an average request's
// queries of a key head, so that its keys are read once. (16 trees of 100 to
// 250 queries: 135 us with blocks of 256, 141 with 128, 181 with 64. Four waves
// of 64 queries each instead of eight of 32 took 200: their sums leave the
// vector registers.)
struct Plan {
  int mt, tile;
};
Plan plan_of(const AttentionArgs& a) {
  const int64_t mean = (static_cast<int64_t>(a.R) + a.B - 1) / a.B;
  const int64_t m = mean * (a.H / a.KV);
  if (m <= 16) return {16, 128};
  if (m <= 32) return {32, 128};
  if (m <= 64) return {64, 64};
  // (a row of 256 columns leaves no LDS to join 256 queries in)
  return m <= 128 || a.D > 128 ? Plan{128, 64} : Plan{256, 64};
}
int workers_of(const AttentionArgs& a) {
  const int w = (a.cus > 0 ? a.cus : 256) * 2;
  return w < kMaxWorkers ? w : kMaxWorkers;
}

size_t align256(size_t b) { return (b + 255) / 256 * 256; }

// An instantiation, and what a call of it needs: workgroups, and where the
// parts of its scratch lie.
template <typename E, int D, int QT, int WQ, int WK> struct Kernel {};
struct Scratch {
  int workers;
  size_t part_ml, part, bytes;
};
template <typename E, int D, int QT, int WQ, int WK>
Scratch scratch_of(Kernel<E, D, QT, WQ, WK>, const AttentionArgs& a) {
  using S = Shape<E, D, QT, WQ, WK>;
  Scratch c;
  c.workers = workers_of(a) / 2 * S::kGroups;
  const size_t pieces = static_cast<size_t>(c.workers) * 2 * S::kMT;
  c.part_ml = align256(static_cast<size_t>(c.workers) * sizeof(int4));
  c.part = c.part_ml + align256(pieces * sizeof(float2));
  c.bytes = c.part + align256(pieces * D * sizeof(float));
  return c;
}

template <typename E, int D, int QT, int WQ, int WK>
hipError_t launch_t(Kernel<E, D, QT, WQ, WK> kernel, AttentionArgs a, hipStream_t s) {
  using S = Shape<E, D, QT, WQ, WK>;
  const Scratch c = scratch_of(kernel, a);
  a.G = a.H / a.KV;
  a.workers = c.workers;
  char* p = static_cast<char*>(a.work);
  a.piece = reinterpret_cast<int4*>(p);
  a.part_ml = reinterpret_cast<float2*>(p + c.part_ml);
  a.part = reinterpret_cast<float*>(p + c.part);
  attention_kernel<E, D, QT, WQ, WK><<<dim3(a.workers), dim3(S::kThreads), 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  attention_join_kernel<E, D, S::kMT><<<dim3(kJoinGroups), dim3(kJoinThreads), 0, s>>>(a);
  return hipGetLastError();
}

// f of the instantiation that a call takes.
template <typename E, int D, typename F>
auto with_blocks(const AttentionArgs& a, F f) {
  const int mt = plan_of(a).mt;
  if (mt == 16) return f(Kernel<E, D, 1, 1, 4>());
  if (mt == 32) return f(Kernel<E, D, 2, 1, 4>());
  if (mt == 64) return f(Kernel<E, D, 2, 2, 2>());
  if constexpr (D <= 128) {
    if (mt == 256) return f(Kernel<E, D, 2, 8, 1>());
  }
  return f(Kernel<E, D, 2, 4, 1>());
}
template <typename F>
auto with_kernel(const AttentionArgs& a, F f) {
  if (a.dtype == VSV_BF16) {
    if (a.D == 64) return with_blocks<uint16_t, 64>(a, f);
    if (a.D == 128) return with_blocks<uint16_t, 128>(a, f);
    return with_blocks<uint16_t, 256>(a, f);
  }
  return a.D == 64 ? with_blocks<float, 64>(a, f) : with_blocks<float, 128>(a, f);
}

}  // namespace

int64_t attention_tiles(const AttentionArgs& a) {
  const Plan p = plan_of(a);
  const int64_t tokens = (static_cast<int64_t>(a.table_width) << a.page_shift) + VSV_MAX_TREE_ROWS;
  const int64_t blocks = (static_cast<int64_t>(VSV_MAX_TREE_ROWS) * (a.H / a.KV) + p.mt - 1) / p.mt;
  const int64_t tiles = (tokens + p.tile - 1) / p.tile;
  if (tiles > (int64_t{1} << 40) / blocks / a.KV) return INT64_MAX;
  return tiles * blocks * a.KV;
}

size_t attention_workspace(const AttentionArgs& a) {
  return with_kernel(a, [&](auto kernel) { return scratch_of(kernel, a).bytes; });
}

hipError_t launch_attention(const AttentionArgs& a, hipStream_t s) {
  return with_kernel(a, [&](auto kernel) { return launch_t(kernel, a, s); });
}

}  // namespace vsv
