// Penalties, biases and grammar masks on packed rows of logits (gfx950).
//
// Row r of request i stands behind a path of drafts: in a chain the drafts
// before it, in a tree those on the way from the root to its node, its own
// included. With c the number of times a token occurs in the request's
// output and on that path, and "seen" if it occurs there or in the prompt,
//   y = seen ? (x > 0 ? x / rho : x * rho) : x
//   y = y - f c - p [c > 0]
//   y = y + b
//   y = -inf where the row's grammar mask has a 0 bit
// in float32 (x / rho as x times the rounded reciprocal), rounded once to the
// logits' type.
//
// A workgroup takes a slice of one request's vocabulary and holds a word per
// token of it in LDS: twice the count, plus one if the token is in the
// prompt. It reads the request's history, counting the tokens inside the slice
// with LDS atomics on integers (their order cannot show), and then streams
// its slice of a block of the request's rows one after another, moving the counts from
// row to row by the drafts that the paths do not share. A bit per token
// tells the stream which 8 logits to look up at all, so the untouched rest
// goes from load to store as it is. The history is read once per slice
// and block of rows (mostly from L2) instead of once per row, and no dense
// count matrix exists.
// Bound by HBM: each logit read and written once. 640 rows of 152064 bf16
// logits with histories of up to 1024 tokens, biases and half the rows masked
// take 90 us, 4.4 TB/s (the same rows copied by this kernel 79, 5.0); 397
// rows of 50021 fp32 logits with histories of up to 16000 tokens 49 us.
// In place, only the vectors that a count, a bias or a mask touches move.
#include "adjust.hpp"
#include "tree.hpp"

namespace vsv {

namespace {

// Vectors of 8 logits: 16 bytes of bfloat16, 32 of float32. Rows need only
// the element's alignment; gfx950 loads and stores 16 bytes at any address.
typedef uint32_t u32x4_2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// All ones if bit k of `bits` is set, else 0.
__device__ __forceinline__ uint32_t bit_mask(uint32_t bits, int k) {
  return static_cast<uint32_t>(static_cast<int32_t>(bits << (31 - k)) >> 31);
}

template <typename E> struct Vec8;
template <> struct Vec8<uint16_t> {
  u32x4 w;
  __device__ __forceinline__ void load(const uint16_t* p) { w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_2*>(p)); }
  __device__ __forceinline__ void store(uint16_t* p) const { __builtin_nontemporal_store(u32x4_2(w), reinterpret_cast<u32x4_2*>(p)); }
  __device__ __forceinline__ void get(float* f) const { Elem<uint16_t>::decode(w, f); }
  __device__ __forceinline__ void set(const float* f) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(f[2 * k]), static_cast<__bf16>(f[2 * k + 1])});
  }
  // -inf wherever `allow` has a 0 bit
  __device__ __forceinline__ void mask(uint32_t allow) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t keep = (bit_mask(allow, 2 * k) & 0xFFFFu) | (bit_mask(allow, 2 * k + 1) & 0xFFFF0000u);
      w[k] = (w[k] & keep) | (0xFF80FF80u & ~keep);
    }
  }
};
template <> struct Vec8<float> {
  u32x4 w[2];
  __device__ __forceinline__ void load(const float* p) {
    w[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_4*>(p));
    w[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_4*>(p) + 1);
  }
  __device__ __forceinline__ void store(float* p) const {
    __builtin_nontemporal_store(u32x4_4(w[0]), reinterpret_cast<u32x4_4*>(p));
    __builtin_nontemporal_store(u32x4_4(w[1]), reinterpret_cast<u32x4_4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(w[k >> 2][k & 3]);
  }
  __device__ __forceinline__ void set(const float* f) {
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k >> 2][k & 3] = __float_as_uint(f[k]);
  }
  __device__ __forceinline__ void mask(uint32_t allow) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t keep = bit_mask(allow, k);
      w[k >> 2][k & 3] = (w[k >> 2][k & 3] & keep) | (0xFF800000u & ~keep);
    }
  }
};

// Nearest bfloat16, ties to even; a NaN stays one.
__device__ __forceinline__ uint32_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f)); }

__device__ __forceinline__ float widen(float f) { return f; }
__device__ __forceinline__ float widen(uint16_t h) { return __uint_as_float(static_cast<uint32_t>(h) << 16); }
__device__ __forceinline__ void narrow(float f, float* p) { *p = f; }
__device__ __forceinline__ void narrow(float f, uint16_t* p) { *p = static_cast<uint16_t>(to_bf16(f)); }

// A slice of 2048 tokens: its table leaves eight workgroups a CU. 4096 (four)
// took 60 instead of 51 us on 397 rows of 50021 fp32 logits; on 640 rows of
// 152064 bf16 ones 2048, 4096 and 8192 are within 1 us of one another.
constexpr int kThreads = 256;
constexpr int kSliceTokens = 2048;
constexpr int kMostRows = 8;         // rows of a request a workgroup takes at a time
constexpr int kShortHistory = 4096;  // tokens

// (words are read four at a time)
struct alignas(16) AdjustScratch {
  uint32_t count[kSliceTokens];       // 2 * occurrences in output and path, + 1 if in the prompt
  uint32_t bias[kSliceTokens];        // the last entry's number + 1, then its value's bits
  uint32_t touched[kSliceTokens / 32];
  int draft[VSV_MAX_TREE_ROWS];
  uint64_t path[VSV_MAX_TREE_ROWS];
};

template <typename E, bool kInPlace>
__global__ __launch_bounds__(kThreads) void adjust_kernel(AdjustArgs a) {
  __shared__ AdjustScratch s;
  constexpr int NT = kThreads, SL = kSliceTokens;
  constexpr int kPer = SL / 8 / NT;   // vectors a thread streams of a row
  static_assert(kPer * NT * 8 == SL, "whole vectors per thread");
  const int tid = threadIdx.x;
  const int slice = static_cast<int>(blockIdx.x) % a.slices;
  const int rest = static_cast<int>(blockIdx.x) / a.slices;
  const int group = rest % a.groups;
  const int i = rest / a.groups;
  const int v0 = slice * SL, vn = min(SL, a.V - v0);
  int bits = 0;

  const int o0 = a.offsets[i], o1 = a.offsets[i + 1];
  if (o0 < 0 || o1 < o0 || o1 > a.R || (a.parents && o1 - o0 > VSV_MAX_TREE_ROWS)) {
    if (tid == 0 && a.error_flag) atomicOr(a.error_flag, VSV_FLAG_LAYOUT);
    return;
  }
  const int n = o1 - o0;
  // this workgroup's rows of the request: every groups-th block of a.rows
  const int j0 = group * a.rows;
  if (j0 >= n) return;
  int block_end = j0 + a.rows;

  float rho = a.repetition ? a.repetition[i] : 1.f;
  float freq = a.frequency ? a.frequency[i] : 0.f;
  float pres = a.presence ? a.presence[i] : 0.f;
  // (the reciprocal has to be a normal number)
  const bool rho_ok = rho >= 0x1p-126f && rho <= 0x1p126f;
  if (!rho_ok || !(fabsf(freq) < INFINITY) || !(fabsf(pres) < INFINITY)) {
    bits |= VSV_FLAG_PARAMS;
    if (!rho_ok) rho = 1.f;
    if (!(fabsf(freq) < INFINITY)) freq = 0.f;
    if (!(fabsf(pres) < INFINITY)) pres = 0.f;
  }
  const bool penal = rho != 1.f || freq != 0.f || pres != 0.f;
  int b0 = 0, b1 = 0;
  if (a.bias_offsets) {
    b0 = a.bias_offsets[i];
    b1 = a.bias_offsets[i + 1];
    if (b0 < 0 || b1 < b0 || b1 > a.bias_count) {
      bits |= VSV_FLAG_LAYOUT;
      b0 = b1 = 0;
    }
  }
  const bool biased = b1 > b0;

  // ---- the slice's table
  if (penal) {
    for (int k = tid; k < SL / 4; k += NT) reinterpret_cast<u32x4*>(s.count)[k] = u32x4{0, 0, 0, 0};
  }
  if (biased) {
    for (int k = tid; k < SL / 4; k += NT) reinterpret_cast<u32x4*>(s.bias)[k] = u32x4{0, 0, 0, 0};
  }
  for (int k = tid; k < SL / 32; k += NT) s.touched[k] = 0;
  lds_barrier();
  auto touch = [&](int q) { atomicOr(&s.touched[q >> 5], 1u << (q & 31)); };
  // One occurrence of a token more or less; those outside the vocabulary
  // count nowhere.
  auto add = [&](int token, uint32_t what) {
    if (token < 0 || token >= a.V) {
      bits |= VSV_FLAG_TOKEN;
      return;
    }
    const int q = token - v0;
    if (q < 0 || q >= vn) return;
    if (what == 1u)
      atomicOr(&s.count[q], 1u);
    else
      atomicAdd(&s.count[q], what);
    touch(q);
  };
  // the draft that row r > 0 of the request carries
  auto draft_of = [&](int r) {
    const int dq = o0 + r - i - 1;
    if (dq >= 0 && dq < a.num_drafts) return a.drafts[dq];
    bits |= VSV_FLAG_LAYOUT;
    return -1;
  };
  if (penal && a.history) {
    int end = a.history_len[i], prompt = a.prompt_len ? a.prompt_len[i] : 0;
    if (end < 0 || end > a.hist_width || prompt < 0 || prompt > end) {
      bits |= VSV_FLAG_LAYOUT;
      end = max(0, min(end, a.hist_width));
      prompt = max(0, min(prompt, end));
    }
    const int* __restrict__ h = a.history + static_cast<int64_t>(i) * a.hist_ld;
    // four tokens a load, kU loads under way
    constexpr int kU = 4;
    const int quads = end >> 2;
    for (int k = tid; k < quads; k += NT * kU) {
      u32x4 tok[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) tok[u] = reinterpret_cast<const u32x4_4*>(h)[min(k + u * NT, quads - 1)];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int at = (k + u * NT) * 4;
        if (at >= end - 3) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) add(static_cast<int>(tok[u][e]), at + e < prompt ? 1u : 2u);
      }
    }
    for (int k = quads * 4 + tid; k < end; k += NT) add(h[k], k < prompt ? 1u : 2u);
  }
  if (biased) {
    for (int k = b0 + tid; k < b1; k += NT) {
      const int token = a.bias_tokens[k], q = token - v0;
      const float value = a.bias_values[k];
      if (token < 0 || token >= a.V) {
        bits |= VSV_FLAG_TOKEN;
      } else if (!(value < INFINITY)) {
        bits |= VSV_FLAG_PARAMS;
      } else if (q >= 0 && q < vn) {
        atomicMax(&s.bias[q], static_cast<uint32_t>(k - b0) + 1u);
        touch(q);
      }
    }
  }
  // the drafts of the request's first rows, and a tree's paths
  if (penal && tid < kWave) {
    const int up = a.parents && tid < n ? a.parents[o0 + tid] : 0;
    s.draft[tid] = tid > 0 && tid < n ? draft_of(tid) : -1;
    if (a.parents) {
      bool bad;
      s.path[tid] = tree_paths(tid, n, up, false, bad);
      if (bad) bits |= VSV_FLAG_LAYOUT;
    }
  }
  lds_barrier();
  if (biased) {
    for (int q = tid; q < vn; q += NT) {
      const uint32_t e = s.bias[q];
      if (e) s.bias[q] = __float_as_uint(a.bias_values[b0 + static_cast<int>(e) - 1]);
    }
  }

  // (the reciprocal costs a second rounding of 2^-24 and saves a division per
  // touched logit)
  const float inv_rho = 1.f / rho;
  auto adjusted = [&](float x, uint32_t c, uint32_t b) {
    if (penal) {
      float y = x > 0.f ? x * inv_rho : x * rho;
      y = y - freq * static_cast<float>(c >> 1);
      y = c > 1u ? y - pres : y;
      x = c ? y : x;
    }
    return biased ? x + __uint_as_float(b) : x;
  };

  // ---- the rows
  const E* xs = static_cast<const E*>(a.x) + v0;
  E* ys = static_cast<E*>(a.y) + v0;
  const uint8_t* touched = reinterpret_cast<const uint8_t*>(s.touched);
  // a row's logits and the bytes of its mask, one row ahead of its use
  Vec8<E> buf[kPer];
  uint32_t allow_buf[kPer];
  const uint8_t* mask_buf = nullptr;
  auto load_row = [&](int j) {
    const E* row = xs + static_cast<int64_t>(o0 + j) * a.ld;
    mask_buf = nullptr;
    if (a.mask) {
      const int m = a.mask_index ? a.mask_index[o0 + j] : o0 + j;
      if (m >= a.mask_rows)
        bits |= VSV_FLAG_LAYOUT;
      else if (m >= 0)
        mask_buf = reinterpret_cast<const uint8_t*>(a.mask + static_cast<int64_t>(m) * a.mask_ld) + (v0 >> 3);
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int q = (k * NT + tid) * 8;
      allow_buf[k] = 0xFFu;
      if (q + 8 <= vn) {
        if (!kInPlace) buf[k].load(row + q);
        if (mask_buf) allow_buf[k] = mask_buf[q >> 3];
      }
    }
  };
  // Counts of row j's path, from those of row `from` (-1: none).
  auto move_path = [&](int from, int j) {
    if (!penal) return;
    if (a.parents) {
      if (tid < kWave) {
        const uint64_t was = from < 0 ? 0 : s.path[from], now = s.path[j];
        const uint64_t bit = 1ull << tid;
        if (tid > 0 && ((was ^ now) & bit)) add(s.draft[tid], now & bit ? 2u : ~1u);
      }
    } else {
      // the rows of the chain up to j
      for (int r = max(from, 0) + 1 + tid; r <= j; r += NT) add(r < VSV_MAX_TREE_ROWS ? s.draft[r] : draft_of(r), 2u);
    }
  };
  load_row(j0);
  for (int j = j0, from = -1, next; j < n; from = j, j = next) {
    next = j + 1;
    if (next == block_end) {
      next += (a.groups - 1) * a.rows;
      block_end = next + a.rows;
    }
    move_path(from, j);
    lds_barrier();
    const E* row = xs + static_cast<int64_t>(o0 + j) * a.ld;
    E* out = ys + static_cast<int64_t>(o0 + j) * a.out_ld;
    Vec8<E> cur[kPer];
    uint32_t allow[kPer];
    const uint8_t* mask = mask_buf;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      cur[k] = buf[k];
      allow[k] = allow_buf[k];
    }
    if (next < n) load_row(next);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int q = (k * NT + tid) * 8;
      if (q + 8 <= vn) {
        const uint32_t hit = touched[q >> 3] & allow[k];
        if (kInPlace) {
          if (hit == 0 && allow[k] == 0xFFu) continue;
          if (allow[k]) cur[k].load(row + q);
        }
        if (hit) {
          float f[8];
          cur[k].get(f);
          const u32x4* c = reinterpret_cast<const u32x4*>(s.count + q);
          const u32x4* b = reinterpret_cast<const u32x4*>(s.bias + q);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4 ch = penal ? c[h] : u32x4{0, 0, 0, 0}, bh = biased ? b[h] : u32x4{0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = adjusted(f[h * 4 + e], ch[e], bh[e]);
              f[h * 4 + e] = hit >> (h * 4 + e) & 1u ? y : f[h * 4 + e];
            }
          }
          cur[k].set(f);
        }
        if (allow[k] != 0xFFu) cur[k].mask(allow[k]);
        cur[k].store(out + q);
      } else {
        for (int e = q; e < vn && e < q + 8; ++e) {
          float x = widen(row[e]);
          if (touched[e >> 3] >> (e & 7) & 1) x = adjusted(x, penal ? s.count[e] : 0, biased ? s.bias[e] : 0);
          if (mask && !(mask[e >> 3] >> (e & 7) & 1)) x = -INFINITY;
          narrow(x, out + e);
        }
      }
    }
    lds_barrier();   // the counts move on
  }
  if (bits && a.error_flag) atomicOr(a.error_flag, bits);
}

template <typename E>
hipError_t launch_t(AdjustArgs a, hipStream_t s) {
  a.slices = (a.V + kSliceTokens - 1) / kSliceTokens;
  // A request's rows go in blocks of a.rows to as many workgroups as twice the
  // mean request fills (longer ones go round). Blocks are as long as gives
  // each of the eight workgroups that fit a CU one, or two where histories are short
  // and a table is soon built: 397 fp32 rows of 50021 logits take 39 us with two
  // and 42 with one for histories of 64 tokens, 58 and 52 for 16000.
  const int64_t base = static_cast<int64_t>(a.B) * a.slices;
  const int64_t mean = (a.R + a.B - 1) / a.B;
  const int64_t fit = static_cast<int64_t>(a.cus > 0 ? a.cus : 256) * 8 * (a.hist_width > kShortHistory ? 1 : 2);
  int64_t rows = static_cast<int64_t>(a.R) * a.slices / fit;
  rows = rows < 1 ? 1 : rows > kMostRows ? kMostRows : rows;
  a.rows = static_cast<int32_t>(rows);
  a.groups = mean <= rows ? 1 : static_cast<int32_t>((2 * mean + rows - 1) / rows);
  const int64_t grid = base * a.groups;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  if (a.x == a.y)
    adjust_kernel<E, true><<<dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s>>>(a);
  else
    adjust_kernel<E, false><<<dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adjust(const AdjustArgs& a, hipStream_t s) {
  return a.dtype == VSV_BF16 ? launch_t<uint16_t>(a, s) : launch_t<float>(a, s);
}

}  // namespace vsv
