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
// in float32, rounded once to the logits' type.
//
// A workgroup takes a slice of one request's vocabulary and holds a word per
// token of it in LDS: twice the count, plus one if the token is in the
// prompt. It reads the request's history once, counting the tokens inside the slice
// with LDS atomics on integers (their order cannot show), and then streams
// its slice of the request's rows one after another, moving the counts from
// row to row by the drafts that the paths do not share. A bit per token
// tells the stream which 8 logits to look up at all, so the untouched rest
// goes from load to store as it is. The history is read once per slice from
// L2 instead of once per row, and no dense count matrix exists.
// Bound by HBM: each logit read and written once.
#include "adjust.hpp"
#include "tree.hpp"

namespace vsv {

namespace {

// Vectors of 8 logits: 16 bytes of bfloat16, 32 of float32. Rows need only
// the element's alignment; gfx950 loads and stores 16 bytes at any address.
typedef uint32_t u32x4_2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));

template <typename E> struct Vec8;
template <> struct Vec8<uint16_t> {
  u32x4 w;
  __device__ __forceinline__ void load(const uint16_t* p) { w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_2*>(p)); }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<u32x4_2*>(p) = w; }
  __device__ __forceinline__ float get(int k) const {
    const uint32_t v = w[k >> 1];
    return __uint_as_float(k & 1 ? v & 0xFFFF0000u : v << 16);
  }
  __device__ __forceinline__ void put(int k, float f);
};
template <> struct Vec8<float> {
  u32x4 w[2];
  __device__ __forceinline__ void load(const float* p) {
    w[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_4*>(p));
    w[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_4*>(p) + 1);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<u32x4_4*>(p)[0] = w[0];
    reinterpret_cast<u32x4_4*>(p)[1] = w[1];
  }
  __device__ __forceinline__ float get(int k) const { return __uint_as_float(w[k >> 2][k & 3]); }
  __device__ __forceinline__ void put(int k, float f) { w[k >> 2][k & 3] = __float_as_uint(f); }
};

// Nearest bfloat16, ties to even; a NaN stays one.
__device__ __forceinline__ uint32_t to_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u >> 16) | 0x40u;
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}
__device__ __forceinline__ void Vec8<uint16_t>::put(int k, float f) {
  const uint32_t h = to_bf16(f);
  w[k >> 1] = k & 1 ? (w[k >> 1] & 0xFFFFu) | (h << 16) : (w[k >> 1] & 0xFFFF0000u) | h;
}

__device__ __forceinline__ float widen(float f) { return f; }
__device__ __forceinline__ float widen(uint16_t h) { return __uint_as_float(static_cast<uint32_t>(h) << 16); }
__device__ __forceinline__ void narrow(float f, float* p) { *p = f; }
__device__ __forceinline__ void narrow(float f, uint16_t* p) { *p = static_cast<uint16_t>(to_bf16(f)); }

constexpr int kRows = 8;   // rows of a request a workgroup takes at a time

template <int SL>
struct AdjustScratch {
  uint32_t count[SL];       // 2 * occurrences in output and path, + 1 if in the prompt
  uint32_t bias[SL];        // the last entry's number + 1, then its value's bits
  uint32_t touched[SL / 32];
  int draft[VSV_MAX_TREE_ROWS];
  uint64_t path[VSV_MAX_TREE_ROWS];
};

template <typename E, int NT, int SL, bool kInPlace>
__global__ __launch_bounds__(NT) void adjust_kernel(AdjustArgs a) {
  __shared__ AdjustScratch<SL> s;
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
  // this workgroup's rows of the request: every groups-th block of kRows
  const int j0 = group * kRows;
  if (j0 >= n) return;
  auto row_after = [&](int j) { return (j + 1) % kRows ? j + 1 : j + 1 + (a.groups - 1) * kRows; };

  float rho = a.repetition ? a.repetition[i] : 1.f;
  float freq = a.frequency ? a.frequency[i] : 0.f;
  float pres = a.presence ? a.presence[i] : 0.f;
  if (!(rho > 0.f) || !(rho < INFINITY) || !(fabsf(freq) < INFINITY) || !(fabsf(pres) < INFINITY)) {
    bits |= VSV_FLAG_PARAMS;
    if (!(rho > 0.f) || !(rho < INFINITY)) rho = 1.f;
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
  // the tree's paths (a chain of any length needs none)
  if (a.parents && penal) {
    if (tid < kWave) {
      const int up = tid < n ? a.parents[o0 + tid] : 0;
      const int dq = o0 + tid - i - 1;   // the row's own draft
      int d = -1;
      if (tid > 0 && tid < n) {
        if (dq >= 0 && dq < a.R - a.B)
          d = a.drafts[dq];
        else
          bits |= VSV_FLAG_LAYOUT;
      }
      bool bad;
      s.path[tid] = tree_paths(tid, n, up, false, bad);
      s.draft[tid] = d;
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

  auto fix = [&](float x, int q) {
    if (penal) {
      const uint32_t c = s.count[q];
      if (c) {
        x = x > 0.f ? x / rho : x * rho;
        if (c > 1u) {
          x -= freq * static_cast<float>(c >> 1);
          x -= pres;
        }
      }
    }
    if (biased) x += __uint_as_float(s.bias[q]);
    return x;
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
      // rows 1 .. j of the chain carry drafts 0 .. j - 1
      const int first = from < 0 ? 1 : from + 1;
      for (int r = first + tid; r <= j; r += NT) {
        const int dq = o0 + r - i - 1;
        if (dq >= 0 && dq < a.R - a.B)
          add(a.drafts[dq], 2u);
        else
          bits |= VSV_FLAG_LAYOUT;
      }
    }
  };
  load_row(j0);
  for (int j = j0, from = -1; j < n; from = j, j = row_after(j)) {
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
    if (row_after(j) < n) load_row(row_after(j));
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
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (hit >> e & 1u) cur[k].put(e, fix(cur[k].get(e), q + e));
        }
        if (allow[k] != 0xFFu) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!(allow[k] >> e & 1u)) cur[k].put(e, -INFINITY);
        }
        cur[k].store(out + q);
      } else {
        for (int e = q; e < vn && e < q + 8; ++e) {
          float x = widen(row[e]);
          if (touched[e >> 3] >> (e & 7) & 1) x = fix(x, e);
          if (mask && !(mask[e >> 3] >> (e & 7) & 1)) x = -INFINITY;
          narrow(x, out + e);
        }
      }
    }
    lds_barrier();   // the counts move on
  }
  if (bits && a.error_flag) atomicOr(a.error_flag, bits);
}

template <typename E, int NT, int SL>
hipError_t launch_t(AdjustArgs a, hipStream_t s) {
  a.slices = (a.V + SL - 1) / SL;
  // a request's rows in blocks of kRows to as many workgroups as twice the
  // mean request fills (longer ones go round)
  const int64_t base = static_cast<int64_t>(a.B) * a.slices;
  const int64_t mean = (a.R + a.B - 1) / a.B;
  a.groups = mean <= kRows ? 1 : static_cast<int32_t>((2 * mean + kRows - 1) / kRows);
  const int64_t grid = base * a.groups;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  if (a.x == a.y)
    adjust_kernel<E, NT, SL, true><<<dim3(static_cast<unsigned>(grid)), dim3(NT), 0, s>>>(a);
  else
    adjust_kernel<E, NT, SL, false><<<dim3(static_cast<unsigned>(grid)), dim3(NT), 0, s>>>(a);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_e(const AdjustArgs& a, hipStream_t s) {
#ifdef VSV_SL
  return launch_t<E, VSV_NT, VSV_SL>(a, s);
#else
  const int64_t large = static_cast<int64_t>(a.B) * ((a.V + 8191) / 8192);
  return large >= 2 * static_cast<int64_t>(a.cus > 0 ? a.cus : 256) ? launch_t<E, 512, 8192>(a, s)
                                                                     : launch_t<E, 256, 2048>(a, s);
#endif
}

}  // namespace

hipError_t launch_adjust(const AdjustArgs& a, hipStream_t s) {
  return a.dtype == VSV_BF16 ? launch_e<uint16_t>(a, s) : launch_e<float>(a, s);
}

}  // namespace vsv
