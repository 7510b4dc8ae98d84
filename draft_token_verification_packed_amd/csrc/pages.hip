// Page plan (gfx950): block tables and slots of the rows to be stored, from
// lengths that only the device knows.
//
// With l_i tokens stored, n_i rows to store and pages of s tokens, request i
// needs p_i = ceil((l_i + n_i) / s) pages and holds h_i. Free pages are a
// stack. Requests that hold more than they need give theirs back first, in
// request order; then those that need more take from the top, in request
// order. With G_i and T_i the sums of the pages given back and taken by the
// requests before i, c the stack's height and t = c + G_B:
//   page h_i <= p < p_i of a taker is stack entry t - 1 - (T_i + p - h_i),
//   entry e >= c of the stack is the given-back page e - c, found in the
//   table of the giver i with G_i <= e - c < G_(i+1).
// Nothing that a call reads is written by it (takers' new table entries and
// the stack above c are only written, and the counts have outputs of their
// own), so every workgroup works the sums out for itself, no two need to
// meet, and a call repeated on the same inputs writes the same results.
//
// The call is bound by latency: four loads a request, a block scan, then a
// search, a load and a store a row, one row a thread: 6.6 us for 128 requests
// and 384 rows, 8.3 us for 512 and 96,000.
#include "device.hpp"
#include "pages.hpp"
#include "vspec_verify.h"

namespace vsv {

namespace {

template <int CAP>
struct PagesScratch {
  int off[CAP + 1];        // rows before the request
  int taken[CAP + 1];      // T_i
  int given[CAP + 1];      // G_i
  int scan[16];
};

// What a request asks for; nothing where its inputs make no sense.
struct Ask {
  int n, need, give, take;
  bool bad;
};

__device__ __forceinline__ Ask ask_of(const PagesArgs& a, int i) {
  const int o0 = a.offsets[i], o1 = a.offsets[i + 1], len = a.length[i], held = a.held[i];
  Ask q{0, held, 0, 0, true};
  if (o0 < 0 || o1 < o0 || o1 > a.R || len < 0 || held < 0 || held > a.width) return q;
  const int64_t end = static_cast<int64_t>(len) + (o1 - o0);
  const int64_t need = (end + a.page_size - 1) / a.page_size;
  if (end > INT32_MAX || need > a.width) return q;
  q.bad = false;
  q.n = o1 - o0;
  q.need = static_cast<int>(need);
  q.give = max(held - q.need, 0);
  q.take = max(q.need - held, 0);
  return q;
}

// The last i in [0, n) with v[i] <= x (v[0] <= x and v does not fall).
__device__ __forceinline__ int last_at_most(const int* v, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <int NT, int CAP>
__global__ __launch_bounds__(NT) void pages_kernel(PagesArgs a) {
  __shared__ PagesScratch<CAP> s;
  const int t = threadIdx.x, B = a.B;
  // (indexes that a step may carry past 2^31 have 64 bits)
  const int step = static_cast<int>(gridDim.x) * NT;
  const int first = static_cast<int>(blockIdx.x) * NT + t;
  int bits = 0;

  int count = a.count[0];
  if (count < 0 || count > a.pool_size) {
    bits |= VSV_FLAG_LAYOUT;
    count = max(0, min(count, a.pool_size));
  }
  // the sums: with the stack they cannot pass 2^31, as a request holds at most
  // `width` and the host bounds B * width + pool_size
  int takes = 0, gives = 0;
  for (int base = 0; base < B; base += NT) {
    const int i = base + t;
    Ask q{0, 0, 0, 0, false};
    if (i < B) q = ask_of(a, i);
    int total_take, total_give;
    const int before_take = block_exclusive_scan<NT>(q.take, s.scan, total_take);
    const int before_give = block_exclusive_scan<NT>(q.give, s.scan, total_give);
    if (i < B) {
      s.off[i] = a.offsets[i];
      s.taken[i] = takes + before_take;
      s.given[i] = gives + before_give;
      if (q.bad) bits |= VSV_FLAG_LAYOUT;
    }
    takes += total_take;
    gives += total_give;
  }
  if (t == 0) {
    s.off[B] = a.offsets[B];
    s.taken[B] = takes;
    s.given[B] = gives;
  }
  lds_barrier();
  const int top = count + gives;
  if (top > a.pool_size) bits |= VSV_FLAG_LAYOUT;

  // A taker is served while the stack lasts, in request order.
  auto served = [&](int i) { return s.taken[i + 1] == s.taken[i] || s.taken[i + 1] <= top; };
  // Page on entry e of the stack once the givers' pages are on it.
  auto entry = [&](int e) -> int {
    if (e < count) return a.pool[e];
    const int g = e - count;
    const int i = last_at_most(s.given, B, g);
    // the giver keeps its first h - (pages given) pages
    const int keeps = a.held[i] - (s.given[i + 1] - s.given[i]);
    return a.table[static_cast<int64_t>(i) * a.ld + keeps + (g - s.given[i])];
  };

  // rows: the page is an old one of the request or one it takes
  for (int64_t row = first; row < a.R; row += step) {
    const int r = static_cast<int>(row);
    int64_t slot = -1;
    int pos = -1;
    if (B > 0 && r < s.off[B]) {
      const int i = last_at_most(s.off, B, r);
      const Ask q = ask_of(a, i);
      if (!q.bad && r >= s.off[i] && r < s.off[i + 1] && served(i)) {
        pos = a.length[i] + (r - s.off[i]);
        const int p = pos / a.page_size;
        const int held = a.held[i];
        const int id = p < held ? a.table[static_cast<int64_t>(i) * a.ld + p] : entry(top - 1 - (s.taken[i] + p - held));
        if (id >= 0) {
          slot = static_cast<int64_t>(id) * a.page_size + (pos - p * a.page_size);
        } else {
          bits |= VSV_FLAG_LAYOUT;
        }
      }
    }
    a.slot[row] = slot;
    if (a.position) a.position[row] = pos;
  }
  // the takers' new table entries
  for (int64_t entry_of = first; entry_of < takes && entry_of < top; entry_of += step) {
    const int k = static_cast<int>(entry_of);
    const int i = last_at_most(s.taken, B, k);
    if (served(i)) a.table[static_cast<int64_t>(i) * a.ld + a.held[i] + (k - s.taken[i])] = entry(top - 1 - k);
  }
  // the givers' pages
  for (int64_t g = first; g < gives && count + g < a.pool_size; g += step)
    a.pool[count + g] = entry(static_cast<int>(count + g));
  // the requests
  for (int i = first; i < B; i += step) {
    const Ask q = ask_of(a, i);
    const bool ok = !q.bad && served(i);
    if (!q.bad && !ok) bits |= VSV_FLAG_PAGES;
    a.new_held[i] = ok ? q.need : a.held[i];
    a.new_length[i] = ok ? a.length[i] + q.n : a.length[i];
  }
  if (first == 0) {
    // pages taken by the served requests: the last sum that the stack covers
    int spent = takes;
    if (takes > top) {
      int lo = 0, hi = B;   // largest i with taken[i] <= top
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.taken[mid] <= top) lo = mid; else hi = mid - 1;
      }
      spent = s.taken[lo];
    }
    a.new_count[0] = min(top - spent, a.pool_size);
  }
  if (bits && a.error_flag) atomicOr(a.error_flag, bits);
}

template <int NT, int CAP>
hipError_t launch_t(const PagesArgs& a, hipStream_t s) {
  // a row a thread, up to a workgroup per CU; the loops take the rest
  int64_t groups = (static_cast<int64_t>(a.R > a.B ? a.R : a.B) + NT - 1) / NT;
  if (groups > 256) groups = 256;
  if (groups < 1) groups = 1;
  pages_kernel<NT, CAP><<<dim3(static_cast<unsigned>(groups)), dim3(NT), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_pages(const PagesArgs& a, hipStream_t s) {
  return a.B <= 256 ? launch_t<256, 256>(a, s) : launch_t<1024, kMaxPlanRequests>(a, s);
}

}  // namespace vsv
