// The per-request scan of tree verification (gfx950): run by the workgroup
// that ends the launch, once the rows' arg-maxes are on their way.
//
// From the root the walk moves to the lowest row whose parent is the current
// row and whose draft is the current row's arg-max, until there is none. The
// rows of a window (whole requests, at most kTreeStage rows) look their
// parent's arg-max up all at once and leave themselves at the parent if they
// fit (the lowest row wins); the walk of a request is then a chase of LDS
// words by one thread. 709 rows of 24 trees (V = 152064, bf16) verify in 43 us,
// 5.0 TB/s: the rows' stream and about 3 us for the scan.
#pragma once

#include "verify_common.hpp"

namespace vsv {

// Rows of a window. Its words and links are 16 KiB, what the linear scan's
// LDS comes to: twice as many would cut the workgroups a CU holds while it
// streams the rows.
constexpr int kTreeStage = 2048;
constexpr int kNoChild = INT32_MAX;

template <int NT>
struct TreeScratch {
  uint32_t words[kTreeStage];
  int child[kTreeStage];   // lowest fitting child, counted from the window's first row
  int scan[16];
};

template <int NT>
__device__ __forceinline__ void tree_tail(const VerifyArgs& a, uint32_t tag, TreeScratch<NT>& t) {
  const int tid = threadIdx.x;
  int stalled = 0, budget = kPollBudget, carry = 0, bits = 0;
  for (int i0 = 0; i0 < a.B;) {
    // this window: requests i0 .. i1 - 1, at least one. Layouts that do not
    // rise are caught request by request below; here they only end a window.
    const int w0 = a.offsets[i0];
    const int i = i0 + tid;
    int r0 = 0, r1 = 0;
    if (i < a.B) {
      r0 = a.offsets[i];
      r1 = a.offsets[i + 1];
    }
    const bool sound = i < a.B && r0 >= 0 && r1 > r0 && r1 <= a.R && r1 - r0 <= VSV_MAX_TREE_ROWS &&
                       (i != 0 || r0 == 0) && (i != a.B - 1 || r1 == a.R);
    const bool fits = sound && r0 >= w0 && r1 - w0 <= kTreeStage;
    int in_front = fits ? 0 : 1, stops;
    in_front = block_exclusive_scan<NT>(in_front, t.scan, stops) + in_front;
    const bool inside = in_front == 0;   // no request up to this one ended the window
    int count;
    block_exclusive_scan<NT>(inside ? 1 : 0, t.scan, count);
    const int i1 = i0 + (count > 0 ? count : 1);
    int rows = 0;
    if (count > 0) rows = a.offsets[i1] - w0;   // sound requests alone: 0 < rows <= kTreeStage

    // the rows' links: metadata first, so that it is under way while the
    // words are waited for
    for (int q = tid; q < rows; q += NT) t.child[q] = kNoChild;
    constexpr int kAhead = 4;
    int draft[kAhead], at[kAhead];
    auto link = [&](int q, int& d, int& p) {
      const int r = w0 + q;
      const int own = a.owner[r];
      d = -1;
      p = -1;
      if (own < i0 || own >= i1) {
        bits |= VSV_FLAG_LAYOUT;
        return;
      }
      const int s0 = a.offsets[own], s1 = a.offsets[own + 1];
      if (r < s0 || r >= s1) {
        bits |= VSV_FLAG_LAYOUT;
        return;
      }
      if (r == s0) return;
      const int up = a.parents ? a.parents[r] : r - s0 - 1;
      const int dq = r - own - 1;
      const int tok = dq >= 0 && dq < a.R - a.B ? a.drafts[dq] : -1;
      if (up < 0 || up >= r - s0) {
        bits |= VSV_FLAG_LAYOUT;
      } else if (tok < 0 || tok >= a.V) {
        bits |= VSV_FLAG_TOKEN;
      } else {
        d = tok;
        p = s0 - w0 + up;
      }
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      draft[k] = at[k] = -1;
      if (tid + k * NT < rows) link(tid + k * NT, draft[k], at[k]);
    }
    for (int k0 = tid; k0 < rows; k0 += NT * kGatherBatch) {
      uint64_t w[kGatherBatch];
#pragma unroll
      for (int b = 0; b < kGatherBatch; ++b) {
        const int q = k0 + b * NT;
        w[b] = load_agent64(a.ws_row + w0 + (q < rows ? q : 0));
      }
#pragma unroll
      for (int b = 0; b < kGatherBatch; ++b) {
        const int q = k0 + b * NT;
        if (q < rows) {
          uint32_t v = static_cast<uint32_t>(w[b]);
          if (static_cast<uint32_t>(w[b] >> 32) != tag) v = poll_tagged(a.ws_row + w0 + q, tag, budget, stalled);
          t.words[q] = v & kTokenMask;
        }
      }
    }
    lds_barrier();
    auto join = [&](int q, int d, int p) {
      if (p >= 0 && t.words[p] == static_cast<uint32_t>(d)) atomicMin(&t.child[p], q);
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) join(tid + k * NT, draft[k], at[k]);
    for (int q = tid + kAhead * NT; q < rows; q += NT) {
      int d, p;
      link(q, d, p);
      join(q, d, p);
    }
    lds_barrier();

    // the walks; a request that is not sound emits the token 0 alone
    int acc = 0, last = 0;
    if (inside) {
      last = r0 - w0;
      for (int c = t.child[last]; c != kNoChild; c = t.child[last]) {
        last = c;
        ++acc;
      }
    }
    const bool mine = inside || (count == 0 && tid == 0);
    const int len = mine ? acc + 1 : 0;
    int total = 0;
    const int pos = carry + block_exclusive_scan<NT>(len, t.scan, total);
    if (mine) {
      const int token = inside ? static_cast<int>(t.words[last]) : 0;
      if (!inside) bits |= VSV_FLAG_LAYOUT;
      a.accepted_len[i] = acc;
      a.next_token[i] = token;
      a.out_offsets[i] = pos;
      int q = r0 - w0;
      for (int k = 0; k <= acc; ++k) {
        if (pos + k < a.R) {
          // the accepted child carries the arg-max of the row it hangs on
          a.out_tokens[pos + k] = inside ? static_cast<int>(t.words[q]) : 0;
          if (a.out_rows) a.out_rows[pos + k] = inside ? w0 + q : -1;
        }
        if (k < acc) q = t.child[q];
      }
    }
    carry += total;
    i0 = i1;
    lds_barrier();   // the next window reuses the words and links
  }
  if (tid == 0) a.out_offsets[a.B] = carry;
  for (int p = carry + tid; p < a.R; p += NT) {
    a.out_tokens[p] = -1;
    if (a.out_rows) a.out_rows[p] = -1;
  }
  if (stalled) bits |= VSV_FLAG_STALLED;
  if (bits) set_flag(a, bits);
  end_call(a, tag);
}

}  // namespace vsv
