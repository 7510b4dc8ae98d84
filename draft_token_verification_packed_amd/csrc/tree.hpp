// Trees of drafted tokens (gfx950): a request's packed rows are the nodes of
// a tree, its first row the root (the last token already emitted) and every
// later row a draft whose parent is an earlier row of the request. A chain,
// the layout linear verification uses, is the tree in which row j's parent
// is row j - 1.
#pragma once

#include "device.hpp"

namespace vsv {

// The path from the root to row `lane` of a request of n <= 64 rows, as bits
// of the request's rows: every lane joins its own path with that of the row
// its pointer has reached, which doubles both at each of six steps. `parent`
// is lane's entry of the parents; one that is no earlier row sets `bad` and
// leaves the lane a root of its own. Every lane of the wave must be active.
__device__ __forceinline__ uint64_t tree_paths(int lane, int n, int parent, bool chain, bool& bad) {
  uint64_t path = lane < n ? 1ull << lane : 0ull;
  int up = -1;
  bad = false;
  if (lane > 0 && lane < n) {
    up = chain ? lane - 1 : parent;
    bad = up < 0 || up >= lane;
    up = bad ? -1 : up;
  }
#pragma unroll
  for (int step = 0; step < 6; ++step) {
    const int at = up < 0 ? lane : up;
    const uint32_t lo = __shfl(static_cast<uint32_t>(path), at);
    const uint32_t hi = __shfl(static_cast<uint32_t>(path >> 32), at);
    const int next = __shfl(up, at);
    if (up >= 0) {
      path |= (static_cast<uint64_t>(hi) << 32) | lo;
      up = next;
    }
  }
  return path;
}

}  // namespace vsv
