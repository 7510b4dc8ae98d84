// Host program of tests/test_overlap_host.py: random strided sets of places,
// against a byte map.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "overlap.hpp"

using vsv::Places;

static char memory[1 << 16];

static std::vector<char> bytes_of(const Places& p, bool& twice) {
  std::vector<char> m(sizeof(memory), 0);
  twice = false;
  const int64_t at = static_cast<const char*>(p.base) - memory;
  for (int64_t x = 0; x < p.count[0]; ++x)
    for (int64_t y = 0; y < p.count[1]; ++y)
      for (int64_t z = 0; z < p.count[2]; ++z)
        for (int64_t b = 0; b < p.bytes; ++b) {
          char& c = m[at + x * p.stride[0] + y * p.stride[1] + z * p.stride[2] + b];
          twice |= c;
          c = 1;
        }
  return m;
}

int main(int argc, char** argv) {
  std::mt19937 rng(atoi(argv[1]));
  auto pick = [&](int lo, int hi) { return static_cast<int64_t>(std::uniform_int_distribution<int>(lo, hi)(rng)); };
  int meeting = 0, apart = 0, inside = 0;
  for (int n = 0; n < 20000; ++n) {
    const int64_t bytes = 8 << pick(0, 2);
    // sets with steps of one another's, of their own, in any order
    auto places = [&](int dims, int64_t unit) {
      Places p{memory + 8192 + 8 * pick(0, 150), bytes, {0, 0, 0}, {1, 1, 1}};
      int64_t step = bytes;
      for (int d = 0; d < dims; ++d) {
        p.count[d] = pick(1, 5);
        p.stride[d] = pick(0, 3) ? step + 8 * pick(0, 6) : unit;
        if (p.stride[d] < step && pick(0, 9)) p.stride[d] = step;
        step = p.count[d] * p.stride[d] + (pick(0, 1) ? 0 : bytes * pick(0, 3));
      }
      for (int d = 0; d < dims; ++d) {
        const int e = static_cast<int>(pick(0, dims - 1));
        std::swap(p.count[d], p.count[e]);
        std::swap(p.stride[d], p.stride[e]);
      }
      return p;
    };
    const int64_t unit = bytes * pick(1, 9);
    Places out = places(2, unit), in = places(static_cast<int>(pick(1, 3)), unit);
    if (pick(0, 1)) {   // slices of the same rows
      const int64_t row = out.stride[0] + in.stride[0] + bytes * pick(0, 4);
      out.stride[0] = in.stride[0] = row;
      out.count[0] = in.count[0] = pick(1, 5);
    }
    if (pick(0, 9) == 0) in = {memory + 8192 + 8 * pick(0, 150), 8 * pick(1, 60), {0, 0, 0}, {1, 1, 1}};
    bool twice, self;
    const auto a = bytes_of(out, self), b = bytes_of(in, twice);
    bool meet = false;
    for (size_t k = 0; k < a.size() && !meet; ++k) meet = a[k] && b[k];
    const bool said = vsv::places_meet(out, in);
    if (meet && !said) return printf("case %d: shared memory is not seen\n", n), 2;
    if (!meet && said) {
      // allowed where `in` has steps inside its inner ones alone
      std::vector<std::pair<int64_t, int64_t>> dims;
      for (int d = 0; d < 3; ++d)
        if (in.count[d] > 1 && in.stride[d] > 0) dims.push_back({in.stride[d], in.count[d]});
      std::sort(dims.begin(), dims.end());
      int64_t inner = in.bytes;
      bool nested = true;
      for (auto& d : dims) {
        nested &= d.first >= inner;
        inner += (d.second - 1) * d.first;
      }
      if (nested) return printf("case %d: nothing is shared\n", n), 3;
      ++inside;
    }
    (meet ? meeting : apart)++;
  }
  printf("ok %d meet, %d do not, %d overlap themselves\n", meeting, apart, inside);
  return 0;
}
