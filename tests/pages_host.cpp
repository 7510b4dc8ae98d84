// Host program of tests/test_pages_large_host.py: the last workgroup of a page
// plan over as many rows as a call may have. Its steps over the rows pass
// 2^31, and nothing before or behind the arrays may be touched.
#include "kernel.hpp"

int main(int argc, char** argv) {
  const int B = atoi(argv[1]);
  vsv::PagesArgs a{};
  a.B = B;
  a.R = INT32_MAX;
  a.width = a.ld = 4;
  a.page_size = 16;
  a.pool_size = 2 * B + 1;
  auto ints = [](size_t n) { return reinterpret_cast<int32_t*>(emu::array(n * 4)); };
  a.table = ints(4 * B);
  int32_t* held = ints(B), *length = ints(B), *offsets = ints(B + 1), *count = ints(1);
  for (int i = 0; i < B; ++i) {
    held[i] = 1;
    length[i] = 10;
    a.table[4 * i] = i;
    offsets[i + 1] = 2 * (i + 1);
  }
  a.held = held;
  a.length = length;
  a.offsets = offsets;
  a.count = count;
  a.pool = ints(a.pool_size);
  // (the rows' results: their pages exist once they are written to)
  a.slot = reinterpret_cast<int64_t*>(emu::array(static_cast<size_t>(a.R) * 8));
  a.position = nullptr;
  a.new_held = ints(B);
  a.new_length = ints(B);
  a.new_count = ints(1);
  const int threads = B <= 256 ? 256 : 1024;
  emu::only = 255;
  if (vsv::launch_pages(a, nullptr) != hipSuccess) return 1;
  // the workgroup's rows, first and last step
  for (int64_t r = 255 * threads; r < a.R; r += 256 * threads) {
    for (int64_t k = r; k < r + threads && k < a.R; k += threads - 1)
      if (a.slot[k] != (k < 2 * B ? k / 2 * 16 + 10 + k % 2 : -1)) return 2;
  }
  printf("ok\n");
  return 0;
}
