// Host program of tests/test_malformed_host.py: page plans and adjustments
// whose inputs on the device make no sense. Nothing beyond the arrays may be
// touched, and rows behind the last request stay as they are.
#include <random>

#include "kernel.hpp"

static std::mt19937 rng;
static int pick(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }
// mostly a sound value, else one of those that break things
static int odd(int sound) {
  static const int far[] = {-1, -2, INT32_MIN, INT32_MAX, INT32_MAX - 1, 1 << 30, 65536, 0, 1, 7};
  return pick(0, 5) ? sound : far[pick(0, 9)];
}
template <typename T, typename F>
static T* array(int64_t n, F f) {
  T* p = reinterpret_cast<T*>(emu::array(n * sizeof(T)));
  for (int64_t k = 0; k < n; ++k) p[k] = f(k);
  return p;
}

#ifdef PAGES
static int run() {
  vsv::PagesArgs a{};
  const int B = a.B = pick(0, 3) ? pick(1, 40) : pick(257, 400);
  a.width = pick(1, 6);
  a.ld = a.width + pick(0, 2);
  a.page_size = pick(1, 40);
  a.pool_size = pick(1, 3 * B);
  a.R = pick(0, 3 * B);
  a.table = array<int32_t>((B - 1) * a.ld + a.width, [&](int64_t) { return odd(pick(0, 3 * B)); });
  a.held = array<int32_t>(B, [&](int64_t) { return odd(pick(0, a.width)); });
  a.length = array<int32_t>(B, [&](int64_t) { return odd(pick(0, a.width * a.page_size)); });
  int at = 0;
  a.offsets = array<int32_t>(B + 1, [&](int64_t) { at += pick(0, 3); return odd(at); });
  a.count = array<int32_t>(1, [&](int64_t) { return odd(pick(0, a.pool_size)); });
  a.pool = array<int32_t>(a.pool_size, [&](int64_t) { return odd(pick(0, 3 * B)); });
  a.slot = array<int64_t>(a.R, [](int64_t) { return 0; });
  a.position = array<int32_t>(a.R, [](int64_t) { return 0; });
  a.new_held = array<int32_t>(B, [](int64_t) { return 0; });
  a.new_length = array<int32_t>(B, [](int64_t) { return 0; });
  a.new_count = array<int32_t>(1, [](int64_t) { return 0; });
  a.error_flag = array<int32_t>(1, [](int64_t) { return 0; });
  if (vsv::launch_pages(a, nullptr) != hipSuccess) return 1;
  if (a.new_count[0] < 0 || a.new_count[0] > a.pool_size) return 2;
  return 0;
}
#else
template <typename E>
static int run_t() {
  vsv::AdjustArgs a{};
  const int B = a.B = pick(1, 6);
  std::vector<int> off{0};
  for (int i = 0; i < B; ++i) off.push_back(off.back() + pick(1, pick(0, 3) ? 6 : 70));
  const int real = off.back(), R = a.R = real + pick(0, 3);
  const int V = a.V = pick(0, 3) ? pick(1, 300) : pick(2000, 5000);
  a.ld = V + pick(0, 9);
  a.out_ld = V + pick(0, 9);
  a.dtype = sizeof(E) == 2 ? VSV_BF16 : VSV_F32;
  const bool in_place = pick(0, 2) == 0;
  E* x = array<E>((R - 1) * a.ld + V, [&](int64_t) { return static_cast<E>(pick(0, 1 << 15)); });
  E* y = in_place ? x : array<E>((R - 1) * a.out_ld + V, [](int64_t) { return E(3); });
  if (in_place) a.out_ld = a.ld;
  a.x = x;
  a.y = y;
  const bool sound = pick(0, 2) == 0;   // offsets that can be relied on
  a.offsets = array<int32_t>(B + 1, [&](int64_t k) { return sound ? off[k] : odd(off[k]); });
  a.num_drafts = R - B;
  a.drafts = array<int32_t>(R - B, [&](int64_t) { return odd(pick(0, V - 1)); });
  if (pick(0, 1)) a.parents = array<int32_t>(R, [&](int64_t k) { return odd(pick(0, 3)); });
  if (pick(0, 2)) {
    a.hist_width = pick(1, 50);
    a.hist_ld = a.hist_width + pick(0, 3);
    a.history = array<int32_t>((B - 1) * a.hist_ld + a.hist_width, [&](int64_t) { return odd(pick(0, V - 1)); });
    a.history_len = array<int32_t>(B, [&](int64_t) { return odd(pick(0, a.hist_width)); });
    if (pick(0, 1)) a.prompt_len = array<int32_t>(B, [&](int64_t) { return odd(pick(0, a.hist_width)); });
  }
  auto floats = [&](float one) {
    return array<float>(B, [&](int64_t) {
      static const float far[] = {NAN, INFINITY, -INFINITY, 0.f, -1.f, 1e-44f, 3e38f};
      return pick(0, 3) ? one : far[pick(0, 6)];
    });
  };
  if (pick(0, 3)) a.repetition = floats(1.3f);
  if (pick(0, 1)) a.frequency = floats(0.5f);
  if (pick(0, 1)) a.presence = floats(-0.5f);
  if (pick(0, 1)) {
    a.bias_count = pick(1, 20);
    int at = 0;
    a.bias_offsets = array<int32_t>(B + 1, [&](int64_t) { at = min(at + pick(0, 4), a.bias_count); return odd(at); });
    a.bias_tokens = array<int32_t>(a.bias_count, [&](int64_t) { return odd(pick(0, V - 1)); });
    a.bias_values = array<float>(a.bias_count, [&](int64_t) { return pick(0, 4) ? 2.f : NAN; });
  }
  if (pick(0, 1)) {
    a.mask_rows = pick(1, 9);
    a.mask_ld = (V + 31) / 32 + pick(0, 2);
    a.mask = array<uint32_t>((a.mask_rows - 1) * a.mask_ld + (V + 31) / 32, [&](int64_t) { return static_cast<uint32_t>(rng()); });
    a.mask_index = array<int32_t>(R, [&](int64_t) { return odd(pick(-1, a.mask_rows - 1)); });
  }
  a.error_flag = array<int32_t>(1, [](int64_t) { return 0; });
  a.cus = pick(0, 1) ? 1 : 256;
  const std::vector<E> before(x, x + (R - 1) * a.ld + V);
  if (vsv::launch_adjust(a, nullptr) != hipSuccess) return 1;
  if (sound)
    for (int r = real; r < R; ++r)
      for (int v = 0; v < V; ++v)
        if (in_place ? x[r * a.ld + v] != before[r * a.ld + v] : y[r * a.out_ld + v] != E(3)) return 2;
  for (int r = 0; r < R - 1; ++r)
    for (int64_t v = V; v < a.out_ld; ++v)
      if (in_place ? x[r * a.ld + v] != before[r * a.ld + v] : y[r * a.out_ld + v] != E(3)) return 3;
  return 0;
}
static int run() { return pick(0, 1) ? run_t<uint16_t>() : run_t<float>(); }
#endif

int main(int argc, char** argv) {
  for (int seed = atoi(argv[1]); seed < atoi(argv[2]); ++seed) {
    rng.seed(seed);
    printf("seed %d\n", seed);
    fflush(stdout);
    emu::backward = seed & 1;
    const int bad = run();
    if (bad) return bad;
    emu::release();
  }
  return 0;
}
