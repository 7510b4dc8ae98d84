// Host program of tests/test_attention_host.py: one batch through the
// attention kernel's own source, against sums in 64 bits. Loads into LDS come
// as early and as late as their waits allow, in both orders of waves and
// workgroups, and all four runs have to agree to the bit. Every load into LDS
// is held against the chunks that the batch may read, LDS and scratch start as NaN, and
// arrays end at pages without access.
#include <random>

static const char* tile_lo;
static const char* tile_hi;
static void emu_tiles(void* lds, size_t all, void* tiles, size_t bytes);

#include "kernel.hpp"

static void emu_tiles(void* lds, size_t all, void* tiles, size_t bytes) {
  if (threadIdx.x == 0) memset(lds, 0xFF, all);
  tile_lo = static_cast<char*>(tiles);
  tile_hi = tile_lo + bytes;
}

template <typename E> float wide(E v);
template <> float wide(float v) { return v; }
template <> float wide(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
template <typename E> E narrow(float f);
template <> float narrow(float f) { return f; }
template <> uint16_t narrow(float f) { return __builtin_bit_cast(uint16_t, __truncsfbf2(f)); }

struct Span { const char* lo; std::vector<bool> may; };   // an array's chunks of 16 bytes

template <typename E>
int batch(int D, int H, int KV, int page, int cus, int B, int rows_lo, int rows_hi, int len_lo, int len_hi, int kind, int seed, int block) {
  std::mt19937 rng(seed);
  auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  std::normal_distribution<float> normal;
  const bool rising = kind == 2, malformed = kind == 3;
  std::vector<int> off{0}, len, par;
  for (int i = 0; i < B; ++i) {
    const int n = pick(rows_lo, rows_hi);
    off.push_back(off.back() + n);
    len.push_back(pick(len_lo, len_hi));
    for (int j = 0; j < n; ++j) par.push_back(j == 0 ? -1 : kind == 1 ? j - 1 : pick(0, j - 1));
  }
  const int R = off[B], G = H / KV;
  int pages = 3, W = 1;
  for (int n : len) pages += (n + page - 1) / page, W = max(W, (n + page - 1) / page + 1);
  std::vector<int> ids(pages), table(static_cast<size_t>(B) * W, -7);
  for (int p = 0; p < pages; ++p) ids[p] = p;
  std::shuffle(ids.begin(), ids.end(), rng);
  for (int i = 0, at = 0; i < B; ++i)
    for (int p = 0; p < (len[i] + page - 1) / page; ++p) table[static_cast<size_t>(i) * W + p] = ids[at++];

  auto fill = [&](size_t n) {
    E* p = reinterpret_cast<E*>(emu::array(n * sizeof(E)));
    for (size_t k = 0; k < n; ++k) p[k] = narrow<E>(normal(rng));
    return p;
  };
  const size_t cache = static_cast<size_t>(pages) * page * KV * D, own = static_cast<size_t>(R) * KV * D;
  E* q = fill(static_cast<size_t>(R) * H * D);
  E *k = fill(own), *v = fill(own), *kc = fill(cache), *vc = fill(cache);
  auto place = [&](int i, int t, int h) {
    return ((static_cast<size_t>(table[static_cast<size_t>(i) * W + t / page]) * page + t % page) * KV + h) * D;
  };
  if (rising)   // scores grow by more than the slack from step to step
    for (int i = 0; i < B; ++i)
      for (int t = 0; t < len[i]; ++t)
        for (int h = 0; h < KV; ++h)
          for (int d = 0; d < D; ++d) kc[place(i, t, h) + d] = narrow<E>(wide(kc[place(i, t, h) + d]) * 0.03f * t);
  auto ints = [&](const std::vector<int>& x) {
    int32_t* p = reinterpret_cast<int32_t*>(emu::array(x.size() * 4));
    std::copy(x.begin(), x.end(), p);
    return p;
  };
  // what may be brought into LDS; malformed requests read page 0 or nothing
  Span spans[4] = {{reinterpret_cast<char*>(k), {}}, {reinterpret_cast<char*>(v), {}}, {reinterpret_cast<char*>(kc), {}},
                   {reinterpret_cast<char*>(vc), {}}};
  for (int s = 0; s < 4; ++s) spans[s].may.assign((s < 2 ? own : cache) * sizeof(E) / 16, s < 2);
  for (int i = 0; i < B; ++i)
    for (int t = 0; t < len[i]; ++t)
      for (int h = 0; h < KV; ++h)
        for (size_t c = place(i, t, h) * sizeof(E) / 16, n = 0; n < D * sizeof(E) / 16; ++n)
          spans[2].may[c + n] = spans[3].may[c + n] = true;
  std::vector<bool> sound(B, true);
  if (malformed) {
    for (int s = 2; s < 4; ++s) spans[s].may.assign(spans[s].may.size(), true);
    const std::vector<int> real = off;
    for (int i = 0; i < B; ++i) {
      const int what = pick(0, 5);
      sound[i] = what > 3;
      if (what == 0) len[i] = pick(0, 1) ? -pick(1, 9) : W * page + pick(1, 1 << 28);
      if (what == 1 && len[i] > 0) table[static_cast<size_t>(i) * W + pick(0, (len[i] - 1) / page)] = pick(0, 1) ? -1 : pages + pick(0, 1 << 30);
      if (what == 2) par[real[i] + pick(0, real[i + 1] - real[i] - 1)] = pick(0, 1) ? 1 << 30 : -5;
      if (what == 3 && i + 1 < B) off[i + 1] = pick(0, 1) ? -3 : R + 70000;
    }
    for (int i = 0; i < B; ++i) sound[i] = sound[i] && off[i] == real[i] && off[i + 1] == real[i + 1];
  }
  emu::check = [&](const char* from, const char* to) {
    if (to < tile_lo || to + 16 > tile_hi) emu::fail("a load goes beyond the tiles");
    for (const Span& s : spans)
      if (from >= s.lo && from < s.lo + s.may.size() * 16) {
        if (!s.may[(from - s.lo) / 16]) emu::fail("a load reads what no row sees");
        return;
      }
    emu::fail("a load reads outside the arrays");
  };

  vsv::AttentionArgs a{};
  a.q = q; a.k = k; a.v = v; a.k_cache = kc; a.v_cache = vc;
  E* out = reinterpret_cast<E*>(emu::array(static_cast<size_t>(R) * H * D * sizeof(E)));
  a.lse = reinterpret_cast<float*>(emu::array(static_cast<size_t>(R) * H * 4));
  a.out = out;
  a.q_row = a.o_row = H * D;
  a.q_head = a.o_head = a.k_head = a.v_head = a.c_head = D;
  a.k_row = a.v_row = a.c_token = KV * D;
  a.c_page = static_cast<int64_t>(page) * KV * D;
  a.table = ints(table); a.table_ld = a.table_width = W; a.num_pages = pages;
  while ((1 << a.page_shift) < page) ++a.page_shift;
  a.length = ints(len); a.offsets = ints(off);
  a.parents = kind == 1 ? nullptr : ints(par);
  a.B = B; a.R = R; a.H = H; a.KV = KV; a.D = D;
  a.dtype = sizeof(E) == 2 ? VSV_BF16 : VSV_F32;
  const double scale = 1 / sqrt(static_cast<double>(D));
  a.scale = static_cast<float>(1.44269504088896340736 * scale);
  int32_t* flag = ints({0});
  a.error_flag = flag;
  a.cus = cus;
  const size_t scratch = vsv::attention_workspace(a);
  a.work = emu::array(scratch);

  std::vector<E> first;
  for (int mode = 0; mode < 4; ++mode) {
    emu::early = mode & 1;
    emu::backward = mode >> 1;
    for (size_t n = 0; n < static_cast<size_t>(R) * H * D; ++n) out[n] = narrow<E>(NAN);
    memset(a.work, 0xFF, scratch);
    if (vsv::launch_attention(a, nullptr) != hipSuccess) return 1;
    std::vector<E> now(out, out + static_cast<size_t>(R) * H * D);
    if (mode == 0) first = now;
    if (memcmp(first.data(), now.data(), now.size() * sizeof(E))) {
      printf("run %d differs\n", mode);
      return 2;
    }
  }
  // the scratch is the launch's workgroups' own
  const size_t workers = emu::launches[0], pieces = workers * 2 * block;
  auto whole = [](size_t b) { return (b + 255) / 256 * 256; };
  if (emu::launches.size() != 8 || scratch != whole(workers * 16) + whole(pieces * 8) + whole(pieces * D * 4))
    return printf("%zu bytes of scratch for %zu workgroups\n", scratch, workers), 7;
  if (!malformed && *flag) return printf("flags %d\n", *flag), 4;
  // against 64 bits; tolerances as in tests/test_gpu_attention.py, with the
  // sum of |q k| of each token in place of a bound for all of them
  double worst = 0;
  for (int i = 0; i < B; ++i) {
    if (!sound[i]) continue;
    for (int r = off[i]; r < off[i + 1]; ++r) {
      std::vector<bool> sees(off[i + 1] - off[i], false);
      for (int j = r - off[i]; j >= 0; j = kind == 1 ? j - 1 : j ? par[off[i] + j] : -1) sees[j] = true;
      for (int h = 0; h < H; ++h) {
        std::vector<std::pair<const E*, const E*>> seen;
        for (int t = 0; t < len[i]; ++t) seen.push_back({kc + place(i, t, h / G), vc + place(i, t, h / G)});
        for (size_t j = 0; j < sees.size(); ++j)
          if (sees[j]) seen.push_back({k + ((off[i] + j) * KV + h / G) * D, v + ((off[i] + j) * KV + h / G) * D});
        const E* x = q + (static_cast<size_t>(r) * H + h) * D;
        std::vector<double> s(seen.size());
        double top = -INFINITY, most = 0;
        for (size_t t = 0; t < seen.size(); ++t) {
          double dot = 0, mag = 0;
          for (int d = 0; d < D; ++d) {
            const double p = static_cast<double>(wide(x[d])) * wide(seen[t].first[d]);
            dot += p;
            mag += fabs(p);
          }
          s[t] = dot * scale;
          top = max(top, s[t]);
          most = max(most, mag * scale);
        }
        double sum = 0;
        for (double& w : s) sum += w = exp(w - top);
        const double e = 2 * D * 0x1p-24 * most + 0x1p-21 * (1 + most), T = static_cast<double>(seen.size());
        const double half = sizeof(E) == 2 ? 0x1p-8 : 0x1p-24, weight = sizeof(E) == 2 ? 0x1p-8 : 0;
        for (int d = 0; d < D; ++d) {
          double o = 0, mag = 0;
          for (size_t t = 0; t < seen.size(); ++t) {
            o += s[t] / sum * wide(seen[t].second[d]);
            mag += s[t] / sum * fabs(wide(seen[t].second[d]));
          }
          const double tol = (2 * e + weight + T * 0x1p-23) * mag + half * fabs(o) + 1e-30;
          const double err = fabs(wide(first[(static_cast<size_t>(r) * H + h) * D + d]) - o);
          if (!(err <= tol)) return printf("request %d row %d head %d column %d: off by %g of %g\n", i, r, h, d, err, tol), 5;
          worst = max(worst, err / tol);
        }
        const double lse = top + log(sum);
        if (!(fabs(a.lse[static_cast<size_t>(r) * H + h] - lse) <= e + 0x1p-22 * (1 + fabs(lse)))) return printf("row %d: lse\n", r), 6;
      }
    }
  }
  printf("ok %d rows, largest error %.2f of its bound\n", R, worst);
  emu::release();
  return 0;
}

int main(int argc, char** argv) {
  std::vector<int> n;
  for (int k = 1; k < argc; ++k) n.push_back(atoi(argv[k]));
  auto f = n[0] ? batch<uint16_t> : batch<float>;
  return f(n[1], n[2], n[3], n[4], n[5], n[6], n[7], n[8], n[9], n[10], n[11], n[12], n[13]);
}
