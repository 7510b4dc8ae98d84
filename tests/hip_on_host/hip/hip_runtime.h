// A stand-in for HIP's header that runs a kernel's own source on the CPU, for
// tests of its indexes and waits: threads of a workgroup are fibers, the lanes
// of a wave meet at every exchange between lanes, and a load into LDS arrives
// either as early or as late as its waits allow. Inputs lie before pages that
// cannot be touched, so an access past an end stops the program.
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <sys/mman.h>
#include <unistd.h>

#include <algorithm>
#include <deque>
#include <functional>
#include <vector>

#define __global__
#define __device__
#define __host__
#define __constant__
#define __shared__ static
#define __forceinline__ inline
#define __launch_bounds__(...)
#define address_space(n)

struct int2 { int x, y; };
struct int4 { int x, y, z, w; };
struct float2 { float x, y; };
inline int4 make_int4(int x, int y, int z, int w) { return {x, y, z, w}; }
inline float2 make_float2(float x, float y) { return {x, y}; }
struct dim3 { unsigned x; explicit dim3(unsigned n) : x(n) {} };
typedef void* hipStream_t;
enum hipError_t { hipSuccess = 0, hipErrorInvalidValue = 1 };
inline hipError_t hipGetLastError() { return hipSuccess; }
using std::max;
using std::min;

namespace emu {

constexpr int kWave = 64;
struct Index { unsigned x; };
inline Index thread, block, grid;

[[noreturn]] inline void fail(const char* what) {
  fprintf(stdout, "FAIL workgroup %u thread %u: %s\n", block.x, thread.x, what);
  fflush(stdout);
  _exit(3);
}

// ---- memory: arrays that end at a page without access
inline std::vector<std::pair<const char*, const char*>>& arrays() {
  static std::vector<std::pair<const char*, const char*>> a;
  return a;
}
inline char* array(size_t bytes) {
  const size_t page = 4096, room = (bytes + page - 1) / page * page;
  char* p = static_cast<char*>(mmap(nullptr, room + 2 * page, PROT_NONE, MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0));
  if (p == MAP_FAILED || (room && mprotect(p + page, room, PROT_READ | PROT_WRITE))) fail("no memory");
  char* at = p + page + room - bytes;
  arrays().push_back({at, at + bytes});
  return at;
}
inline void release() {
  for (auto& a : arrays()) {
    const uintptr_t page = 4096, lo = reinterpret_cast<uintptr_t>(a.first) / page * page - page;
    munmap(reinterpret_cast<void*>(lo), reinterpret_cast<uintptr_t>(a.second) + page - lo);
  }
  arrays().clear();
}

// ---- lanes
enum State { kRunning, kExchange, kBarrier, kDone };
struct Copy { const char* from; char* to; };
// Leaves the running stack for another one (registers that a call keeps).
extern "C" void emu_swap(void** leave, void* enter);
asm(R"(
.text
.type emu_swap, @function
emu_swap:
  push %rbp
  push %rbx
  push %r12
  push %r13
  push %r14
  push %r15
  mov %rsp, (%rdi)
  mov %rsi, %rsp
  pop %r15
  pop %r14
  pop %r13
  pop %r12
  pop %rbx
  pop %rbp
  ret
)");
struct Lane {
  void* at = nullptr;        // its stack's top while it is not running
  State state = kDone;
  int op = 0;
  unsigned count = 0;        // exchanges so far
  std::deque<Copy> loads;    // under way
  std::vector<char> stack;
};
inline void* scheduler = nullptr;
inline std::vector<Lane> lanes;
inline Lane* me = nullptr;
inline std::function<void()>* body = nullptr;
// What the lanes of a wave hand one another; two sets in turn, so that a lane
// that runs ahead overwrites nothing that another one still reads.
struct Slot { alignas(16) char bytes[96]; };
inline std::vector<Slot> board[2];

inline void yield(State s, int op) {
  me->state = s;
  me->op = op;
  emu_swap(&me->at, scheduler);
}
// Every lane of the wave gives `v`; returns where they lie, lane 0 first.
template <typename T>
const Slot* exchange(const T& v, int op) {
  static_assert(sizeof(T) <= sizeof(Slot), "room");
  const unsigned parity = me->count++ & 1, t = thread.x;
  memcpy(board[parity][t].bytes, &v, sizeof(T));
  yield(kExchange, op);
  return &board[parity][t / kWave * kWave];
}
template <typename T>
T of(const Slot* s, int lane) {
  T v;
  memcpy(&v, s[lane].bytes, sizeof(T));
  return v;
}
inline int lane() { return static_cast<int>(thread.x % kWave); }
inline void meet() { exchange(0, 1); }

inline void entry() {
  (*body)();
  me->state = kDone;
  if (!me->loads.empty()) fail("a load is under way where the kernel ends");
  emu_swap(&me->at, scheduler);
}

inline bool early = false;    // loads arrive at once, or where they are waited for
inline bool backward = false; // order of the waves
inline int64_t only = -1;     // workgroup to run, or all

inline void run_block(int threads, std::function<void()> f) {
  if (static_cast<int>(lanes.size()) < threads) lanes.resize(threads);
  for (auto& b : board) b.resize(threads);
  body = &f;
  for (int t = 0; t < threads; ++t) {
    Lane& l = lanes[t];
    if (l.stack.empty()) l.stack.resize(256 * 1024);
    // six registers, entry's address, and a return address that is never used
    void** top = reinterpret_cast<void**>((reinterpret_cast<uintptr_t>(l.stack.data() + l.stack.size()) & ~uintptr_t{15}) - 64);
    memset(top, 0, 64);
    top[6] = reinterpret_cast<void*>(&entry);
    l.at = top;
    l.state = kRunning;
    l.count = 0;
  }
  const int waves = threads / kWave;
  for (;;) {
    int ended = 0, waiting = 0;
    for (int k = 0; k < waves; ++k) {
      const int w = backward ? waves - 1 - k : k;
      Lane* wave = &lanes[w * kWave];
      // until the wave's lanes stand at a barrier or at the end
      while (wave[0].state != kBarrier && wave[0].state != kDone) {
        for (int l = 0; l < kWave; ++l) {
          me = &wave[l];
          thread.x = static_cast<unsigned>(w * kWave + l);
          emu_swap(&scheduler, me->at);
        }
        for (int l = 1; l < kWave; ++l)
          if (wave[l].state != wave[0].state || (wave[0].state == kExchange && wave[l].op != wave[0].op)) fail("lanes part at an exchange");
      }
      ended += wave[0].state == kDone;
      waiting += wave[0].state == kBarrier;
    }
    if (ended == waves) return;
    if (waiting != waves) fail("waves part at a barrier");
    for (int t = 0; t < threads; ++t) lanes[t].state = kRunning;
  }
}

inline std::vector<unsigned> launches;   // workgroups of every launch
template <typename K, typename A>
void launch(K kernel, dim3 groups, dim3 threads, const A& args) {
  grid.x = groups.x;
  launches.push_back(groups.x);
  for (unsigned k = 0; k < groups.x; ++k) {
    block.x = backward ? groups.x - 1 - k : k;
    if (only >= 0 && block.x != static_cast<unsigned>(only)) continue;
    run_block(static_cast<int>(threads.x), [&] { kernel(args); });
  }
}

// ---- loads into LDS: 16 bytes a lane, at `to` + 16 * lane
inline std::function<void(const char*, const char*)> check;   // (global address, LDS address)
inline void load_to_lds(int64_t from, uint32_t to) {
  const Slot* all = exchange(to, 2);
  if (of<uint32_t>(all, 0) != to) fail("m0 is not uniform");
  const Copy c{reinterpret_cast<const char*>(from), reinterpret_cast<char*>(static_cast<uintptr_t>(to)) + 16 * lane()};
  if (from % 16) fail("a load is not aligned");
  if (check) check(c.from, c.to);
  if (early) memcpy(c.to, c.from, 16);
  me->loads.push_back(c);
}
inline void wait_loads(size_t n) {
  while (me->loads.size() > n) {
    const Copy c = me->loads.front();
    me->loads.pop_front();
    if (!early) memcpy(c.to, c.from, 16);
  }
  meet();
}

}  // namespace emu

#define threadIdx emu::thread
#define blockIdx emu::block
#define gridDim emu::grid

// ---- what the kernels use of the language and the compiler
template <typename T> T __shfl(T v, int lane) { return emu::of<T>(emu::exchange(v, 3), lane & 63); }
template <typename T> T __shfl_xor(T v, int mask) { return emu::of<T>(emu::exchange(v, 4), emu::lane() ^ mask); }
inline float __uint_as_float(uint32_t v) { return __builtin_bit_cast(float, v); }
inline uint32_t __float_as_uint(float v) { return __builtin_bit_cast(uint32_t, v); }
inline float __log2f(float v) { return log2f(v); }
inline uint32_t __umulhi(uint32_t a, uint32_t b) { return static_cast<uint32_t>((static_cast<uint64_t>(a) * b) >> 32); }
template <typename T, typename U> T atomicOr(T* p, U v) { T old = *p; *p = static_cast<T>(old | v); return old; }
template <typename T, typename U> T atomicAdd(T* p, U v) { T old = *p; *p = static_cast<T>(old + v); return old; }
template <typename T, typename U> T atomicMax(T* p, U v) { T old = *p; if (v > old) *p = v; return old; }
// (at any address that its type allows)
#define __builtin_nontemporal_load(p) (*(p))
#define __builtin_nontemporal_store(v, p) (*(p) = (v))
template <typename T> T emu_load(T* p) { return *p; }
#define __hip_atomic_load(p, ...) emu_load(p)
#define __hip_atomic_store(p, v, ...) (*(p) = (v))

template <typename T> T emu_first_lane(T v) {
  const emu::Slot* s = emu::exchange(v, 5);
  if (emu::of<T>(s, 0) != v) emu::fail("a value read from the first lane differs between lanes");
  return v;
}
inline int emu_dpp(int old, int v, int control, int rows, int banks) {
  const emu::Slot* s = emu::exchange(v, 6 + control);
  const int l = emu::lane(), row = l / 16, in = l % 16;
  if (!(rows >> row & 1) || !(banks >> (in / 4) & 1)) return old;
  if (control >= 0x150 && control < 0x160) return emu::of<int>(s, row * 16 + control - 0x150);
  if (control > 0x110 && control < 0x120) return in >= control - 0x110 ? emu::of<int>(s, l - (control - 0x110)) : old;
  if (control > 0x120 && control < 0x130) return emu::of<int>(s, row * 16 + ((in - (control - 0x120)) & 15));
  if (control == 0x142) return row ? emu::of<int>(s, row * 16 - 1) : old;
  if (control == 0x143) return row >= 2 ? emu::of<int>(s, 31) : old;
  emu::fail("an exchange that is not modelled");
}
#define __builtin_amdgcn_readfirstlane(v) emu_first_lane(v)
#define __builtin_amdgcn_readlane(v, l) emu::of<int>(emu::exchange(static_cast<int>(v), 7), l)
#define __builtin_amdgcn_update_dpp(old, v, control, rows, banks, bound) emu_dpp(old, v, control, rows, banks)
#define __builtin_amdgcn_fence(...) ((void)0)
#define __builtin_amdgcn_s_barrier() emu::yield(emu::kBarrier, 0)
#define __builtin_amdgcn_wave_barrier() emu::meet()
#define __builtin_amdgcn_s_waitcnt(n) ((void)0)
#define __builtin_amdgcn_s_sleep(n) ((void)0)
#define __builtin_amdgcn_exp2f(x) exp2f(x)

inline uint64_t emu_ballot(bool b) {
  const emu::Slot* s = emu::exchange(b, 8);
  uint64_t bits = 0;
  for (int l = 0; l < 64; ++l) bits |= static_cast<uint64_t>(emu::of<bool>(s, l)) << l;
  return bits;
}
#define __builtin_amdgcn_ballot_w64(b) emu_ballot(b)

// Products of 16 x 16: lane l holds row (column) l % 16 of a factor and, of
// the inner dimension, the elements N (l / 16) .. + N - 1; of the result,
// column l % 16 and rows 4 (l / 16) .. + 3.
typedef float emu_f32x4 __attribute__((ext_vector_type(4)));
template <int N>
emu_f32x4 emu_mma(const float* a, const float* b, emu_f32x4 c, int op) {
  struct In { float a[N], b[N]; } in;
  memcpy(in.a, a, sizeof(in.a));
  memcpy(in.b, b, sizeof(in.b));
  const emu::Slot* s = emu::exchange(in, op);
  const int l = emu::lane();
  for (int k = 0; k < 4; ++k) {
    const In y = emu::of<In>(s, k * 16 + l % 16);
    for (int e = 0; e < 4; ++e) {
      const In x = emu::of<In>(s, k * 16 + l / 16 * 4 + e);
      for (int n = 0; n < N; ++n) c[e] = fmaf(x.a[n], y.b[n], c[e]);
    }
  }
  return c;
}
typedef __bf16 emu_bf16x8 __attribute__((ext_vector_type(8)));
inline emu_f32x4 emu_mma_bf16(emu_bf16x8 a, emu_bf16x8 b, emu_f32x4 c) {
  const auto wide = [](__bf16 h) { return __builtin_bit_cast(float, static_cast<uint32_t>(__builtin_bit_cast(uint16_t, h)) << 16); };
  float x[8], y[8];
  for (int e = 0; e < 8; ++e) x[e] = wide(a[e]), y[e] = wide(b[e]);
  return emu_mma<8>(x, y, c, 9);
}
#define __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, x, y, z) emu_mma_bf16(a, b, c)
inline emu_f32x4 emu_mma_f32(float a, float b, emu_f32x4 c) { return emu_mma<1>(&a, &b, c, 10); }
#define __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, x, y, z) emu_mma_f32(a, b, c)

// The transposing LDS read: the 16 lanes of a group read four 16-bit elements
// each, and lane c receives element c % 4 of the lanes c / 4, + 4, + 8 and + 12.
typedef short emu_s16x4 __attribute__((ext_vector_type(4)));
inline emu_s16x4 emu_read_tr16(const emu_s16x4* p) {
  const emu::Slot* s = emu::exchange(*p, 11);
  const int l = emu::lane(), group = l / 16 * 16, c = l % 16;
  emu_s16x4 r;
  for (int e = 0; e < 4; ++e) r[e] = emu::of<emu_s16x4>(s, group + 4 * e + c / 4)[c % 4];
  return r;
}
#define __builtin_amdgcn_ds_read_tr16_b64_v4i16(p) emu_read_tr16(p)

// the compiler's own narrowing, to the nearest, ties to even
extern "C" inline __bf16 __truncsfbf2(float f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, f);
  const uint32_t r = (u & 0x7FFFFFFFu) > 0x7F800000u ? (u >> 16 | 0x40u) : (u + 0x7FFFu + (u >> 16 & 1u)) >> 16;
  return __builtin_bit_cast(__bf16, static_cast<uint16_t>(r));
}
