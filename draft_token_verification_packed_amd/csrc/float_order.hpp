// Floats in the order of their values, as unsigned keys. Host and device code.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace vsv {

// Order-preserving unsigned key of a float (-0 mapped to +0), and back.
__host__ __device__ __forceinline__ uint32_t up_key(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x == 0.0f ? 0.0f : x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__host__ __device__ __forceinline__ float key_value(uint32_t k) {
  return __builtin_bit_cast(float, (k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
// The next float by value, downwards and upwards; the two zeros count as one,
// so the key of -0, which up_key never gives, is stepped over.
__host__ __device__ __forceinline__ float next_down(float x) {
  const uint32_t k = up_key(x) - 1u;
  return key_value(k == 0x7FFFFFFFu ? k - 1u : k);
}
__host__ __device__ __forceinline__ float next_up(float x) {
  const uint32_t k = up_key(x) + 1u;
  return key_value(k == 0x7FFFFFFFu ? k + 1u : k);
}

}  // namespace vsv
