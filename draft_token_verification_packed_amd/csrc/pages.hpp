// Internal interface between the C ABI (abi.cpp) and the page plan
// (pages.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace vsv {

// Every workgroup holds the batch's prefix sums in LDS.
constexpr int kMaxPlanRequests = 8192;

struct PagesArgs {
  int32_t* table;           // [B, ld]
  int64_t ld;
  int32_t width;            // pages a request may hold
  int32_t B, R, page_size;
  const int32_t* held;      // [B] pages of every request
  const int32_t* length;    // [B] tokens stored
  const int32_t* offsets;   // [B + 1] rows to store
  int32_t* pool;            // [pool_size] ids of the free pages, a stack
  int32_t pool_size;
  const int32_t* count;     // [1] pages on it
  int64_t* slot;            // [R]
  int32_t* position;        // [R] or NULL
  int32_t* new_held;        // [B]
  int32_t* new_length;      // [B]
  int32_t* new_count;       // [1]
  int32_t* error_flag;
};

hipError_t launch_pages(const PagesArgs& a, hipStream_t s);

}  // namespace vsv
