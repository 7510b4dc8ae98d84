// Internal interface between the C ABI (abi.cpp) and the adjustment of
// logits (adjust.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "vspec_verify.h"

namespace vsv {

struct AdjustArgs {
  const void* x;            // [R, ld]
  void* y;                  // [R, out_ld]; may be x itself
  int64_t ld, out_ld;
  int32_t V, B, R, dtype;
  const int32_t* offsets;   // [B + 1]
  const int32_t* drafts;    // [num_drafts]
  const int32_t* parents;   // [R], or NULL: chains
  const int32_t* history;   // [B, hist_ld] or NULL
  int64_t hist_ld;
  int32_t hist_width;
  const int32_t* prompt_len;    // [B], or NULL: 0
  const int32_t* history_len;   // [B]
  const float* repetition;      // [B] or NULL each
  const float* frequency;
  const float* presence;
  const int32_t* bias_offsets;  // [B + 1] or NULL
  const int32_t* bias_tokens;
  const float* bias_values;
  int32_t bias_count;
  const uint32_t* mask;         // [mask_rows, mask_ld] words, or NULL
  int64_t mask_ld;
  int32_t mask_rows;
  const int32_t* mask_index;    // [R], or NULL: row r's mask is row r
  int32_t num_drafts;
  int32_t* error_flag;
  int32_t cus;
  // set at launch
  int32_t slices, rows, groups;   // parts of the vocabulary; rows of a block; blocks side by side
};

hipError_t launch_adjust(const AdjustArgs& a, hipStream_t s);

}  // namespace vsv
