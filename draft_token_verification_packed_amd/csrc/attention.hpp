// Internal interface between the C ABI (abi.cpp) and the attention of draft
// trees over a paged cache (attention.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace vsv {

struct AttentionArgs {
  const void* q;            // [R, H, D]
  const void* k;            // [R, KV, D] the rows' own keys and values
  const void* v;
  const void* k_cache;      // [pages, page tokens, KV, D]
  const void* v_cache;
  void* out;                // [R, H, D]
  float* lse;               // [R, H] or NULL
  // strides in elements
  int64_t q_row, q_head, k_row, k_head, v_row, v_head, c_page, c_token, c_head, o_row, o_head;
  const int32_t* table;     // [B, table_ld]
  int64_t table_ld;
  int32_t table_width, num_pages, page_shift;
  const int32_t* length;    // [B]
  const int32_t* offsets;   // [B + 1]
  const int32_t* parents;   // [R], or NULL: chains
  int32_t B, R, H, KV, D, dtype;
  float scale;              // of the scores, times log2(e)
  int32_t* error_flag;
  int32_t cus;
  void* work;               // attention_workspace() bytes
  // set at launch
  int32_t G;                // query heads per key head
  int32_t workers;
  int4* piece;              // [workers] item that starts in a worker and ends in a later one
  float2* part_ml;          // [2 * workers][MT] references and weights of the pieces
  float* part;              // [2 * workers][MT][D] unnormalised sums
};

// Most tiles that one request may come to (host check).
int64_t attention_tiles(const AttentionArgs& a);
size_t attention_workspace(const AttentionArgs& a);
hipError_t launch_attention(const AttentionArgs& a, hipStream_t s);

}  // namespace vsv
