// Interface between the C ABI (abi.cpp) and the logit-row operators next to
// verification: drawing tokens, a teacher's top logits, distillation.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "vspec_verify.h"

namespace vsv {

// A packed matrix of logits.
struct RowsIn {
  const void* p;
  int64_t ld;
  int32_t V, N, dtype;
};

struct DistillArgs {
  RowsIn x;                // the student's rows
  const int32_t* ids;      // [N, K]
  const float* top;        // [N, K]
  const float* tlse;       // [N] or NULL: renormalise over the entries
  int32_t K;
  float c;                 // log2(e) / T
  double inv_t;            // 1 / T
  const float* weight;     // [N] upstream gradient of the losses
  float* loss;             // [N]
  double* state;           // [N, kStateWords]
  void* grad;              // [N, grad_ld], the student's type
  int64_t grad_ld;
  int32_t* error_flag;
  double* part;            // [N, parts, kPartDoubles] when parts > 1
  int32_t parts;
};

// What the backward pass needs of a row: the student's exponent references of
// the unnamed tokens and of the whole row (two floats), one over the row's
// sum relative to its own, the factor of the unnamed tokens relative to
// theirs, the teacher's total, and the teacher's log-sum-exp (over the
// entries where none was given).
constexpr int kStateWords = VSV_DISTILL_STATE;
constexpr int kPartDoubles = 4;   // two sums, two exponent references, two maxima (floats)

// Parts a row is cut into, so that a call of few rows still gives every CU
// something to stream; a function of the call's sizes alone, because the
// workspace size depends on it.
int32_t distill_parts(int32_t num_rows, int32_t vocab, int32_t dtype);

hipError_t launch_distill_forward(const DistillArgs& a, hipStream_t s);
hipError_t launch_distill_backward(const DistillArgs& a, hipStream_t s);
hipError_t launch_distill_grad(const DistillArgs& a, hipStream_t s);

struct TopArgs {
  RowsIn x;
  int32_t k;
  float c;                 // log2(e) / T
  float* values;           // [N, k]
  int32_t* ids;            // [N, k]
  float* lse;              // [N] or NULL
  int32_t* error_flag;
  void* part;              // [N, parts] of top_part_bytes when parts > 1
  int32_t parts;
};
// Parts a row is cut into (by the call's sizes alone), and a part's scratch.
int32_t top_parts(int32_t num_rows, int32_t vocab, int32_t dtype, int32_t k);
size_t top_part_bytes(int32_t k);
hipError_t launch_top(const TopArgs& a, hipStream_t s);

struct DrawArgs {
  RowsIn x;
  const float* temperature;   // [N] each
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* uniform;
  int32_t* token;
  float* logprob;
  float* lse;
  int32_t* error_flag;
  void* part;              // [N, parts] of draw_part_bytes when parts > 1
  int32_t parts;
};
// Parts a row is cut into (by the call's sizes alone), and a part's scratch.
int32_t draw_parts(int32_t num_rows, int32_t vocab, int32_t dtype);
size_t draw_part_bytes(int32_t dtype);
hipError_t launch_draw(const DrawArgs& a, hipStream_t s);

}  // namespace vsv
