// C ABI entry points: host-side validation, workspace carving and launch.
// Nothing here synchronises, allocates or reads device memory.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "adjust.hpp"
#include "allocate.hpp"
#include "attention.hpp"
#include "kernels.hpp"
#include "overlap.hpp"
#include "pages.hpp"
#include "probabilistic.hpp"
#include "rows.hpp"

using vsv::VerifyArgs;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t elem_size(int32_t dtype) { return dtype == VSV_BF16 ? 2 : 4; }

bool dtype_ok(int32_t dtype) { return dtype == VSV_F32 || dtype == VSV_BF16; }

// Row whose result word the next launches leave unpublished (-1: none); set
// only by vsv_test_withhold_row_word.
std::atomic<int32_t> g_withheld_row{-1};

// CUs of the current device (cached per device); 0 if the count is unknown.
int device_cus() {
  static int cached[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 0;
  if (dev < 64 && cached[dev] > 0) return cached[dev];
  int cus = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) return 0;
  if (dev < 64) cached[dev] = cus;
  return cus;
}

// Common checks of a batch and its outputs; fills the shared launch args.
vsv_status prepare(const vsv_batch* b, const vsv_outputs* o, void* ws, size_t ws_bytes, int32_t sampled,
                   VerifyArgs* a, bool* empty) {
  *empty = false;
  if (!b || !o) return VSV_EINVAL;
  if (b->num_requests < 0 || b->num_rows < b->num_requests) return VSV_EINVAL;
  if (b->num_requests == 0) {
    if (b->num_rows != 0) return VSV_EINVAL;
    *empty = true;
    return VSV_OK;
  }
  if (!dtype_ok(b->dtype) || b->vocab < 1 || b->vocab > vsv::kMaxVocab || b->ld < b->vocab) return VSV_EINVAL;
  // a row is addressed through a buffer resource with a 32-bit byte size
  if (static_cast<int64_t>(b->vocab) * elem_size(b->dtype) > vsv::kMaxRowBytes) return VSV_EINVAL;
  if (!b->logits || !aligned(b->logits, elem_size(b->dtype))) return VSV_EINVAL;
  if (!b->row_offsets || !b->row_owner) return VSV_EINVAL;
  if (b->num_rows > b->num_requests && !b->draft_tokens) return VSV_EINVAL;
  if (!o->accepted_len || !o->next_token || !o->out_offsets || !o->out_tokens) return VSV_EINVAL;
  // the last row must be addressable with 64-bit element offsets
  if (b->ld > (INT64_MAX / 4) / (b->num_rows > 0 ? b->num_rows : 1)) return VSV_EINVAL;
  if (!ws || !aligned(ws, vsv::kWsAlign)) return VSV_EWORKSPACE;
  if (ws_bytes < vsv::ws_bytes(b->num_requests, b->num_rows, sampled)) return VSV_EWORKSPACE;

  VerifyArgs& v = *a;
  v = VerifyArgs{};
  v.logits = b->logits;
  v.ld = b->ld;
  v.V = b->vocab;
  v.B = b->num_requests;
  v.R = b->num_rows;
  v.dtype = b->dtype;
  v.offsets = b->row_offsets;
  v.owner = b->row_owner;
  v.drafts = b->draft_tokens;
  v.relaxed_k = 1;
  v.accepted_len = o->accepted_len;
  v.next_token = o->next_token;
  v.out_offsets = o->out_offsets;
  v.out_tokens = o->out_tokens;
  v.row_token = o->row_token;
  v.row_lse = o->row_lse;
  v.error_flag = o->error_flag;
  v.slow_rows = o->slow_rows;
  v.withheld_row = g_withheld_row.load(std::memory_order_relaxed);
  char* w = static_cast<char*>(ws);
  v.ws_epoch = reinterpret_cast<uint32_t*>(w);
  v.ws_queue = reinterpret_cast<uint32_t*>(w + 64);
  v.ws_row = reinterpret_cast<uint64_t*>(w + vsv::kWsAlign);
  v.ws_part = reinterpret_cast<uint64_t*>(w + vsv::kWsAlign + vsv::ws_row_bytes(b->num_rows));
  v.cus = device_cus();
  return VSV_OK;
}

// Checks of a matrix of logits given by itself.
bool rows_ok(const void* p, int32_t dtype, int32_t vocab, int64_t ld, int32_t rows) {
  if (!dtype_ok(dtype) || vocab < 1 || vocab > vsv::kMaxVocab || ld < vocab) return false;
  if (static_cast<int64_t>(vocab) * static_cast<int64_t>(elem_size(dtype)) > vsv::kMaxRowBytes) return false;
  return p && aligned(p, elem_size(dtype)) && ld <= (INT64_MAX / 4) / rows;
}

// log2(e) / T as the kernels take it, false unless T and it are positive and
// finite (it is infinite for T below 4.24e-39, where 0 / T would be NaN).
bool exponent_scale(float temperature, float* c) {
  if (!(temperature > 0.f) || !(temperature < INFINITY)) return false;
  *c = static_cast<float>(1.44269504088896340736 / static_cast<double>(temperature));
  return *c < INFINITY;
}

// Checks of a distillation's inputs; fills the shared launch args. The
// caller has dealt with num_rows == 0.
vsv_status prepare_distill(const vsv_distill* d, vsv::DistillArgs* a) {
  if (d->num_top < 1 || d->num_top > VSV_MAX_TOP || !d->ids || !d->top) return VSV_EINVAL;
  float c;
  if (!exponent_scale(d->temperature, &c)) return VSV_EINVAL;
  if (!rows_ok(d->logits, d->dtype, d->vocab, d->ld, d->num_rows)) return VSV_EINVAL;
  *a = vsv::DistillArgs{};
  a->x = vsv::RowsIn{d->logits, d->ld, d->vocab, d->num_rows, d->dtype};
  a->ids = d->ids;
  a->top = d->top;
  a->tlse = d->teacher_lse;
  a->K = d->num_top;
  a->c = c;
  a->inv_t = 1.0 / static_cast<double>(d->temperature);
  a->parts = vsv::distill_parts(d->num_rows, d->vocab, d->dtype);
  return VSV_OK;
}

vsv_status distill_scratch(vsv::DistillArgs* a, void* ws, size_t bytes) {
  if (a->parts < 2) return VSV_OK;
  if (!ws || !aligned(ws, 8) || bytes < vsv_distill_workspace_bytes(a->x.N, a->x.V, a->x.dtype)) return VSV_EWORKSPACE;
  a->part = static_cast<double*>(ws);
  return VSV_OK;
}

bool distill_grad_ok(const vsv::DistillArgs& a, const void* grad, int64_t grad_ld) {
  return grad && aligned(grad, elem_size(a.x.dtype)) && grad_ld >= a.x.V && grad_ld <= (INT64_MAX / 4) / a.x.N;
}

// Checks of an attention's sizes and types, and its launch args without pointers.
bool prepare_attention(const vsv_attention* d, vsv::AttentionArgs* a) {
  if (!dtype_ok(d->dtype)) return false;
  if (d->head_dim != 64 && d->head_dim != 128 && !(d->head_dim == 256 && d->dtype == VSV_BF16)) return false;
  if (d->num_kv_heads < 1 || d->num_heads < d->num_kv_heads || d->num_heads % d->num_kv_heads) return false;
  if (d->num_heads > 65536 || static_cast<int64_t>(d->num_rows) * d->num_heads > INT32_MAX) return false;
  if (d->num_requests < 1 || d->num_requests > VSV_MAX_TREE_REQUESTS || d->num_rows < 1) return false;
  if (d->table_width < 1 || d->num_pages < 1 || d->page_size < 1 || (d->page_size & (d->page_size - 1))) return false;
  *a = vsv::AttentionArgs{};
  a->B = d->num_requests;
  a->R = d->num_rows;
  a->H = d->num_heads;
  a->KV = d->num_kv_heads;
  a->D = d->head_dim;
  a->dtype = d->dtype;
  a->table_width = d->table_width;
  a->num_pages = d->num_pages;
  while ((1 << a->page_shift) < d->page_size) ++a->page_shift;
  a->cus = device_cus();
  return (static_cast<int64_t>(d->table_width) << a->page_shift) <= INT32_MAX - 1024 &&
         vsv::attention_tiles(*a) <= INT32_MAX;
}

}  // namespace

extern "C" {

size_t vsv_workspace_bytes(int32_t num_requests, int32_t num_rows, int32_t sampled) {
  if (num_requests < 0 || num_rows < 0) return 0;
  return vsv::ws_bytes(num_requests, num_rows, sampled);
}

vsv_status vsv_workspace_init(void* workspace, size_t bytes, hipStream_t stream) {
  if (!workspace || !aligned(workspace, 4) || bytes % 4) return VSV_EINVAL;
  return vsv::launch_zero(workspace, bytes, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

vsv_status vsv_verify_greedy(const vsv_batch* batch, int32_t relaxed_topk, const vsv_outputs* out,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  VerifyArgs a;
  bool empty = false;
  const vsv_status st = prepare(batch, out, workspace, workspace_bytes, 0, &a, &empty);
  if (st != VSV_OK || empty) return st;
  if (relaxed_topk < 1 || relaxed_topk > batch->vocab) return VSV_EINVAL;
  a.relaxed_k = relaxed_topk;
  return vsv::launch_verify_greedy(a, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

vsv_status vsv_verify_greedy_relaxed(const vsv_batch* batch, const vsv_relax* relax, const vsv_outputs* out,
                                     void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!relax) return VSV_EINVAL;
  VerifyArgs a;
  bool empty = false;
  const vsv_status st = prepare(batch, out, workspace, workspace_bytes, 0, &a, &empty);
  if (st != VSV_OK || empty) return st;
  if (relax->topk < 1 || relax->topk > batch->vocab) return VSV_EINVAL;
  if (!(relax->margin >= 0.f) || !(relax->margin < INFINITY)) return VSV_EINVAL;
  if (relax->from_position < 0 || relax->after_tokens < 0) return VSV_EINVAL;
  if (relax->num_protected < 0 || relax->num_protected > VSV_MAX_PROTECTED) return VSV_EINVAL;
  if (relax->num_protected > 0 && !relax->protected_ids) return VSV_EINVAL;
  a.relaxed_k = relax->topk;
  a.margin = relax->margin;
  a.from_pos = relax->from_position;
  a.after_tok = relax->after_tokens;
  a.generated = relax->generated;
  a.prot = relax->num_protected > 0 ? relax->protected_ids : nullptr;
  a.nprot = relax->num_protected;
  // top-K alone needs none of the extra decision inputs
  a.relax_var = (relax->margin > 0.f || relax->from_position > 0 || relax->after_tokens > 0 ||
                 relax->num_protected > 0) ? 1 : 0;
  return vsv::launch_verify_greedy(a, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

vsv_status vsv_verify_greedy_tree(const vsv_batch* batch, const int32_t* parents, const vsv_outputs* out,
                                  int32_t* out_rows, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  VerifyArgs a;
  bool empty = false;
  const vsv_status st = prepare(batch, out, workspace, workspace_bytes, 0, &a, &empty);
  if (st != VSV_OK || empty) return st;
  a.parents = parents;
  a.out_rows = out_rows;
  return vsv::launch_verify_greedy_tree(a, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

vsv_status vsv_verify_sampled(const vsv_batch* batch, const float* temperature, const int32_t* top_k,
                              const float* top_p, const float* min_p, uint64_t seed, uint64_t offset,
                              const vsv_outputs* out, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
  VerifyArgs a;
  bool empty = false;
  const vsv_status st = prepare(batch, out, workspace, workspace_bytes, 1, &a, &empty);
  if (st != VSV_OK || empty) return st;
  if (!temperature || !top_k || !top_p || !min_p) return VSV_EINVAL;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.seed = seed;
  a.offset = offset;
  return vsv::launch_verify_sampled(a, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

vsv_status vsv_verify_probabilistic(const vsv_batch* batch, const void* draft_logits, int64_t draft_ld,
                                    const float* temperature, const int32_t* top_k, const float* top_p,
                                    const float* min_p, const float* draft_temperature, uint64_t seed,
                                    uint64_t offset, const vsv_outputs* out, void* workspace,
                                    size_t workspace_bytes, hipStream_t stream) {
  VerifyArgs a;
  bool empty = false;
  const vsv_status st = prepare(batch, out, workspace, workspace_bytes, 0, &a, &empty);
  if (st != VSV_OK || empty) return st;
  if (!temperature || !top_k || !top_p || !min_p || !draft_temperature) return VSV_EINVAL;
  const int32_t D = batch->num_rows - batch->num_requests;
  if (D > 0) {
    if (!draft_logits || !aligned(draft_logits, elem_size(batch->dtype))) return VSV_EINVAL;
    if (draft_ld < batch->vocab || draft_ld > (INT64_MAX / 4) / D) return VSV_EINVAL;
  }
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.seed = seed;
  a.offset = offset;
  const vsv::ProbArgs p{draft_logits, draft_ld, draft_temperature};
  return vsv::launch_verify_probabilistic(a, p, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

vsv_status vsv_draft_confidence(const void* draft_logits, int32_t dtype, int32_t vocab, int64_t ld,
                                int32_t num_draft_rows, const int32_t* selected, float* confidence,
                                float* lse, int32_t* error_flag, hipStream_t stream) {
  if (num_draft_rows < 0) return VSV_EINVAL;
  if (num_draft_rows == 0) return VSV_OK;
  if (!dtype_ok(dtype) || vocab < 1 || ld < vocab) return VSV_EINVAL;
  if (!draft_logits || !aligned(draft_logits, elem_size(dtype)) || !confidence) return VSV_EINVAL;
  if (ld > (INT64_MAX / 4) / num_draft_rows) return VSV_EINVAL;
  vsv::ConfidenceArgs a{draft_logits, ld, vocab, num_draft_rows, dtype, selected, confidence, lse, error_flag};
  return vsv::launch_confidence(a, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

size_t vsv_sample_workspace_bytes(int32_t num_rows, int32_t vocab, int32_t dtype) {
  if (num_rows < 1 || vocab < 1 || !dtype_ok(dtype)) return 0;
  const size_t parts = static_cast<size_t>(vsv::draw_parts(num_rows, vocab, dtype));
  return parts < 2 ? 0 : static_cast<size_t>(num_rows) * parts * vsv::draw_part_bytes(dtype);
}

vsv_status vsv_sample_rows(const void* logits, int32_t dtype, int32_t vocab, int64_t ld, int32_t num_rows,
                           const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                           const float* uniform, int32_t* token, float* logprob, float* lse, int32_t* error_flag,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (num_rows < 0) return VSV_EINVAL;
  if (num_rows == 0) return VSV_OK;
  if (!rows_ok(logits, dtype, vocab, ld, num_rows)) return VSV_EINVAL;
  if (!temperature || !top_k || !top_p || !min_p || !uniform || !token) return VSV_EINVAL;
  const int32_t parts = vsv::draw_parts(num_rows, vocab, dtype);
  if (parts > 1 && (!workspace || !aligned(workspace, 16) ||
                    workspace_bytes < vsv_sample_workspace_bytes(num_rows, vocab, dtype)))
    return VSV_EWORKSPACE;
  const vsv::DrawArgs a{{logits, ld, vocab, num_rows, dtype}, temperature, top_k, top_p, min_p, uniform,
                        token, logprob, lse, error_flag, workspace, parts};
  return vsv::launch_draw(a, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

size_t vsv_top_workspace_bytes(int32_t num_rows, int32_t vocab, int32_t dtype, int32_t k) {
  if (num_rows < 1 || vocab < 1 || k < 1 || k > VSV_MAX_TOP || !dtype_ok(dtype)) return 0;
  const size_t parts = static_cast<size_t>(vsv::top_parts(num_rows, vocab, dtype, k));
  return parts < 2 ? 0 : static_cast<size_t>(num_rows) * parts * vsv::top_part_bytes(k);
}

vsv_status vsv_top_logits(const void* logits, int32_t dtype, int32_t vocab, int64_t ld, int32_t num_rows, int32_t k,
                          float temperature, float* values, int32_t* ids, float* lse, int32_t* error_flag,
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (num_rows < 0) return VSV_EINVAL;
  if (num_rows == 0) return VSV_OK;
  if (!rows_ok(logits, dtype, vocab, ld, num_rows) || !values || !ids) return VSV_EINVAL;
  if (k < 1 || k > VSV_MAX_TOP || k > vocab) return VSV_EINVAL;
  float c;
  if (!exponent_scale(temperature, &c)) return VSV_EINVAL;
  const int32_t parts = vsv::top_parts(num_rows, vocab, dtype, k);
  if (parts > 1 && (!workspace || !aligned(workspace, 16) ||
                    workspace_bytes < vsv_top_workspace_bytes(num_rows, vocab, dtype, k)))
    return VSV_EWORKSPACE;
  const vsv::TopArgs a{{logits, ld, vocab, num_rows, dtype}, k, c, values, ids, lse, error_flag, workspace, parts};
  return vsv::launch_top(a, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

size_t vsv_distill_workspace_bytes(int32_t num_rows, int32_t vocab, int32_t dtype) {
  if (num_rows < 1 || vocab < 1 || !dtype_ok(dtype)) return 0;
  const size_t parts = static_cast<size_t>(vsv::distill_parts(num_rows, vocab, dtype));
  return parts < 2 ? 0 : static_cast<size_t>(num_rows) * (parts * vsv::kPartDoubles + vsv::kStateWords) * sizeof(double);
}

vsv_status vsv_distill_forward(const vsv_distill* d, float* loss, double* state, int32_t* error_flag, void* workspace,
                               size_t workspace_bytes, hipStream_t stream) {
  if (!d || d->num_rows < 0) return VSV_EINVAL;
  if (d->num_rows == 0) return VSV_OK;
  vsv::DistillArgs a;
  vsv_status st = prepare_distill(d, &a);
  if (st != VSV_OK) return st;
  if (!loss || !aligned(state, 8)) return VSV_EINVAL;
  st = distill_scratch(&a, workspace, workspace_bytes);
  if (st != VSV_OK) return st;
  a.loss = loss;
  a.state = state;
  a.error_flag = error_flag;
  return vsv::launch_distill_forward(a, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

vsv_status vsv_distill_backward(const vsv_distill* d, const double* state, const float* weight, void* grad,
                                int64_t grad_ld, hipStream_t stream) {
  if (!d || d->num_rows < 0) return VSV_EINVAL;
  if (d->num_rows == 0) return VSV_OK;
  vsv::DistillArgs a;
  const vsv_status st = prepare_distill(d, &a);
  if (st != VSV_OK) return st;
  if (!state || !aligned(state, 8) || !distill_grad_ok(a, grad, grad_ld)) return VSV_EINVAL;
  a.state = const_cast<double*>(state);
  a.weight = weight;
  a.grad = grad;
  a.grad_ld = grad_ld;
  return vsv::launch_distill_backward(a, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

vsv_status vsv_distill_grad(const vsv_distill* d, const float* weight, float* loss, void* grad, int64_t grad_ld,
                            int32_t* error_flag, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!d || d->num_rows < 0) return VSV_EINVAL;
  if (d->num_rows == 0) return VSV_OK;
  vsv::DistillArgs a;
  vsv_status st = prepare_distill(d, &a);
  if (st != VSV_OK) return st;
  if (!loss || !distill_grad_ok(a, grad, grad_ld)) return VSV_EINVAL;
  st = distill_scratch(&a, workspace, workspace_bytes);
  if (st != VSV_OK) return st;
  a.loss = loss;
  a.weight = weight;
  a.grad = grad;
  a.grad_ld = grad_ld;
  a.error_flag = error_flag;
  // with parts the rows' states pass through the scratch, behind the sums
  if (a.parts > 1) a.state = a.part + static_cast<size_t>(a.x.N) * a.parts * vsv::kPartDoubles;
  return vsv::launch_distill_grad(a, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

vsv_status vsv_allocate_verify(const float* confidence, const int32_t* draft_tokens, int32_t num_requests,
                               int32_t num_drafts, int32_t row_budget, int32_t* verify_len, int32_t* row_offsets,
                               int32_t* row_owner, int32_t* row_source, int32_t* packed_drafts, float* prefix,
                               hipStream_t stream) {
  const int32_t B = num_requests, K = num_drafts, G = row_budget;
  if (B < 0 || K < 0 || G < B) return VSV_EINVAL;
  if (static_cast<int64_t>(G) > static_cast<int64_t>(B) * (K + 1)) return VSV_EINVAL;
  if (B == 0) return VSV_OK;
  if (B > vsv::kMaxAllocRequests || static_cast<int64_t>(B) * K > vsv::kMaxAllocPositions) return VSV_EINVAL;
  if (K > 0 && !confidence) return VSV_EINVAL;
  if (!verify_len || !row_offsets || !row_owner) return VSV_EINVAL;
  if ((draft_tokens == nullptr) != (packed_drafts == nullptr)) return VSV_EINVAL;
  vsv::AllocArgs a{confidence, draft_tokens, B, K, G, verify_len, row_offsets, row_owner, row_source,
                   G > B ? packed_drafts : nullptr, prefix};
  return vsv::launch_allocate(a, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

size_t vsv_tree_attention_workspace_bytes(const vsv_attention* d) {
  vsv::AttentionArgs a;
  return d && prepare_attention(d, &a) ? vsv::attention_workspace(a) : 0;
}

vsv_status vsv_tree_attention(const vsv_attention* d, int32_t* error_flag, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
  if (!d || d->num_requests < 0 || d->num_rows < 0) return VSV_EINVAL;
  if (d->num_requests == 0 || d->num_rows == 0) return VSV_OK;
  vsv::AttentionArgs a;
  if (!prepare_attention(d, &a)) return VSV_EINVAL;
  if (!d->q || !d->k || !d->v || !d->k_cache || !d->v_cache || !d->out) return VSV_EINVAL;
  if (!d->row_offsets || !d->length || !d->block_table) return VSV_EINVAL;
  for (const void* p : {d->q, d->k, d->v, d->k_cache, d->v_cache, static_cast<const void*>(d->out)})
    if (!aligned(p, 16)) return VSV_EINVAL;
  // every stride keeps the 16-byte loads aligned and the last element
  // addressable in 64 bits
  const int64_t unit = 16 / static_cast<int64_t>(elem_size(d->dtype));
  const int64_t strides[][2] = {{d->q_row, d->num_rows},       {d->q_head, d->num_heads},   {d->k_row, d->num_rows},
                                {d->k_head, d->num_kv_heads},  {d->v_row, d->num_rows},     {d->v_head, d->num_kv_heads},
                                {d->out_row, d->num_rows},     {d->out_head, d->num_heads}, {d->cache_page, d->num_pages},
                                {d->cache_token, d->page_size}, {d->cache_head, d->num_kv_heads}};
  for (const auto& s : strides)
    if (s[0] < 0 || s[0] % unit || s[0] > (INT64_MAX / 16) / s[1]) return VSV_EINVAL;
  // no two results in one place
  const int64_t rows_of_head = (d->num_rows - 1) * d->out_row + d->head_dim;
  const int64_t heads_of_row = (d->num_heads - 1) * d->out_head + d->head_dim;
  if ((d->num_heads > 1 && d->out_head < d->head_dim) || (d->num_rows > 1 && d->out_row < d->head_dim)) return VSV_EINVAL;
  if (d->num_heads > 1 && d->num_rows > 1 && d->out_row < heads_of_row && d->out_head < rows_of_head) return VSV_EINVAL;
  if (d->table_ld < d->table_width || d->table_ld > (INT64_MAX / 4) / d->num_requests) return VSV_EINVAL;
  if (!(d->scale > 0.f) || !(d->scale < INFINITY)) return VSV_EINVAL;
  a.scale = static_cast<float>(1.44269504088896340736 * static_cast<double>(d->scale));
  if (!(a.scale > 0.f) || !(a.scale < INFINITY)) return VSV_EINVAL;
  if (!workspace || !aligned(workspace, vsv::kWsAlign) || workspace_bytes < vsv::attention_workspace(a)) return VSV_EWORKSPACE;
  // results go where no other workgroup still reads
  const int64_t e = static_cast<int64_t>(elem_size(d->dtype)), row = d->head_dim * e;
  const int64_t R = d->num_rows, H = d->num_heads, KV = d->num_kv_heads;
  const vsv::Places out{d->out, row, {d->out_row * e, d->out_head * e, 0}, {R, H, 1}};
  const int64_t cache_stride[3] = {d->cache_page * e, d->cache_token * e, d->cache_head * e};
  const vsv::Places others[] = {{d->q, row, {d->q_row * e, d->q_head * e, 0}, {R, H, 1}},
                                {d->k, row, {d->k_row * e, d->k_head * e, 0}, {R, KV, 1}},
                                {d->v, row, {d->v_row * e, d->v_head * e, 0}, {R, KV, 1}},
                                {d->k_cache, row, {cache_stride[0], cache_stride[1], cache_stride[2]}, {d->num_pages, d->page_size, KV}},
                                {d->v_cache, row, {cache_stride[0], cache_stride[1], cache_stride[2]}, {d->num_pages, d->page_size, KV}},
                                {d->lse ? d->lse : workspace, d->lse ? R * H * 4 : 1, {0, 0, 0}, {1, 1, 1}},
                                {workspace, static_cast<int64_t>(vsv::attention_workspace(a)), {0, 0, 0}, {1, 1, 1}}};
  for (const vsv::Places& p : others)
    if (vsv::places_meet(out, p)) return VSV_EINVAL;
  a.q = d->q;
  a.k = d->k;
  a.v = d->v;
  a.k_cache = d->k_cache;
  a.v_cache = d->v_cache;
  a.out = d->out;
  a.lse = d->lse;
  a.q_row = d->q_row;
  a.q_head = d->q_head;
  a.k_row = d->k_row;
  a.k_head = d->k_head;
  a.v_row = d->v_row;
  a.v_head = d->v_head;
  a.o_row = d->out_row;
  a.o_head = d->out_head;
  a.c_page = d->cache_page;
  a.c_token = d->cache_token;
  a.c_head = d->cache_head;
  a.table = d->block_table;
  a.table_ld = d->table_ld;
  a.length = d->length;
  a.offsets = d->row_offsets;
  a.parents = d->parents;
  a.error_flag = error_flag;
  a.work = workspace;
  return vsv::launch_attention(a, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

vsv_status vsv_adjust_logits(const vsv_adjust* d, int32_t* error_flag, hipStream_t stream) {
  if (!d || d->num_requests < 0 || d->num_rows < 0) return VSV_EINVAL;
  if (d->num_requests == 0 || d->num_rows == 0) return VSV_OK;
  if (!rows_ok(d->logits, d->dtype, d->vocab, d->ld, d->num_rows)) return VSV_EINVAL;
  if (!rows_ok(d->out, d->dtype, d->vocab, d->out_ld, d->num_rows)) return VSV_EINVAL;
  if (d->out == d->logits) {
    if (d->out_ld != d->ld) return VSV_EINVAL;
  } else {
    const size_t e = elem_size(d->dtype);
    const uintptr_t x = reinterpret_cast<uintptr_t>(d->logits), y = reinterpret_cast<uintptr_t>(d->out);
    const uintptr_t xe = x + (static_cast<uintptr_t>(d->num_rows - 1) * d->ld + d->vocab) * e;
    const uintptr_t ye = y + (static_cast<uintptr_t>(d->num_rows - 1) * d->out_ld + d->vocab) * e;
    if (x < ye && y < xe) return VSV_EINVAL;
  }
  // (requests without rows leave more drafts than num_rows - num_requests)
  const int64_t least = static_cast<int64_t>(d->num_rows) - d->num_requests;
  const int64_t drafts = d->num_drafts ? d->num_drafts : least > 0 ? least : 0;
  if (!d->row_offsets || drafts < least || drafts < 0 || drafts > d->num_rows || (drafts > 0 && !d->draft_tokens)) return VSV_EINVAL;
  if (d->history &&
      (!d->history_len || d->history_width < 0 || d->history_ld < d->history_width ||
       d->history_ld > (INT64_MAX / 4) / d->num_requests))
    return VSV_EINVAL;
  if (d->num_bias < 0 || (d->bias_offsets && d->num_bias > 0 && (!d->bias_tokens || !d->bias_values))) return VSV_EINVAL;
  if (d->mask && (d->num_masks < 0 || d->mask_ld < (static_cast<int64_t>(d->vocab) + 31) / 32 ||
                  (d->num_masks > 0 && d->mask_ld > (INT64_MAX / 4) / d->num_masks) ||
                  (!d->mask_index && d->num_masks < d->num_rows)))
    return VSV_EINVAL;
  vsv::AdjustArgs a{};
  a.x = d->logits;
  a.y = d->out;
  a.ld = d->ld;
  a.out_ld = d->out_ld;
  a.V = d->vocab;
  a.B = d->num_requests;
  a.R = d->num_rows;
  a.dtype = d->dtype;
  a.offsets = d->row_offsets;
  a.drafts = d->draft_tokens;
  a.parents = d->parents;
  a.history = d->history_width > 0 ? d->history : nullptr;
  a.hist_ld = d->history_ld;
  a.hist_width = d->history_width;
  a.prompt_len = d->prompt_len;
  a.history_len = d->history_len;
  a.repetition = d->repetition;
  a.frequency = d->frequency;
  a.presence = d->presence;
  a.bias_offsets = d->num_bias > 0 ? d->bias_offsets : nullptr;
  a.bias_tokens = d->bias_tokens;
  a.bias_values = d->bias_values;
  a.bias_count = d->num_bias;
  a.mask = d->mask;
  a.mask_ld = d->mask_ld;
  a.mask_rows = d->num_masks;
  a.mask_index = d->mask_index;
  a.num_drafts = static_cast<int32_t>(drafts);
  a.error_flag = error_flag;
  a.cus = device_cus();
  return vsv::launch_adjust(a, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

vsv_status vsv_plan_pages(int32_t* block_table, int64_t table_ld, int32_t table_width, const int32_t* held,
                          const int32_t* length, const int32_t* row_offsets, int32_t num_requests, int32_t num_rows,
                          int32_t* free_pages, int32_t pool_size, const int32_t* free_count, int32_t page_size,
                          int64_t* slot, int32_t* position, int32_t* new_held, int32_t* new_length,
                          int32_t* new_free_count, int32_t* error_flag, hipStream_t stream) {
  const int32_t B = num_requests, R = num_rows;
  if (B < 0 || B > vsv::kMaxPlanRequests || R < 0 || page_size < 1 || pool_size < 1) return VSV_EINVAL;
  if (!row_offsets || !free_pages || !free_count || !new_free_count || (R > 0 && !slot)) return VSV_EINVAL;
  if (B > 0) {
    if (!block_table || !held || !length || !new_held || !new_length) return VSV_EINVAL;
    if (table_width < 1 || table_ld < table_width || table_ld > (INT64_MAX / 4) / B) return VSV_EINVAL;
    // every sum of pages fits 32 bits
    if (static_cast<int64_t>(B) * table_width + pool_size > INT32_MAX) return VSV_EINVAL;
    if (new_held == held || new_length == length) return VSV_EINVAL;
  }
  if (new_free_count == free_count || !aligned(slot, 8)) return VSV_EINVAL;
  const vsv::PagesArgs a{block_table, table_ld, table_width, B, R, page_size, held, length, row_offsets,
                         free_pages, pool_size, free_count, slot, position, new_held, new_length, new_free_count,
                         error_flag};
  return vsv::launch_pages(a, stream) == hipSuccess ? VSV_OK : VSV_EHIP;
}

const char* vsv_status_string(vsv_status status) {
  switch (status) {
    case VSV_OK: return "ok";
    case VSV_EINVAL: return "invalid argument";
    case VSV_EUNSUPPORTED: return "unsupported option";
    case VSV_EWORKSPACE: return "workspace missing, misaligned or too small";
    case VSV_EHIP: return "HIP launch failed";
    case VSV_ELIMIT: return "batch larger than the static scratch serves";
  }
  return "unknown status";
}

vsv_status vsv_test_withhold_row_word(int32_t row) {
  if (row < -1) return VSV_EINVAL;
  g_withheld_row.store(row, std::memory_order_relaxed);
  return VSV_OK;
}

int32_t vsv_version(void) { return 106; }

}  // extern "C"
