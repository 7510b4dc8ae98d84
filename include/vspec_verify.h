/*
 * vspec_verify.h -- C ABI of the packed draft-token verification library
 * (MI355X / gfx950).
 *
 * One call verifies a whole ragged batch of speculative-decoding requests
 * whose target logits rows are packed into one matrix. Request i owns the
 * consecutive rows row_offsets[i] .. row_offsets[i+1]-1: its K_i draft-verify
 * rows first, then its bonus row (K_i = row_offsets[i+1] - row_offsets[i] - 1
 * may be 0). Per-request data is reached from a row through the row-owner
 * map, as the xLLM documentation describes its ragged verifier ("Adaptive
 * speculative inference", DSpark section "Launch example": per-request
 * sampling parameters are mapped through device-side packed-row owners, and
 * packing boundaries are never read back to the host).
 *
 * Conventions shared by every entry point:
 *  - Every data pointer is a caller-owned DEVICE pointer unless stated. The
 *    library allocates nothing. What carries over from one verify call to
 *    the next lives in the caller's workspace (see vsv_workspace_bytes): a
 *    call counter, the row queue of sampled verification, and tagged words
 *    through which workgroups hand results to the batch scan. The workspace
 *    is zero-filled once before its first use and every call leaves it
 *    ready for the next; one workspace serves one call at a time, so calls
 *    that may overlap in time (on different streams) need workspaces and
 *    outputs of their own. The host side keeps only a per-device cache of
 *    the CU count; vsv_verify_greedy_static alone uses library-owned device
 *    memory (its own comment states the contract).
 *  - All work is enqueued on `stream` (0 = the null stream). Nothing is
 *    synchronised and nothing is read back to the host; results are valid
 *    once the stream reaches them.
 *  - Host-side argument errors return a status before anything is enqueued.
 *    Conditions that only the device can see (layout, token range, logits,
 *    sampling parameters) set bits in the optional sticky `error_flag` word;
 *    outputs are then unspecified but every write stays inside the buffers.
 *  - bfloat16 logits are raw 16-bit patterns; float32 logits are IEEE single.
 *    Row r starts at element r * ld; only its first `vocab` entries are read.
 *    The logits pointer must be aligned to the element size.
 *  - Token ties are broken by lowest index; values compare as IEEE numbers
 *    (so -0 == +0).
 */
#ifndef VSPEC_VERIFY_H
#define VSPEC_VERIFY_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  VSV_OK = 0,
  VSV_EINVAL = 1,        /* NULL required pointer, bad size, dtype or option  */
  VSV_EUNSUPPORTED = 2,  /* option not built into this library                */
  VSV_EWORKSPACE = 3,    /* workspace NULL, misaligned or smaller than needed */
  VSV_EHIP = 4,          /* the HIP runtime refused the launch                */
  VSV_ELIMIT = 5         /* batch beyond the fixed capacity of an entry point */
                         /* that allocates nothing                            */
} vsv_status;

typedef enum { VSV_F32 = 0, VSV_BF16 = 1 } vsv_dtype;

/* Bits of the sticky device error word (OR-ed in, never cleared). */
#define VSV_FLAG_LAYOUT 1  /* offsets not 0 .. R strictly increasing, or owner map inconsistent */
#define VSV_FLAG_TOKEN 2   /* a draft / selected token outside [0, vocab): treated as a mismatch */
#define VSV_FLAG_LOGITS 4  /* NaN or +inf logit, or a row with no finite logit                  */
#define VSV_FLAG_PARAMS 8  /* temperature < 0, top_p outside (0, 1], min_p outside [0, 1]       */
#define VSV_FLAG_STALLED 16 /* a row's result did not reach the batch scan within the scan's    */
                            /* bounded wait (rows of one launch could not all be resident;   */
                            /* not expected on a dedicated GPU); outputs are unspecified     */
#define VSV_FLAG_PAGES 32  /* the pool of free pages is empty, or a block table names a page     */
                           /* that the cache does not have                                       */

typedef struct {
  const void* logits;          /* [num_rows, ld] vocab-wide target logits             */
  int32_t dtype;               /* vsv_dtype                                           */
  int32_t vocab;               /* 1 <= V < 2^30, and a row of V logits < 2 GiB        */
  int64_t ld;                  /* row stride in elements, >= vocab                    */
  int32_t num_requests;        /* B >= 0                                              */
  int32_t num_rows;            /* R = sum_i (K_i + 1) >= B                            */
  const int32_t* row_offsets;  /* [B + 1]: 0 = off[0] < off[1] < ... < off[B] = R     */
  const int32_t* row_owner;    /* [R]: owner[r] = i for off[i] <= r < off[i+1]        */
  const int32_t* draft_tokens; /* [R - B]: draft j of request i at off[i] - i + j;     */
                               /* may be NULL when R == B                             */
} vsv_batch;

typedef struct {
  int32_t* accepted_len; /* [B] a_i = number of leading accepted drafts              */
  int32_t* next_token;   /* [B] replacement token (a_i < K_i) or bonus (a_i = K_i)   */
  int32_t* out_offsets;  /* [B + 1] exclusive scan of (a_i + 1); out_offsets[B] = total */
  int32_t* out_tokens;   /* [R] capacity; request i writes its a_i accepted drafts   */
                         /* and then next_token[i] at out_offsets[i]                 */
  int32_t* row_token;    /* [R] or NULL: the target token chosen for every row       */
  float* row_lse;        /* [R] or NULL: log-sum-exp of the logits the row uses:     */
                         /* x for greedy rows, x / T for sampled rows                */
  int32_t* error_flag;   /* [1] or NULL: sticky VSV_FLAG_* bits                      */
  int32_t* slow_rows;    /* [1] or NULL: incremented once per sampled row whose     */
                         /* draw needed the exact whole-row path (the row is read  */
                         /* again); diagnostics only, results are identical        */
} vsv_outputs;

/* Bytes of device workspace a verify call needs (B requests, R rows): the
 * words through which rows and workgroups hand their results to the
 * batch-wide scan, a call counter, and the row queue of sampled and
 * probabilistic verification. `sampled` is accepted for compatibility; the
 * size is the same for every entry point. The workspace
 * must be zero-filled before its first use (vsv_workspace_init or any
 * zeroed allocation); after that every call leaves it ready for the next
 * one, so one workspace serves any later call on the same stream. Two calls
 * that may overlap in time need two workspaces. */
size_t vsv_workspace_bytes(int32_t num_requests, int32_t num_rows, int32_t sampled);

/* Zero-fill `bytes` of workspace on `stream` with a kernel (no memset node,
 * so it can be captured into a HIP graph). */
vsv_status vsv_workspace_init(void* workspace, size_t bytes, hipStream_t stream);

/* Greedy target verification.
 * Every row's target token is its arg-max (vllm-hust-vspec 0.13.0 README,
 * "EAGLE features": strict greedy top-1 acceptance on a linear, D2H-free
 * acceptance path). relaxed_topk = 1 accepts a draft iff it equals that
 * token; relaxed_topk = K > 1 accepts a draft whose rank in the order
 * (value desc, index asc) is below K, and then emits the draft token itself
 * (same README, "Scope of support": relaxed top-K acceptance is an explicit
 * quality trade-off whose output may differ from strict greedy). The scan
 * accepts the longest run of leading accepted drafts; the next token is the
 * target token of the first rejected row, or of the bonus row if all pass.
 * Errors: VSV_EINVAL (NULL logits/offsets/owner/required output, vocab < 1,
 * ld < vocab, num_rows < num_requests, relaxed_topk outside [1, vocab],
 * misaligned logits, unknown dtype), VSV_EWORKSPACE, VSV_EHIP. */
vsv_status vsv_verify_greedy(const vsv_batch* batch, int32_t relaxed_topk,
                             const vsv_outputs* out, void* workspace,
                             size_t workspace_bytes, hipStream_t stream);

/* Relaxed greedy acceptance, as the serving switches name it without a
 * formula (vllm-hust-vspec 0.13.0 README: section "Launch" sets a
 * confidence-accept margin of 5.25 and says it relaxes greedy acceptance,
 * output no longer matching the target alone token for token; section
 * "General parameters" lists the margin, its from-position and after-tokens
 * gates and protected token ids; section "EAGLE features" lists top-K
 * relaxed acceptance with an after-tokens gate and the strict prefix).
 * A draft equal to the row's greedy token is always accepted. Any other
 * draft d at draft position j of request i is accepted only if
 * j >= from_position, generated[i] + j >= after_tokens, neither d nor the
 * greedy token is in protected_ids, and either top-K holds (topk > 1 and
 * rank(d) < topk, rank in the order value desc, index asc) or the margin
 * holds (margin > 0 and max - x[d] < margin, evaluated in double from the
 * float values: the draft's target log-probability lies within `margin` of
 * the greedy token's). An accepted draft is emitted as itself; replacement
 * and bonus are greedy tokens. topk = 1, margin = 0 is strict top-1. */
#define VSV_MAX_PROTECTED 256
typedef struct {
  int32_t topk;                 /* >= 1; 1: no top-K relaxation                     */
  float margin;                 /* >= 0, finite; 0: no margin relaxation            */
  int32_t from_position;        /* >= 0: first draft position that may relax        */
  int32_t after_tokens;         /* >= 0: generated[i] + j must reach it to relax    */
  const int32_t* generated;     /* [B] device: tokens request i has generated so    */
                                /* far; NULL counts 0 for every request             */
  const int32_t* protected_ids; /* [num_protected] device, any order; NULL if none  */
  int32_t num_protected;        /* 0 .. VSV_MAX_PROTECTED                           */
} vsv_relax;

/* Greedy verification with relaxed acceptance (vsv_relax above); the rest
 * as vsv_verify_greedy, with the same workspace. Errors: as
 * vsv_verify_greedy, plus VSV_EINVAL for a NULL relax, topk outside
 * [1, vocab], a negative or non-finite margin, negative gates,
 * num_protected outside [0, VSV_MAX_PROTECTED] or NULL protected_ids with
 * num_protected > 0. */
vsv_status vsv_verify_greedy_relaxed(const vsv_batch* batch, const vsv_relax* relax,
                                     const vsv_outputs* out, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream);

/* Greedy verification of trees of drafts. A request's rows are the nodes of
 * a tree: its first row is the root (the last token already emitted), every
 * later row a drafted token, and parents[r] the row its draft follows,
 * counted from the request's first row (0 <= parents[r] < r - off[i]; the
 * root's own entry is not read). Row off[i] + j + 1 carries draft j of
 * request i, at off[i] - i + j in draft_tokens as in every batch: a chain is
 * the tree whose row j has the parent j - 1, and parents = NULL stands for
 * chains throughout. From the root, the walk moves to the lowest row whose
 * parent is the current row and whose draft is the current row's arg-max, as
 * long as there is one (vllm-hust-vspec 0.13.0 README, "Scope of support":
 * EAGLE tree verification; acceptance is strict).
 * Outputs as vsv_verify_greedy, with accepted_len the drafts on the path and
 * next_token the arg-max of its last row, and
 *   out_rows [num_rows] or NULL: at out_offsets[i] the accepted_len[i] + 1
 *                       rows of request i's path, root first: the rows whose
 *                       keys and values belong into the cache, at the
 *                       positions that vsv_plan_pages gives for row_offsets =
 *                       out_offsets
 * out_tokens and out_rows are -1 behind the last path.
 * A request may have at most VSV_MAX_TREE_ROWS rows. VSV_FLAG_LAYOUT: layout
 * as above, more rows, or a parent that is no earlier row of the request (the
 * row is then on no path). Workspace: vsv_workspace_bytes(B, R, 0).
 * Errors: as vsv_verify_greedy. */
#define VSV_MAX_TREE_ROWS 64
vsv_status vsv_verify_greedy_tree(const vsv_batch* batch, const int32_t* parents, const vsv_outputs* out,
                                  int32_t* out_rows, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Greedy verification that allocates nothing, for callers that cannot
 * allocate device memory or pass a workspace: code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation. Same arguments,
 * results and errors as vsv_verify_greedy without the workspace: the
 * library keeps one fixed scratch array per GPU for it, sized for
 * VSV_STATIC_MAX_ROWS packed rows (about 0.95 MiB, held until the process
 * ends), zero-filled on the first call on that GPU. Every call on a GPU
 * shares that GPU's array and leaves its contents for the next call, so
 * calls that may overlap in time on one GPU (different streams, threads)
 * race and must not be issued. No hipMalloc, hipFree or other allocation
 * happens in any call.
 * Errors: as vsv_verify_greedy, plus VSV_ELIMIT for num_rows above
 * VSV_STATIC_MAX_ROWS. */
#define VSV_STATIC_MAX_ROWS 16384
vsv_status vsv_verify_greedy_static(const vsv_batch* batch, int32_t relaxed_topk,
                                    const vsv_outputs* out, hipStream_t stream);

/* Sampled (or mixed) target verification with point-mass drafts.
 * Per-request device arrays [B]: temperature (0 = greedy arg-max for that
 * request), top_k (<= 0 or >= vocab: off), top_p (>= 1: off), min_p
 * (<= 0: off). For T > 0 every row draws its own token from the
 * temperature-scaled distribution filtered in this order: top-k, then top-p
 * renormalised over the top-k survivors (shortest prefix of the rank order
 * whose mass reaches top_p, crossing token kept), then min-p (keep
 * (x - max)/T >= ln(min_p)); the draw is the inverse CDF in rank order at
 * u = (w0 >> 8) * 2^-24, w0 = word 0 of Philox4x32-10 with counter
 * (local row j, request i, offset lo, offset hi) and key (seed lo, seed hi).
 * With deterministic drafts this equals rejection sampling against a point
 * mass: the leading matches are accepted, the first mismatching sample is
 * the replacement and the last row's sample is the bonus (xLLM docs,
 * "Adaptive speculative inference", DSpark section "Launch example").
 * Acceptance is strict (draft == sampled token).
 * Errors: as vsv_verify_greedy, plus VSV_EINVAL for NULL parameter arrays. */
vsv_status vsv_verify_sampled(const vsv_batch* batch, const float* temperature,
                              const int32_t* top_k, const float* top_p,
                              const float* min_p, uint64_t seed, uint64_t offset,
                              const vsv_outputs* out, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

/* Verification with probabilistic drafts: the rejection sampler of
 * speculative decoding. The pages support only the point-mass drafts of
 * vsv_verify_sampled and name this general case as unsupported (xLLM docs,
 * "Adaptive speculative inference", DSpark section "Launch example").
 * draft_logits: device [R - B, draft_ld] rows of the batch's dtype and
 * vocabulary; draft j of request i sits at row off[i] - i + j, like its
 * token. draft_temperature [B]: the temperature the draft was drawn at
 * (0: the draft row's lowest arg-max). With p the target row's law (as in
 * vsv_verify_sampled, or the arg-max's point mass when T = 0) and q the
 * draft row's softmax over its temperature: draft j passes iff
 * u_acc * q(d_j) < p(d_j), u_acc = (w1 >> 8) * 2^-24 from word 1 of the
 * same Philox block as u; the first rejected row emits the inverse-CDF draw
 * of max(0, p - q) in rank order at u (its own draw from p if that residual
 * has no mass); a request whose drafts all pass emits the bonus row's draw.
 * row_token holds each row's emitted-if-first-rejected token (the bonus
 * row's own draw); row_lse is not written; slow_rows counts sampled rows
 * whose survivor set reached below the captured head of the rank order and
 * took the exact whole-row path (several more passes over the row).
 * Workspace: vsv_workspace_bytes(B, R, 0) or more.
 * Errors: as vsv_verify_sampled, plus VSV_EINVAL for NULL draft rows (when
 * R > B) or draft temperatures, draft_ld < vocab or misaligned draft rows.
 * NaN in a draft row sets VSV_FLAG_LOGITS; a negative, NaN or infinite
 * draft temperature sets VSV_FLAG_PARAMS and counts as 0. */
vsv_status vsv_verify_probabilistic(const vsv_batch* batch, const void* draft_logits,
                                    int64_t draft_ld, const float* temperature,
                                    const int32_t* top_k, const float* top_p,
                                    const float* min_p, const float* draft_temperature,
                                    uint64_t seed, uint64_t offset, const vsv_outputs* out,
                                    void* workspace, size_t workspace_bytes,
                                    hipStream_t stream);

/* Draft confidence c_q = exp(y[s_q] - logsumexp(y)) for every draft row q of
 * raw draft logits y (no temperature): the draft probability of the selected
 * token, the score adaptive verification budgets consume (xLLM docs,
 * "Adaptive speculative inference", section "Adaptive target verification
 * from MTP logits"). selected = NULL uses each row's arg-max; an out-of-range
 * selected token gives c_q = 0 and sets VSV_FLAG_TOKEN. lse may be NULL.
 * Errors: VSV_EINVAL (NULL logits/confidence, vocab < 1, ld < vocab,
 * num_draft_rows < 0, misaligned logits, unknown dtype), VSV_EHIP. */
vsv_status vsv_draft_confidence(const void* draft_logits, int32_t dtype,
                                int32_t vocab, int64_t ld, int32_t num_draft_rows,
                                const int32_t* selected, float* confidence,
                                float* lse, int32_t* error_flag,
                                hipStream_t stream);

/* One token per row of logits, drawn with a given random number: the draft
 * side's draw (and any other row's, such as the first token after a prompt).
 * Row r of `num_rows` rows [num_rows, ld] has its own temperature[r] (0 = the
 * lowest-index arg-max), top_k[r], top_p[r] and min_p[r], and the draw is the
 * inverse CDF at uniform[r] in [0, 1): filters, order and draw are those of
 * vsv_verify_sampled, so the same number gives the same token. The sums that
 * decide a cut or a draw hold to about 1e-13 of the row's total for a
 * vocabulary up to 2^18 (vocab / 2^18 times that beyond it); two within 2^-42
 * of each other count as equal.
 *   token [num_rows]    the drawn token
 *   logprob [num_rows]  log-probability of the token under the law it was
 *                       drawn from (after temperature and filters; 0 when
 *                       the temperature is 0), or NULL
 *   lse [num_rows]      log-sum-exp of x / T over the whole row (of x when
 *                       the temperature is 0), or NULL: x[t] / T - lse is the
 *                       log-probability without the filters
 * `workspace` is scratch of vsv_sample_workspace_bytes bytes (0 for many rows
 * or short ones; 16-byte aligned): it needs no initial value and nothing in
 * it outlives the call, so calls are independent of each other.
 * VSV_FLAG_LOGITS: a NaN or +inf logit or no finite one (token 0); VSV_FLAG_PARAMS: a
 * parameter or number outside its range (temperature counts as 0, a filter
 * as off, the number as 0).
 * Errors: VSV_EINVAL (num_rows < 0, NULL logits, parameters, uniform or
 * token, vocab outside 1 .. 2^30 - 1 or a row of 2 GiB, ld < vocab,
 * misaligned logits, unknown dtype), VSV_EWORKSPACE, VSV_EHIP. */
size_t vsv_sample_workspace_bytes(int32_t num_rows, int32_t vocab, int32_t dtype);
vsv_status vsv_sample_rows(const void* logits, int32_t dtype, int32_t vocab, int64_t ld, int32_t num_rows,
                           const float* temperature, const int32_t* top_k, const float* top_p,
                           const float* min_p, const float* uniform, int32_t* token, float* logprob,
                           float* lse, int32_t* error_flag, void* workspace, size_t workspace_bytes,
                           hipStream_t stream);

/* The first k logits of every row in the order (value desc, index asc), with
 * the row's log-sum-exp: what vsv_distill reads of a teacher, taken from the
 * target rows that verification has just read.
 *   values [num_rows, k]  the logits, widened to float
 *   ids [num_rows, k]     their tokens
 *   lse [num_rows]        log-sum-exp of x / temperature, or NULL
 * -inf logits count as the last. A NaN or +inf logit, or a row whose largest
 * x / temperature is beyond float range, sets VSV_FLAG_LOGITS (ids stay
 * inside the row). `workspace`: scratch of vsv_top_workspace_bytes bytes, as in
 * vsv_sample_rows.
 * Errors: VSV_EINVAL (num_rows < 0, NULL logits, values or ids, k outside
 * 1 .. min(vocab, VSV_MAX_TOP), temperature not positive and finite or
 * log2(e) / temperature beyond float32 (below 4.24e-39), vocab,
 * ld, alignment and dtype as above), VSV_EWORKSPACE, VSV_EHIP. */
#define VSV_MAX_TOP 256
size_t vsv_top_workspace_bytes(int32_t num_rows, int32_t vocab, int32_t dtype, int32_t k);
vsv_status vsv_top_logits(const void* logits, int32_t dtype, int32_t vocab, int64_t ld, int32_t num_rows,
                          int32_t k, float temperature, float* values, int32_t* ids, float* lse,
                          int32_t* error_flag, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Distillation of a draft head from the target's top logits. With y a
 * student row, q = softmax(y / T), and a row's used entries (ids[r, k] >= 0;
 * the same id may appear more than once):
 *   teacher_lse NULL:  t = softmax(top / T) over the row's entries,
 *                      loss = sum_k t_k (ln t_k - ln q_k)
 *   teacher_lse given: t_k = exp(top_k / T - teacher_lse), what they leave of
 *                      one, t_r = max(0, 1 - sum t), stands against the
 *                      student's mass q_r outside the row's ids:
 *                      loss = sum_k t_k (ln t_k - ln q_k) + t_r (ln t_r - ln q_r)
 * (the Kullback-Leibler divergence, no factor T^2). Where q_r is below 2^-126
 * (a vocabulary mask that leaves only named tokens), a t_r up to
 * 2^-20 (1 + |teacher_lse|) is the rounding of teacher_lse and counts as 0.
 * Logits whose x / T is below the range of float32 count as -inf. Entries of
 * weight 0 add nothing. A row without a used entry has loss 0 and gradient 0 and its
 * logits are not read. */
typedef struct {
  const void* logits;       /* [num_rows, ld] the student's rows                */
  int32_t dtype;            /* vsv_dtype                                        */
  int32_t vocab;            /* as in vsv_batch                                  */
  int64_t ld;
  int32_t num_rows;         /* >= 0                                             */
  int32_t num_top;          /* entries per row, 1 .. VSV_MAX_TOP                */
  const int32_t* ids;       /* [num_rows, num_top] teacher's tokens; < 0: unused */
  const float* top;         /* [num_rows, num_top] teacher's logits             */
  const float* teacher_lse; /* [num_rows] log-sum-exp of the teacher's whole    */
                            /* row / T, or NULL                                 */
  float temperature;        /* T, positive and finite, log2(e) / T too          */
} vsv_distill;

/* Bytes of scratch that vsv_distill_forward and vsv_distill_grad need (0 for
 * batches of many rows). It needs no initial value and nothing in it outlives
 * the call. */
size_t vsv_distill_workspace_bytes(int32_t num_rows, int32_t vocab, int32_t dtype);

/* Loss of every row, and the state vsv_distill_backward takes (doubles
 * [num_rows, VSV_DISTILL_STATE], or NULL). VSV_FLAG_LOGITS: a NaN or +inf
 * logit in a row that has entries, or none finite; VSV_FLAG_TOKEN: an id at
 * or beyond vocab (counts as unused).
 * Errors: VSV_EINVAL (NULL student, ids, top or loss; sizes, alignment of
 * the logits or the state, dtype, temperature), VSV_EWORKSPACE, VSV_EHIP. */
#define VSV_DISTILL_STATE 5
vsv_status vsv_distill_forward(const vsv_distill* d, float* loss, double* state, int32_t* error_flag,
                               void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Gradient of sum_r weight[r] loss[r] in the student's logits, in their type,
 * rows grad_ld apart (columns beyond vocab are left as they are); weight NULL
 * counts 1 for every row. A row of weight 0 gets zeros and is not read. `d`
 * and `state` as in the forward call; grad may not overlap the logits.
 * Errors: VSV_EINVAL (as vsv_distill_forward, NULL state or grad,
 * grad_ld < vocab, misaligned grad), VSV_EHIP. */
vsv_status vsv_distill_backward(const vsv_distill* d, const double* state, const float* weight, void* grad,
                                int64_t grad_ld, hipStream_t stream);

/* Both in one call, for a step whose row weights are known beforehand: the
 * same results, and a large batch's rows cross HBM once each way.
 * Errors: as the two above. */
vsv_status vsv_distill_grad(const vsv_distill* d, const float* weight, float* loss, void* grad, int64_t grad_ld,
                            int32_t* error_flag, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Adaptive target-verify allocation: how many leading drafts of each request
 * the target verifies under a padded row budget, and the packed layout of
 * those verify rows (xLLM docs, "Adaptive speculative inference": the
 * enable_adaptive_target_verify switch, and section "Adaptive target
 * verification from MTP logits": every draft step still runs, the host fixes
 * the padded target-row budget ahead of the round, and the round's draft
 * confidence scores stay on the device to decide the prefix allocation and
 * the packing).
 *
 * Inputs (device, request-major, B requests of K drafts each):
 *   confidence [B * K]  score of draft j of request i at i * K + j, e.g. the
 *                       output of vsv_draft_confidence; clamped to [0, 1],
 *                       NaN counts as 0; may be NULL when K == 0
 *   draft_tokens [B*K]  the drafts in the same layout, or NULL
 *   row_budget G        host value, B <= G <= B * (K + 1): packed target rows
 *                       including every request's bonus row
 * The predicted acceptance of draft j is the float32 running product of its
 * request's clamped scores through j (left to right). The G - B rows beyond
 * the bonus rows go to the positions with the largest products, ties broken
 * by request, then position, ascending; this maximises the expected number
 * of accepted drafts, and each request receives a prefix of its drafts.
 *
 * Outputs (device, caller-allocated):
 *   verify_len [B]      k_i, the number of drafts request i verifies
 *   row_offsets [B+1]   exclusive scan of (k_i + 1); row_offsets[B] = G
 *   row_owner [G]       request of every packed row
 *   row_source [G]      or NULL: full-width row i * (K + 1) + j that packed
 *                       row off[i] + j stands for (j = k_i is the bonus row)
 *   packed_drafts [G-B] or NULL (exactly when draft_tokens is NULL): draft j
 *                       of request i at off[i] - i + j, the layout that
 *                       vsv_verify_greedy / vsv_verify_sampled read
 *   prefix [B * K]      or NULL: the running products
 * The outputs feed vsv_batch directly (num_rows = G).
 * Errors: VSV_EINVAL (B < 0, K < 0, G outside [B, B * (K + 1)],
 * B > 8192 or B * K > 16384, NULL confidence with K > 0, NULL verify_len /
 * row_offsets / row_owner, exactly one of draft_tokens and packed_drafts
 * NULL), VSV_EHIP. B = 0 (with G = 0) is a no-op. */
vsv_status vsv_allocate_verify(const float* confidence, const int32_t* draft_tokens,
                               int32_t num_requests, int32_t num_drafts, int32_t row_budget,
                               int32_t* verify_len, int32_t* row_offsets, int32_t* row_owner,
                               int32_t* row_source, int32_t* packed_drafts, float* prefix,
                               hipStream_t stream);

/* Attention of packed draft rows over a paged cache: the target's (or a draft
 * model's) attention in the forward pass whose logits are verified. Rows are
 * packed as in vsv_batch; row r of request i sees the request's length[i]
 * cached tokens, the rows on its path from the root of its tree (parents as
 * in vsv_verify_greedy_tree, NULL: chains) and itself:
 *   out[r, h] = sum_t p_t v_t,  p = softmax over the seen t of scale q[r, h] . k_t
 * with key head h / (num_heads / num_kv_heads). The rows' own keys and values
 * are given beside q and need not be in the cache: those of accepted rows are
 * stored after verification (out_rows and vsv_plan_pages), so a rejected
 * draft never holds a slot. What a row does not see cannot reach it, infinite
 * and NaN values included. Scores, softmax and sums are float32; with bfloat16
 * the weights are rounded to bfloat16 for their product with the values.
 * Serving only: there is no backward pass. */
#define VSV_MAX_TREE_REQUESTS 65536
typedef struct {
  const void* q;              /* [num_rows, num_heads, head_dim]                        */
  const void* k;              /* [num_rows, num_kv_heads, head_dim]                     */
  const void* v;
  const void* k_cache;        /* [num_pages, page_size, num_kv_heads, head_dim]         */
  const void* v_cache;        /* the same strides as k_cache                            */
  void* out;                  /* [num_rows, num_heads, head_dim], no other's memory     */
  float* lse;                 /* [num_rows, num_heads] log-sum-exp of the seen scores   */
                              /* (natural, scaled), or NULL                             */
  /* strides in elements (the last dimension's is 1): of rows and heads, and   */
  /* of the caches' pages, tokens and heads; every pointer and every stride in */
  /* bytes is a multiple of 16, and no two rows or heads of out overlap        */
  int64_t q_row, q_head, k_row, k_head, v_row, v_head, out_row, out_head;
  int64_t cache_page, cache_token, cache_head;
  int32_t dtype;              /* vsv_dtype of every matrix                              */
  int32_t head_dim;           /* 64, 128, or 256 (bfloat16 alone)                       */
  int32_t num_heads;          /* a multiple of num_kv_heads                             */
  int32_t num_kv_heads;
  int32_t num_requests;       /* 0 .. VSV_MAX_TREE_REQUESTS                             */
  int32_t num_rows;           /* R >= 0                                                 */
  const int32_t* row_offsets; /* [B + 1], not falling, within 0 .. R; at most           */
                              /* VSV_MAX_TREE_ROWS rows a request, which may have none; */
                              /* rows at or beyond off[B] are left as they are          */
  const int32_t* parents;     /* [R] or NULL                                            */
  const int32_t* length;      /* [B] tokens of each request in the cache, may be 0      */
  const int32_t* block_table; /* [B, table_ld] pages of each request                    */
  int64_t table_ld;
  int32_t table_width;        /* pages a request may have                               */
  int32_t num_pages;          /* of the cache                                           */
  int32_t page_size;          /* tokens of a page, a power of two                       */
  float scale;                /* positive and finite, times log2(e) too                 */
} vsv_attention;

/* `workspace`: scratch of vsv_tree_attention_workspace_bytes bytes (256-byte
 * aligned; of the struct it reads sizes and types alone, 0 for an invalid one).
 * It needs no initial value and nothing in it outlives the call; calls that
 * may overlap in time need scratch of their own. Results do not
 * depend on anything but the inputs and the device's number of CUs.
 * VSV_FLAG_LAYOUT: offsets, lengths (beyond table_width pages) or row counts
 * outside their range (the request's rows are left as they are), or a parent that is
 * no earlier row (the row then sees the context and itself alone);
 * VSV_FLAG_PAGES: a page outside 0 .. num_pages - 1 (page 0 is read for it).
 * Errors: VSV_EINVAL (NULL pointers, sizes, strides, alignment, dtype, scale;
 * an out that shares memory with another matrix, lse or the workspace (slices
 * of the same rows are told apart; a matrix that overlaps itself counts whole);
 * num_rows * num_heads beyond 2^31 - 1; table_width * page_size beyond it, or
 * so large that a request's work could pass 2^31 tiles), VSV_EWORKSPACE,
 * VSV_EHIP. */
size_t vsv_tree_attention_workspace_bytes(const vsv_attention* a);
vsv_status vsv_tree_attention(const vsv_attention* a, int32_t* error_flag, void* workspace, size_t workspace_bytes,
                              hipStream_t stream);

/* Penalties, biases and grammar masks on packed rows of logits, before they
 * are verified or drawn from. Row r of request i stands behind a path of
 * drafts (in a chain the drafts before it; with `parents`, those from the
 * root to its node, its own included; draft tokens as in vsv_batch). With c
 * the occurrences of a token in the request's output and on that path, and
 * "seen" if it occurs there or in the prompt:
 *   y = seen ? (x > 0 ? x / repetition[i] : x * repetition[i]) : x
 *   y = y - frequency[i] * c - (c > 0 ? presence[i] : 0)
 *   y = y + bias of the token (the last entry that names it)
 *   y = -inf where the row's mask has a 0 bit
 * in float32 (the division as a product with the rounded reciprocal), rounded
 * once to the logits' type. A mask may leave a row nothing (all -inf). */
typedef struct {
  const void* logits;           /* [num_rows, ld]                                       */
  void* out;                    /* [num_rows, out_ld], or the logits themselves with    */
                                /* out_ld == ld; no other overlap                       */
  int32_t dtype;                /* vsv_dtype                                            */
  int32_t vocab;                /* as in vsv_batch                                      */
  int64_t ld, out_ld;           /* columns beyond vocab are left as they are            */
  int32_t num_requests;         /* B >= 0                                               */
  int32_t num_rows;             /* R >= 0                                               */
  const int32_t* row_offsets;   /* [B + 1], not falling, within 0 .. R: requests        */
                                /* without rows come last, and rows at or beyond        */
                                /* off[B] are left as they are                          */
  const int32_t* draft_tokens;  /* [num_drafts], may be NULL when R <= B and no row     */
                                /* carries one                                          */
  const int32_t* parents;       /* [R] as in vsv_verify_greedy_tree (at most            */
                                /* VSV_MAX_TREE_ROWS rows a request), NULL: chains of   */
                                /* any length                                           */
  const int32_t* history;       /* [B, history_ld] tokens: the prompt, then the output; */
                                /* NULL: none                                           */
  int64_t history_ld;
  int32_t history_width;        /* entries of a row that may be read                    */
  const int32_t* prompt_len;    /* [B] tokens of the prompt, or NULL: 0                 */
  const int32_t* history_len;   /* [B] tokens of both (required with history)           */
  const float* repetition;      /* [B] 2^-126 .. 2^126, or NULL: 1                      */
  const float* frequency;       /* [B] finite, or NULL: 0                               */
  const float* presence;        /* [B] finite, or NULL: 0                               */
  const int32_t* bias_offsets;  /* [B + 1], or NULL: no biases                          */
  const int32_t* bias_tokens;   /* [num_bias]                                           */
  const float* bias_values;     /* [num_bias] finite or -inf                            */
  int32_t num_bias;
  const uint32_t* mask;         /* [num_masks, mask_ld] words, bit v % 32 of word       */
                                /* v / 32 allows token v; NULL: none                    */
  int64_t mask_ld;              /* >= (vocab + 31) / 32                                 */
  int32_t num_masks;
  const int32_t* mask_index;    /* [R] row of `mask`, negative: the row is not masked;  */
                                /* NULL: row r's mask is row r                          */
  int32_t num_drafts;           /* entries of draft_tokens, R - B .. R: with requests   */
                                /* that have no rows there are more drafts than R - B;  */
                                /* 0: R - B                                             */
} vsv_adjust;

/* VSV_FLAG_TOKEN: a token of a history, path or bias outside the vocabulary
 * (it counts nowhere; histories and paths are read for requests with a
 * penalty in force, biases and masks always); VSV_FLAG_PARAMS: a penalty or bias outside its range
 * (counts as off); VSV_FLAG_LAYOUT: offsets, lengths, parents or mask rows
 * outside theirs (a request with bad offsets is left as it is). Bits of
 * requests without any row are not looked at.
 * Errors: VSV_EINVAL (NULL struct, logits, out or row_offsets; draft_tokens
 * NULL with R > B, history without history_len, bias_offsets without tokens
 * and values when num_bias > 0; sizes, strides, alignment or dtype; an
 * overlapping out), VSV_EHIP. */
vsv_status vsv_adjust_logits(const vsv_adjust* a, int32_t* error_flag, hipStream_t stream);

/* Block tables and slots of rows to store, from lengths that only the device
 * knows. Request i has length[i] tokens in a cache of pages of page_size
 * tokens and row_offsets[i + 1] - row_offsets[i] rows to store behind them
 * (out_offsets of a verify call, or the rows of a prompt; none for a request
 * that waits). It needs p = ceil((length[i] + rows) / page_size) pages and
 * holds held[i]. Free pages are a stack, free_pages[0 .. free_count - 1]:
 * first, in request order, every request that holds more than it needs puts
 * its pages p .. held - 1 on it (a request that has ended: length 0 and no
 * rows); then, in request order, those that need more take theirs from its
 * top. A request that the stack cannot serve any more, and every later one that
 * needs pages, is left as it is (VSV_FLAG_PAGES; slots -1).
 *   block_table [B, table_ld]  read, and written at the pages taken; entries
 *                       that are given back keep their values
 *   free_pages [pool_size]  read, and written above free_count
 *   slot [num_rows]     page * page_size + position % page_size of every
 *                       row, -1 for rows at or beyond row_offsets[B]
 *   position [num_rows] or NULL: position of the row in its request, or -1
 *   new_held, new_length [B], new_free_count [1]  the state behind the call;
 *                       none may overlap an input, so that a call that is
 *                       repeated on the same inputs gives the same results
 * VSV_FLAG_LAYOUT: offsets that fall or leave 0 .. R, a negative length, a
 * held or needed count beyond table_width (the request is left as it is), a
 * count beyond pool_size, or a negative page.
 * Errors: VSV_EINVAL (B outside 0 .. 8192, num_rows < 0, page_size < 1, table_width or
 * pool_size < 1, B * table_width + pool_size beyond 2^31 - 1, table_ld <
 * table_width, NULL pointers),
 * VSV_EHIP. B = 0 writes slots, positions and the count alone. */
vsv_status vsv_plan_pages(int32_t* block_table, int64_t table_ld, int32_t table_width, const int32_t* held,
                          const int32_t* length, const int32_t* row_offsets, int32_t num_requests, int32_t num_rows,
                          int32_t* free_pages, int32_t pool_size, const int32_t* free_count, int32_t page_size,
                          int64_t* slot, int32_t* position, int32_t* new_held, int32_t* new_length,
                          int32_t* new_free_count, int32_t* error_flag, hipStream_t stream);

/* Goodput step selection: the step count of the next decode batch from
 * completed verification results (xLLM docs, "Adaptive speculative
 * inference", section "Adaptive draft step (MTP)" and its policy options:
 * one step count s for the whole batch, the one maximising
 * B * (1 + sum(prefix_acceptance[:s])) / cost_ms(s); prefix acceptance
 * counted over a window of completed batches (default 20); candidates
 * re-scored every update_interval batches (default 5); the step changes only
 * when the predicted relative gain is strictly above switch_min_gain
 * (default 0.05)).
 * HOST code and HOST pointers: the caller reads accepted lengths back with
 * its normal results and passes the full-round cost of every candidate.
 * Rules the page leaves open: candidates are 1 .. max_steps and the
 * controller starts at max_steps; prefix acceptance j is the share, among
 * the window's requests that verified at least j + 1 drafts, of those that
 * accepted at least j + 1 (a position no request in the window verified
 * keeps its last estimate, 0 before any); equal scores go to the smaller
 * step count. The caller owns the state; one state per controller, not
 * thread-safe. */
#define VSV_GOODPUT_MAX_STEPS 32
#define VSV_GOODPUT_MAX_WINDOW 64
typedef struct {
  int32_t max_steps;        /* S: largest step count                           */
  int32_t window_size;      /* completed batches counted                       */
  int32_t update_interval;  /* batches between re-scorings                     */
  double switch_min_gain;   /* strict relative gain needed to switch           */
  int32_t current;          /* step count in force                             */
  int32_t since;            /* batches observed since the last re-scoring      */
  int32_t filled;           /* batches in the window                           */
  int32_t head;             /* window slot of the next batch                   */
  int32_t reached[VSV_GOODPUT_MAX_WINDOW][VSV_GOODPUT_MAX_STEPS];   /* per batch: */
  int32_t accepted[VSV_GOODPUT_MAX_WINDOW][VSV_GOODPUT_MAX_STEPS];  /* requests that verified / accepted > j drafts */
  double estimate[VSV_GOODPUT_MAX_STEPS];  /* prefix acceptance per position */
} vsv_goodput;

/* Reset `state`. Errors: VSV_EINVAL (NULL state, max_steps outside
 * [1, VSV_GOODPUT_MAX_STEPS], window_size outside [1, VSV_GOODPUT_MAX_WINDOW],
 * update_interval < 1, non-finite switch_min_gain). */
vsv_status vsv_goodput_init(vsv_goodput* state, int32_t max_steps, int32_t window_size,
                            int32_t update_interval, double switch_min_gain);

/* Record one completed batch: accepted_len[i] and verify_len[i] (drafts the
 * target verified) of its num_requests requests, host arrays. Positions at or
 * beyond max_steps are not counted. Errors: VSV_EINVAL (NULL state or arrays,
 * num_requests < 0, an entry with accepted_len < 0 or > verify_len); the batch
 * is then not recorded. */
vsv_status vsv_goodput_observe(vsv_goodput* state, const int32_t* accepted_len,
                               const int32_t* verify_len, int32_t num_requests);

/* The step count for the next batch of batch_size requests. cost_ms[s - 1] is
 * the full-round cost of s steps (host array of max_steps positive values);
 * re-scores when update_interval batches were observed since the last
 * re-scoring. Errors: VSV_EINVAL (NULL state, cost_ms or step, a cost that is
 * not positive and finite, batch_size < 0). */
vsv_status vsv_goodput_step(vsv_goodput* state, const double* cost_ms, int32_t batch_size,
                            int32_t* step);

/* One scoring without state: the step count among 1 .. max_steps that the
 * rule above picks from `current`, given prefix_acceptance[max_steps] and
 * cost_ms[max_steps] (host arrays). Returns -1 for invalid arguments. */
int32_t vsv_goodput_select(const double* prefix_acceptance, const double* cost_ms,
                           int32_t max_steps, int32_t batch_size, int32_t current,
                           double switch_min_gain);

/* Static description of a status code. */
const char* vsv_status_string(vsv_status status);

/* Test hook for the batch scan's bounded wait (VSV_FLAG_STALLED), which a
 * dedicated GPU never reaches. Until called again with -1, every later
 * verify launch (vsv_verify_greedy, _relaxed and _static,
 * vsv_verify_sampled and vsv_verify_probabilistic) computes row `row` as
 * usual but leaves its result word unpublished. The launch's scan then
 * spends its poll budget on that word (well under a second), sets
 * VSV_FLAG_STALLED, uses the stale word and completes: outputs stay inside
 * their buffers and the workspace serves the next call as usual.
 * Process-wide; read when a call is made.
 * Returns VSV_EINVAL for row < -1. */
vsv_status vsv_test_withhold_row_word(int32_t row);

/* Library ABI version (major * 100 + minor). */
int32_t vsv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* VSPEC_VERIFY_H */
