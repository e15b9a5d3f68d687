/*
 * tide_lm_ops.h -- C ABI of libtide's operators at the two ends of a language
 * model's training step, around the blocks whose operators tide_ops.h declares:
 *
 *   token embedding, and its gradient by sorted tokens
 *   log probabilities of given tokens, entropy and alternatives, and their gradient
 *   the global norm of many gradients, and clipping by it
 *
 * The conventions of tide_ops.h hold: row-major matrices with a row stride in
 * elements, pointers aligned to their element size, work enqueued on `stream`
 * of the current device, no allocation, calls that can be captured into a
 * CUDA graph after a first call of the kind, fp32 arithmetic (or more) with one
 * rounding per output, results that do not depend on timing, caller-owned
 * workspaces of their own for calls that may overlap, outputs that overlap
 * neither inputs nor each other except where said, the same status codes.
 */
#ifndef TIDE_LM_OPS_H
#define TIDE_LM_OPS_H

#include "tide_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Whole numbers that name tokens. */
typedef enum tide_index { TIDE_I32 = 0, TIDE_I64 = 1 } tide_index;

/* ---- token embedding ------------------------------------------------------
 * out[t] = scale * weight[ids[t]]: ids [tokens] of type `index`, weight
 * [vocab, cols] and out [tokens, cols] of `dtype`.  An id outside 0..vocab-1
 * (padding) gives a row of zeros.  At most 2^31 - 1 tokens, 2^31 - 2 rows of weight
 * and 2^24 columns (UNIMPLEMENTED beyond). */
tide_status tide_embedding(int64_t tokens, int64_t vocab, int64_t cols, int32_t index, const void* ids, int32_t dtype,
                           const void* weight, int64_t ldw, float scale, void* out, int64_t ldo, void* stream);

/* dweight[v] = scale * the sum of dy[t] over the t with ids[t] == v, zero
 * where there are none; ids outside 0..vocab-1 take no part.  With accumulate
 * not 0 that is added to what dweight holds (the sum in fp32, rounded once), and rows
 * that no id names are left as they are.  dy [tokens, cols] and dweight
 * [vocab, cols] are of `dtype`.  The sum runs in a fixed order.  Limits as above. */
int64_t tide_embedding_backward_workspace(int64_t tokens, int64_t vocab, int64_t cols);
tide_status tide_embedding_backward(int64_t tokens, int64_t vocab, int64_t cols, int32_t index, const void* ids,
                                    int32_t dtype, const void* dy, int64_t lddy, float scale, void* dweight,
                                    int64_t lddw, int32_t accumulate, void* workspace, int64_t workspace_bytes,
                                    void* stream);

/* ---- log probabilities ----------------------------------------------------
 * For each row of logits [rows, vocab] (`dtype`), with z = scale * logits
 * (scale 2^-120 to 2^64: 1 / temperature) and p = exp(z - lse):
 *   lse [rows]                log(sum over v of exp(z[v]))
 *   lse_parts [rows, 2]       the largest logit, and lse less scale times that
 *   logp [rows]               z[targets] - lse; 0 for a target outside 0..vocab-1
 *   entropy [rows]            -sum over v of p[v] log p[v]
 *   top_tokens, top_logp      the `top` largest logits' tokens, the largest first,
 *   [rows, top]               equal ones by the lower token, and their z - lse
 * All but top_tokens (int32) are fp32; each of lse, lse_parts, entropy,
 * top_logp and top_tokens may be NULL, and targets with logp.  top is 0 to 32 and at most vocab.
 * A logit of -inf is a token of probability 0.  A row without any other (or
 * with vocab 0) has lse and both its parts -inf, entropy 0, logp -inf (0 for a target outside)
 * and top_logp -inf.  A row that holds +inf or NaN has NaN in all of them (and in
 * lse_parts' second) but for targets outside; its top_tokens still go by its logits,
 * NaN counting as -inf.
 * At most 2^31 - 1 rows of 2^31 - 17 logits (UNIMPLEMENTED beyond), here and for the gradient. */
tide_status tide_log_probs(int64_t rows, int64_t vocab, int32_t dtype, const void* logits, int64_t ldl, float scale,
                           int32_t index, const void* targets, float* logp, float* lse, float* lse_parts,
                           float* entropy, int32_t top, float* top_logp, int64_t ld_top_logp, int32_t* top_tokens, int64_t ld_top_tokens,
                           void* stream);

/* The gradient, from what the forward call gave: with g = dlogp [rows] (taken as
 * 0 for a target outside 0..vocab-1), h = dentropy [rows] and p = exp(z - lse),
 *   dlogits = scale * (g * ([v == target] - p) - h * p * (log p + entropy)).
 * targets and dlogp are given together or both NULL (g = 0), likewise entropy
 * and dentropy (h = 0).  lse is the forward call's at the same scale; a row with
 * lse -inf has no gradient.  fp32 holds lse to 2^-24 of it, and ln p is off by as much
 * as lse is; lse_parts, given in lse's place, makes p right whatever the logits' size,
 * as of a row that a finite mask covers whole (lse is not read then, and may be NULL).
 * dlogits [rows, vocab] is of `dtype` and may be logits. */
tide_status tide_log_probs_backward(int64_t rows, int64_t vocab, int32_t dtype, const void* logits, int64_t ldl,
                                    float scale, const float* lse, const float* lse_parts, int32_t index,
                                    const void* targets, const float* dlogp, const float* entropy, const float* dentropy, void* dlogits,
                                    int64_t ldd, void* stream);

/* ---- gradient norm and clipping -------------------------------------------
 * Lists of `count` tensors: host arrays, read during the call only, of device
 * addresses, numbers of (contiguous) elements and element types (tide_dtype).
 * An address may be NULL where the number is 0.  At most 2^40 elements a tensor (UNIMPLEMENTED beyond). */

/* norm[0] = the square root of the sum of all tensors' squared elements.
 * Squares are never lost to fp32's range.  An infinity gives +inf, NaN gives NaN (also beside one).
 * The norm of several lists' norms is the norm of all their tensors. */
int64_t tide_grad_norm_workspace(int32_t count, const int64_t* numels, const int32_t* dtypes);
tide_status tide_grad_norm(int32_t count, const void* const* tensors, const int64_t* numels, const int32_t* dtypes,
                           float* norm, void* workspace, int64_t workspace_bytes, void* stream);

/* outs[i] = tensors[i] * c, c = max_norm / (norm[0] + eps) where that is
 * below 1 (an fp32 number), 1 elsewhere, and NaN where norm[0] is NaN (so +inf clips to zeros, infinite
 * elements to NaN).  outs[i] may be tensors[i] (all of them, then with c = 1 nothing is
 * touched); it has the same number and type of elements.  norm is read on the
 * device.  max_norm and eps are not negative and not NaN. */
tide_status tide_grad_clip(int32_t count, const void* const* tensors, void* const* outs, const int64_t* numels,
                           const int32_t* dtypes, const float* norm, float max_norm, float eps, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TIDE_LM_OPS_H */
