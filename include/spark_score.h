/*
 * spark_score.h -- C ABI of the scores of tokens under the head's logits, for
 * NVIDIA GB300 (sm_103a).  Same library and conventions as spark_attn.h.  The
 * reference stops at the logits (turbospark-runtime 0.3.0,
 * src/families/spark/mod.rs, the head); this entry point is this library's
 * own.
 */
#ifndef SPARK_SCORE_H
#define SPARK_SCORE_H

#include "spark_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* alternatives one call returns at most */
#define SPARK_MAX_TOP 32

/* Bytes of the device workspace of spark_token_logprobs for n_rows rows and
 * top_k alternatives (0 for invalid arguments).  Initialise it once with
 * spark_attn_workspace_init; a larger one serves smaller calls. */
size_t spark_logprobs_workspace_bytes(int32_t n_rows, int32_t top_k);

/* For each row x[0 .. vocab) of the logits, with m = max x and
 * Z = sum exp(x - m):
 *   logprob[r]           x[target] - m - ln Z
 *   entropy[r]           ln Z - sum (x - m) exp(x - m) / Z   (nats)
 *   top_ids[r][i]        the i-th highest logit's index, equal logits by the
 *                        lowest index
 *   top_logprobs[r][i]   its log probability
 * all in fp32.
 *   logits  device rows of element type `dtype` (F32 or BF16), row r at
 *           element r * ld (ld >= vocab; any alignment of the element).
 *   targets device [n_rows] int32: -1 asks for none (logprob 0); any other
 *           value outside [0, vocab) raises bit 2 of the error word and gets
 *           a NaN.
 *   top_ids, top_logprobs  device [n_rows][top_k], ignored for top_k 0.
 * Logits of -inf have probability 0.  A row with no distribution (every
 * logit -inf, a +inf or a NaN in it) has NaN in its three fp32 outputs (a
 * target of -1 still 0); its top_ids keep the order above, NaN below -inf.
 * vocab: 1 .. 2^24; n_rows: 1 .. 2^20; top_k: 0 .. min(SPARK_MAX_TOP, vocab).
 * Errors: INVALID_ARG, WORKSPACE before any work is enqueued; CUDA if a
 * launch fails. */
int spark_token_logprobs(const void* logits, int64_t ld, int32_t dtype, int32_t n_rows, int32_t vocab,
                         const int32_t* targets, int32_t top_k, float* logprob, float* entropy, int32_t* top_ids,
                         float* top_logprobs, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SPARK_SCORE_H */
