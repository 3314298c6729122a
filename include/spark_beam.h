/*
 * spark_beam.h -- C ABI of beam search over the head's logits: the best
 * continuations of every request's beams, and the beams' states in their new
 * order, for NVIDIA GB300 (sm_103a).  Same library and conventions as
 * spark_attn.h.  The reference samples one sequence at a time
 * (turbospark-runtime 0.3.0, src/families/spark/mod.rs, ends at the logits);
 * these entry points are this library's own.
 *
 * A request (group) has n_beams slots next to one another: beam b of group i
 * is slot i * n_beams + b.  The outputs are those spark_pages_remap takes:
 * parent, keep_len and new_len of every slot, on the device, so that a step
 * (select, remap, reorder, decode) is enqueued without a host read.
 */
#ifndef SPARK_BEAM_H
#define SPARK_BEAM_H

#include "spark_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* beams of a group at most */
#define SPARK_MAX_BEAMS 32
/* states one spark_beam_reorder moves at most */
#define SPARK_MAX_BEAM_STATES 32

/* Bytes of the device workspace of spark_beam_select and spark_beam_reorder
 * (0 for invalid arguments).  Initialise it once with
 * spark_attn_workspace_init; it serves one call at a time. */
size_t spark_beam_workspace_bytes(int32_t n_groups, int32_t n_beams);

/* One step of beam search.  With z = log_softmax of a slot's logits, a live
 * beam offers every token v at score[slot] + z[v]; a beam that has ended
 * (done != 0) offers itself, once, at its score, as token `eos`.  The n_beams
 * best offers of a group become its new beams, best first; equal scores go to
 * the lower beam, then the lower token.
 *   logits   device rows of element type `dtype` (F32 or BF16), row of slot s
 *            at element s * ld (ld >= vocab; any alignment of the element).
 *            Rows of beams that have ended, or of score -inf, are not read.
 *   score    device [slots] fp32: summed log probabilities; -inf: the slot
 *            offers nothing (all but the first beam of a group before its
 *            first step; a slot left over).
 *   done     device [slots] int32; null: none has ended.
 *   length   device [slots] int32: positions of each beam; null with keep_len
 *            and new_len: they are not wanted.
 *   eos      the token that ends a beam, or -1: none does (done is null then).
 *   new_score, token, parent, new_done   device [slots]: score, token, the slot
 *            it continues, and whether it has ended (done before, or token ==
 *            eos).  new_done may be null where eos is -1.
 *   keep_len, new_len   device [slots]: length[parent], and one more unless the
 *            parent had ended.
 * A group with fewer offers than beams leaves slots over: score -inf, token
 * and parent -1, done 1, lengths 0.  Logits of -inf are no offers; a row with
 * no distribution (every logit -inf, a +inf or a NaN in it) offers nothing,
 * a score of +inf or NaN neither, nor what would have a score below fp32's
 * range.
 * Sums are fp32, the scores are compared in 64 bits and rounded to fp32 once.
 * new_score may be score, new_done done and new_len length; otherwise no output
 * overlaps another array of the call (this is not checked).
 * n_beams: 1 .. SPARK_MAX_BEAMS; n_groups * n_beams: 1 .. SPARK_MAX_BATCH;
 * vocab: 1 .. 2^24.
 * Errors: INVALID_ARG, WORKSPACE before any work is enqueued; CUDA if a
 * launch fails. */
int spark_beam_select(const void* logits, int64_t ld, int32_t dtype, int32_t n_groups, int32_t n_beams, int32_t vocab,
                      const float* score, const int32_t* done, const int32_t* length, int32_t eos, float* new_score,
                      int32_t* token, int32_t* parent, int32_t* new_done, int32_t* keep_len, int32_t* new_len,
                      void* workspace, size_t workspace_bytes, void* stream);

/* One state of the beams: a row of `pitch` bytes for each slot (a multiple of
 * 4, rows 4-byte aligned).
 *   elem 0   the whole row goes along.
 *   elem > 0 bytes of one position (a multiple of 4): the first keep_len of
 *            them go along (a token history).
 *   push     device [slots] int32 (elem 4 only, or null): where new_len is more
 *            than keep_len, push[s] is written behind the positions kept.
 * No dst overlaps another, a src, a push or the lists of the call. */
typedef struct spark_beam_state {
  const void* src;
  void* dst;
  int64_t pitch;
  int32_t elem;
  const int32_t* push;
} spark_beam_state;

/* dst row s = src row parent[s] of every state (host array).  A slot with
 * parent -1 is left as it was.  A parent outside [-1, n_slots), lengths that a
 * row has no room for or new_len below keep_len: bit 2 of the error word, and
 * the row (of that state) is left as it was.
 *   parent, keep_len, new_len   device [n_slots], as spark_beam_select leaves
 *            them; the lengths may be null where every elem is 0.
 * n_slots: 1 .. SPARK_MAX_BATCH; n_states: 1 .. SPARK_MAX_BEAM_STATES; pitch
 * up to 2^31 - 4.
 *   workspace >= spark_beam_workspace_bytes (of any arguments).
 * Errors as spark_beam_select. */
int spark_beam_reorder(const int32_t* parent, const int32_t* keep_len, const int32_t* new_len, int32_t n_slots,
                       const spark_beam_state* states, int32_t n_states, void* workspace, size_t workspace_bytes,
                       void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SPARK_BEAM_H */
