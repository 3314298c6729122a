/*
 * spark_paged.h -- C ABI of the paged KV cache: page tables, the write of new
 * rows, attention of every sequence's new tokens over its pages, and the
 * attention block on a paged cache, for NVIDIA GB300 (sm_103a).  Same library
 * and conventions as spark_attn.h (device pointers owned by the caller,
 * 16-byte aligned, int32 arrays 4-byte; work enqueued on `stream`; SPARK_OK
 * or a negative spark_status; the current device is the pointers').  Pages
 * have no counterpart in turbospark-runtime 0.3.0, whose cache is one
 * contiguous slot range per sequence (src/kv_write.rs).  The attention is
 * that of spark_attn.h: query head h reads KV head h / (n_q / n_kv), scale
 * `geom.scale`, causal over the whole history (SPARK_FULL) or the last
 * `geom.window` positions (SPARK_SLIDING).
 *
 * A cache is a pool of pages of page_size rows, one pool for each layer, all
 * layers sharing the page numbers.  Position x of sequence s lives in page
 * table[s][x / page_size], row x % page_size.
 *
 * Page tables, starts and lengths are DEVICE arrays, read when the work
 * runs, so a captured call replays with new lengths (spark_attn_paged with
 * the rope positions of its capture, see there).  What the host cannot see
 * the kernels check: an entry out of range raises bit 2 of the workspace's
 * error word (spark_attn_error_word), no memory outside the buffers is read
 * or written, and the results of the sequence it belongs to are unspecified.
 *
 * A workspace serves one call at a time: calls that share one are ordered on
 * a stream, captured graphs that share one do not run at once.  After an
 * error word with bit 1 (a wait that ran out of time) it is initialised
 * again with spark_attn_workspace_init before its next use.
 */
#ifndef SPARK_PAGED_H
#define SPARK_PAGED_H

#include "spark_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* new tokens and page-table entries one call takes at most */
#define SPARK_MAX_PAGED_TOKENS (1 << 17)
#define SPARK_MAX_TABLE_PAGES (1 << 20)
/* layers whose pages one spark_pages_* call moves at most */
#define SPARK_MAX_PAGE_POOLS 128

/* One layer's pages (device, caller-owned): K and V are two buffers of
 * [n_pages][page_size][n_kv][head_dim] elements of `dtype`.
 * page_size: a multiple of 16 in [16, 1024]; n_pages: 1 .. 2^24, with
 * n_pages * page_size < 2^31.
 *
 * SPARK_FP4 pages hold a row of one KV head in 144 bytes: 4-bit codes (a sign
 * and 0, 0.5, 1, 1.5, 2, 3, 4 or 6) and a scale for each 16 dims, which is a
 * number of 5 exponent and 3 mantissa bits (bits 14 .. 7 of an fp16, up to
 * 10240); an element is code * scale, a number of at most 6 significant
 * bits.  With m the largest magnitude of the 16, in fp32: scale = m / 6 and
 * code = x / scale, each division rounded to fp32, then to the nearest of the
 * format, ties to even; magnitudes above 61440 become that; 16 elements with
 * an infinity or a NaN among them become NaN.
 * K and V are [n_pages][page_size / 16][n_kv] blocks of 2304 bytes, one for 16
 * positions: 16 rows of 128 bytes of codes, then 16 rows of 16 scales.  A byte
 * of codes holds dim 2 i in its low half and 2 i + 1 in its high half; the
 * 16-byte chunk c of row r lies at chunk c ^ (r % 2 + 2 (r / 4 % 4)). */
#define SPARK_FP4_BLOCK_BYTES 2304
typedef struct spark_page_pool {
  void* k;
  void* v;
  int64_t n_pages;
  int32_t page_size;
  int32_t dtype; /* spark_dtype */
} spark_page_pool;

/* The sequences of a call.  Sequence s brings the q_start[s + 1] - q_start[s]
 * new tokens (none is allowed) in rows q_start[s] .. q_start[s + 1] - 1 of
 * the call's q, k, v and output; they are the last of its seq_len[s]
 * positions.  Rows at or behind q_start[n_seqs] are not written, and what is in
 * them reaches no result.
 *   table    device [n_seqs][max_pages] int32.  Entries of pages that hold
 *            no position the call reads or writes may be anything.
 *   q_start  device [n_seqs + 1] int32, not decreasing, from >= 0.
 *   seq_len  device [n_seqs] int32.
 * n_seqs: 1 .. SPARK_MAX_BATCH; max_pages: 1 .. SPARK_MAX_TABLE_PAGES;
 * n_tokens: rows of the call's token buffers, 1 .. SPARK_MAX_PAGED_TOKENS;
 * max_q_len: no sequence brings more new tokens (1 .. n_tokens). */
typedef struct spark_paged_batch {
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* seq_len;
  int32_t n_seqs;
  int32_t max_pages;
  int32_t n_tokens;
  int32_t max_q_len;
} spark_paged_batch;

/* Bytes of the device workspace of spark_paged_append and
 * spark_paged_attention (0 for an invalid geometry): the error word, merge
 * tickets and split-K partial results.  It does not depend on the batch.
 * Initialise it once with spark_attn_workspace_init. */
size_t spark_paged_workspace_bytes(const spark_geom* g);

/* Write the k and v rows of the batch's new tokens into their pages, rounded
 * once to the pool's type (SPARK_FP4: see there).
 *   k, v     device [n_tokens][n_kv * head_dim] of element type `dtype`;
 *            row t starts at element t * ld (slices of a fused projection's
 *            rows do; ld >= n_kv * head_dim, rows 16-byte aligned).
 *   workspace >= spark_paged_workspace_bytes, 256-byte aligned.
 * Two new tokens of one call in the same page row (tables that share a page
 * that both write) leave either's values there (SPARK_FP4: codes of one may
 * meet the scale of the other).
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE before any work is enqueued;
 * CUDA if a launch fails. */
int spark_paged_append(const spark_geom* g, const void* k, const void* v, int64_t ld, int32_t dtype,
                       const spark_page_pool* pool, const spark_paged_batch* batch, void* workspace,
                       size_t workspace_bytes, void* stream);

/* The (cos, sin) of a layer class's rope angles position * theta^(-2 i / r) in
 * fp32, computed in 64 bits, for positions 0 .. n_positions - 1: rope, device
 * [n_positions][r / 2][2], with r the class's rotary dim (full_rotary_dim, or
 * head_dim in sliding layers).  All layers of a class share one.
 * n_positions: 1 .. 2^24.
 * Errors: INVALID_ARG, UNSUPPORTED; CUDA if a launch fails. */
int spark_rope_table(const spark_geom* g, int32_t layer_class, int32_t n_positions, float* rope, void* stream);

/* spark_paged_append of new tokens whose queries and keys are not rotated
 * yet: NeoX rope on the way (the class's rotary dim r, pairs i and i + r / 2,
 * the dims behind r as they are), in fp32 within 1.5 ulp, rounded once to its
 * type; the codes of 4-bit pages are those of the exact rotation rounded to fp32.
 *   q       rows [n_q * head_dim] of element type `dtype`, row t at element
 *           t * ld; null: no queries.
 *   k, v    rows [n_kv * head_dim], likewise at t * ld (three slices of a
 *           fused projection's rows).
 *   q_out   rows [n_q * head_dim] of the same type, row t at element
 *           t * q_out_ld: the rotated queries of the tokens that belong to a
 *           sequence, other rows are left as they were.  It is q itself with
 *           q_out_ld == ld (in place), or overlaps no row of q, k or v (with
 *           another q_out_ld, nothing from their first row to their last).
 *   rope    the class's table (spark_rope_table), n_positions long.
 * A token's position is that of its cache row (seq_len, a device value: a
 * captured call replays for the next token).  One at or behind n_positions
 * raises bit 2 and is left out.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE before any work is enqueued;
 * CUDA if a launch fails. */
int spark_paged_rope_append(const spark_geom* g, const void* q, const void* k, const void* v, int64_t ld, int32_t dtype,
                            int32_t layer_class, const float* rope, int32_t n_positions, const spark_page_pool* pool,
                            const spark_paged_batch* batch, void* q_out, int64_t q_out_ld, void* workspace,
                            size_t workspace_bytes, void* stream);

/* The batch's rows out of their pages: k and v (device, element type `dtype`,
 * row t at element t * ld) receive the row of every token that a sequence of
 * the batch counts as new, whoever wrote it (q_start and seq_len choose the
 * positions: a whole prefix with as many "new" tokens as it is long).  Rows
 * behind q_start[n_seqs] are left as they were.  An element that `dtype` does
 * not hold is rounded once (fp32 pages read as bf16).
 * workspace and errors as spark_paged_append. */
int spark_paged_read(const spark_geom* g, const spark_page_pool* pool, const spark_paged_batch* batch, void* k, void* v,
                     int64_t ld, int32_t dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Attention of every new token of the batch over its sequence's pages (its
 * own row included: spark_paged_append comes first).
 *   q     device rows [n_q * head_dim] of element type `dtype` (F32 or
 *         BF16), row t at element t * q_ld (q_ld >= n_q * head_dim, rows
 *         16-byte aligned): rotated queries.
 *   a     device [n_tokens][n_q * head_dim] of the same type: un-gated
 *         attention output, a row written for every new token of a sequence,
 *         the others left as they were.  Does not overlap q.
 * fp32 queries meet a bf16 pool as q = hi + lo in bf16 (16 significant
 * bits), the probabilities too.  bf16 queries meet it as they are, with
 * probabilities of 16 significant bits where max_q_len is 1 and rounded to
 * bf16 (8 bits) where it is more.  An fp32 pool is read by fp32 arithmetic.
 * 4-bit pages are met in fp16, queries scaled by a power of two for each token
 * and head: fp32 ones as q = hi + lo (22 bits of the token's and head's
 * largest element), bf16 ones as they are (elements below 2^-17 of the
 * largest lose bits); probabilities as hi + lo (22 bits), but rounded to fp16
 * (11 bits) for bf16 queries where max_q_len is more than 1, and in steps of
 * 2^-35 of the row's largest at the least.  With max_q_len above 1 scores are
 * expected below 2^27.  Outputs are summed in
 * fp32; what the matrix instructions cut off a sum stays below 2^-14 of the sum
 * of its magnitudes for fp32 queries and 2^-11 for bf16 ones, however long the
 * sequence and whatever the order of large and small terms.
 * Rows that no token of the sequence attends to may hold anything, NaN
 * included; a row that one of its new tokens attends to is expected finite
 * (a non-finite V row may reach every new token of its sequence).
 * max_q_len, with n_tokens and n_seqs, chooses the kernel, and with it the
 * order of the sums and the rounding of the probabilities, not the results
 * beyond these: give the true bound.
 * workspace and errors as spark_paged_append. */
int spark_paged_attention(const spark_geom* g, const void* q, int64_t q_ld, int32_t dtype,
                          const spark_page_pool* pool, int32_t layer_class, const spark_paged_batch* batch,
                          void* a, void* workspace, size_t workspace_bytes, void* stream);

/* The attention block (spark_attn_decode's, spark_attn_prefill's) for the
 * batch's new tokens on a paged cache: input RMSNorm and projections, the
 * append, the attention, gate, o_proj and residual.
 *   h          [n_tokens][hidden] fp32 device; out the same, may equal h.
 *   positions  [n_tokens] HOST int32: the rope position of each row (they
 *              are the call's only host array; the rows of the cache follow
 *              seq_len alone).  They are read during the call, as
 *              spark_attn_decode's are: a captured call replays with the
 *              positions of its capture whatever seq_len says by then, so a
 *              graph of it serves a step again, not the next token.
 *              Rows behind q_start[n_seqs] take any position >= 0, and their
 *              out rows are unspecified.
 *   n_tokens   1 .. SPARK_MAX_BATCH here.
 *   workspace  >= spark_attn_workspace_bytes(g, n_tokens), as for
 *              spark_attn_decode; paged_workspace as for
 *              spark_paged_attention (two buffers).
 * Errors: INVALID_ARG, POSITION, UNSUPPORTED, WORKSPACE before any work is
 * enqueued; CUDA if a launch fails. */
int spark_attn_paged(const spark_geom* g, const float* h, const spark_layer_weights* w,
                     const spark_page_pool* pool, int32_t layer_class, const spark_paged_batch* batch,
                     const int32_t* positions, float* out, void* workspace, size_t workspace_bytes,
                     void* paged_workspace, size_t paged_workspace_bytes, void* stream);

/* Bytes of the device workspace of spark_pages_remap and spark_pages_compact
 * for pools of n_pages pages and tables of n_slots rows (0 for invalid
 * arguments).  Initialise it once with spark_attn_workspace_init. */
size_t spark_pages_workspace_bytes(int64_t n_pages, int32_t n_slots);

/* The page tables of a step.  A sequence slot s of the new table holds the
 * first keep_len[s] positions of the old table's row parent[s] and has room
 * for new_len[s] positions:
 *   parent s, keep = its length          a sequence goes on (new_len more: grows)
 *   keep below its length                it is cut (rejected drafts)
 *   another slot as parent               it is a fork (a beam, a shared prefix)
 *   parent -1, keep 0                    the old sequence ends; new_len > 0: another begins
 * Pages wholly below keep_len are shared by all who keep them.  A page kept
 * in part will be written to, so it becomes the slot's own: if nobody keeps
 * it whole it stays with the lowest slot that keeps it in part, every other
 * one gets a page of its own into which the rows below keep_len are copied,
 * in every pool.  New pages are the ones nobody keeps, the lowest first, in
 * slot order (a slot's copied page before the pages it grows by); a page
 * nobody keeps is free: there are no reference counts, the tables say who
 * holds what (a prefix kept for later is a slot of its own).
 *   pools       n_pools layers (host array), alike in n_pages, page_size, dtype.
 *   table       device [n_slots][max_pages]; new_table the same size, not
 *               overlapping it: pages, then -1.
 *   parent, keep_len, new_len   device [n_slots] int32.
 *   workspace   >= spark_pages_workspace_bytes(n_pages, n_slots).
 * All or nothing: where an argument on the device is out of range (bit 2: a
 * parent outside [-1, n_slots), keep > new, keep without a parent, new_len
 * beyond max_pages, a kept entry outside the pool) or the pool has too few
 * free pages (bit 4), the error word gets the bit and table, new_table and
 * pools stay as they were.
 * n_slots: 1 .. SPARK_MAX_BATCH; n_slots * max_pages <= 2^26.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE before any work is enqueued;
 * CUDA if a launch fails. */
int spark_pages_remap(const spark_geom* g, const spark_page_pool* pools, int32_t n_pools, const int32_t* table,
                      int32_t n_slots, int32_t max_pages, const int32_t* parent, const int32_t* keep_len,
                      const int32_t* new_len, int32_t* new_table, void* workspace, size_t workspace_bytes,
                      void* stream);

/* Move the pages in use to the front of the pools: with n_live pages named
 * by the table (entries >= 0; -1 names none), the i-th used page at or
 * behind n_live goes to the i-th unused page before it, both in ascending
 * order, in every pool, and the new table names the new places.
 *   new_table  device [n_slots][max_pages], may equal table.
 *   n_live     device int32: receives the number of used pages; the pages
 *              behind it may be given back.
 * All or nothing, as spark_pages_remap: an entry below -1 or outside the
 * pool raises bit 2, and only n_live (set to -1) is written. */
int spark_pages_compact(const spark_geom* g, const spark_page_pool* pools, int32_t n_pools, const int32_t* table,
                        int32_t n_slots, int32_t max_pages, int32_t* new_table, int32_t* n_live, void* workspace,
                        size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SPARK_PAGED_H */
