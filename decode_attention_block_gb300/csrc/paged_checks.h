// paged_checks.h -- host-side argument checks of the paged cache's entry
// points, and the kernel arguments they become (every status is decided
// before anything is enqueued).
#pragma once

#include "../../include/spark_paged.h"
#include "../../include/spark_score.h"
#include "checks.h"
#include "paged_launch.h"

namespace spark {

// Workspace of spark_paged_append and spark_paged_attention: error word,
// merge tickets, the chunk kernel's joins, partial states.
struct PagedWsLayout {
  size_t tickets, joins, part, total;
};
inline PagedWsLayout paged_ws_layout() {
  PagedWsLayout L;
  L.tickets = 256;  // the error word sits at 0
  L.joins = align_up(L.tickets + sizeof(uint32_t) * paged::kMaxCtas, 256);
  L.part = align_up(L.joins + sizeof(paged::Join) * paged::kMaxChunkCtas, 256);
  L.total = align_up(L.part + paged::kPartBytes, 256);
  return L;
}

namespace checks {

constexpr int64_t kMaxPoolPages = 1 << 24;
constexpr int32_t kMaxScoreRows = 1 << 20;

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline int check_pool(const spark_page_pool* pool) {
  if (!pool || !pool->k || !pool->v || !aligned16(pool->k) || !aligned16(pool->v)) return SPARK_ERR_INVALID_ARG;
  if (check_dtype(pool->dtype) != SPARK_OK) return SPARK_ERR_INVALID_ARG;
  if (pool->n_pages < 1 || pool->page_size < 1) return SPARK_ERR_INVALID_ARG;
  if (pool->page_size % 16 != 0 || pool->page_size > 1024) return SPARK_ERR_UNSUPPORTED;
  // TMA coordinates of rows are 32-bit
  if (pool->n_pages > kMaxPoolPages || pool->n_pages * pool->page_size >= ((int64_t)1 << 31)) return SPARK_ERR_UNSUPPORTED;
  return SPARK_OK;
}

inline int check_paged_batch(const spark_paged_batch* b) {
  if (!b || !b->table || !b->q_start || !b->seq_len || !aligned4(b->table) || !aligned4(b->q_start) ||
      !aligned4(b->seq_len))
    return SPARK_ERR_INVALID_ARG;
  if (check_batch(b->n_seqs) != SPARK_OK || b->max_pages < 1 || b->n_tokens < 1 || b->max_q_len < 1 ||
      b->max_q_len > b->n_tokens)
    return SPARK_ERR_INVALID_ARG;
  if (b->max_pages > SPARK_MAX_TABLE_PAGES || b->n_tokens > SPARK_MAX_PAGED_TOKENS) return SPARK_ERR_UNSUPPORTED;
  return SPARK_OK;
}

// rows of `width` elements, `ld` apart, read 16 bytes at a time
inline int check_rows(const void* p, int32_t dtype, int64_t ld, int64_t width) {
  if (!p || !aligned16(p) || check_dtype(dtype) != SPARK_OK) return SPARK_ERR_INVALID_ARG;
  if (ld < width || ld > ((int64_t)1 << 32) || ld % (dtype == SPARK_BF16 ? 8 : 4) != 0) return SPARK_ERR_INVALID_ARG;
  return SPARK_OK;
}

inline int check_paged_ws(void* ws, size_t bytes) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return SPARK_ERR_WORKSPACE;
  return bytes < paged_ws_layout().total ? SPARK_ERR_WORKSPACE : SPARK_OK;
}

inline paged::Args paged_args(const spark_geom* g, const spark_page_pool* pool, int32_t layer_class,
                              const spark_paged_batch* b, void* ws) {
  const PagedWsLayout L = paged_ws_layout();
  paged::Args p = {};
  p.table = b->table;
  p.q_start = b->q_start;
  p.seq_len = b->seq_len;
  p.n_seqs = b->n_seqs;
  p.max_pages = b->max_pages;
  p.n_tokens = b->n_tokens;
  p.max_q = b->max_q_len;
  p.n_pages = (int32_t)pool->n_pages;
  p.page_size = pool->page_size;
  p.page_mul = paged::page_mul(pool->page_size);
  p.n_kv = g->n_kv;
  p.window = layer_class == SPARK_FULL ? 0 : g->window;
  p.scale_log2 = g->scale * 1.4426950408889634f;
  p.err = ws_at<uint32_t>(ws, 0);
  p.tickets = ws_at<uint32_t>(ws, L.tickets);
  p.joins = ws_at<paged::Join>(ws, L.joins);
  p.part = ws_at<float>(ws, L.part);
  return p;
}

}  // namespace checks
}  // namespace spark
