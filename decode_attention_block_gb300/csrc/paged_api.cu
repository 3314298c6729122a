// paged_api.cu -- the C ABI of the paged cache and of the token scores
// (declared in include/spark_paged.h and include/spark_score.h): argument
// checks, workspace layouts and launches.  spark_attn_paged, which runs the
// block's projections, is in api.cu.
#include "paged_checks.h"
#include "pages.h"
#include "score.h"

using namespace spark;
using namespace spark::checks;

extern "C" {

size_t spark_paged_workspace_bytes(const spark_geom* g) {
  return check_geom(g) == SPARK_OK ? paged_ws_layout().total : 0;
}

int spark_paged_append(const spark_geom* g, const void* k, const void* v, int64_t ld, int32_t dtype,
                       const spark_page_pool* pool, const spark_paged_batch* batch, void* workspace,
                       size_t workspace_bytes, void* stream) {
  int s;
  if ((s = check_geom(g)) != SPARK_OK) return s;
  if ((s = check_pool(pool)) != SPARK_OK) return s;
  if ((s = check_paged_batch(batch)) != SPARK_OK) return s;
  if ((s = check_rows(k, dtype, ld, (int64_t)g->n_kv * kHeadDim)) != SPARK_OK) return s;
  if ((s = check_rows(v, dtype, ld, (int64_t)g->n_kv * kHeadDim)) != SPARK_OK) return s;
  if ((s = check_paged_ws(workspace, workspace_bytes)) != SPARK_OK) return s;
  const paged::Args p = paged_args(g, pool, SPARK_FULL, batch, workspace);
  return cuda_status(launch_paged_append(p, dtype, pool->dtype, k, v, ld, pool->k, pool->v, (cudaStream_t)stream));
}

int spark_paged_attention(const spark_geom* g, const void* q, int64_t q_ld, int32_t dtype,
                          const spark_page_pool* pool, int32_t layer_class, const spark_paged_batch* batch,
                          void* a, void* workspace, size_t workspace_bytes, void* stream) {
  int s;
  if ((s = check_geom(g)) != SPARK_OK) return s;
  if ((s = check_pool(pool)) != SPARK_OK) return s;
  if (layer_class != SPARK_FULL && layer_class != SPARK_SLIDING) return SPARK_ERR_INVALID_ARG;
  if ((s = check_paged_batch(batch)) != SPARK_OK) return s;
  if ((s = check_rows(q, dtype, q_ld, (int64_t)g->n_q * kHeadDim)) != SPARK_OK) return s;
  if (!a || !aligned16(a)) return SPARK_ERR_INVALID_ARG;
  // rows of q are read while rows of a are written
  const int64_t es = dtype == SPARK_BF16 ? 2 : 4, width = (int64_t)g->n_q * kHeadDim;
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), a0 = reinterpret_cast<uintptr_t>(a);
  const uintptr_t q1 = q0 + (uintptr_t)(((batch->n_tokens - 1) * q_ld + width) * es);
  const uintptr_t a1 = a0 + (uintptr_t)(batch->n_tokens * width * es);
  if (q0 < a1 && a0 < q1) return SPARK_ERR_INVALID_ARG;
  if ((s = check_paged_ws(workspace, workspace_bytes)) != SPARK_OK) return s;
  paged::Args p = paged_args(g, pool, layer_class, batch, workspace);
  p.q = q;
  p.q_ld = q_ld;
  p.a = a;
  return cuda_status(launch_paged_attention(p, dtype, pool->dtype, pool->k, pool->v, (cudaStream_t)stream));
}

size_t spark_pages_workspace_bytes(int64_t n_pages, int32_t n_slots) {
  if (n_pages < 1 || n_pages > kMaxPoolPages || check_batch(n_slots) != SPARK_OK) return 0;
  return pages::ws_layout(n_pages, n_slots).total;
}

namespace {

int pages_call(pages::Call* c, const spark_geom* g, const spark_page_pool* pools, int32_t n_pools, const int32_t* table,
               int32_t n_slots, int32_t max_pages, int32_t* new_table, void* workspace, size_t workspace_bytes) {
  int s;
  if ((s = check_geom(g)) != SPARK_OK) return s;
  if (!pools || n_pools < 1) return SPARK_ERR_INVALID_ARG;
  if (n_pools > SPARK_MAX_PAGE_POOLS) return SPARK_ERR_UNSUPPORTED;
  for (int i = 0; i < n_pools; ++i) {
    if ((s = check_pool(&pools[i])) != SPARK_OK) return s;
    if (pools[i].n_pages != pools[0].n_pages || pools[i].page_size != pools[0].page_size ||
        pools[i].dtype != pools[0].dtype)
      return SPARK_ERR_INVALID_ARG;
    c->pools.p[2 * i] = pools[i].k;
    c->pools.p[2 * i + 1] = pools[i].v;
  }
  if ((s = check_batch(n_slots)) != SPARK_OK) return s;
  if (max_pages < 1) return SPARK_ERR_INVALID_ARG;
  if (max_pages > SPARK_MAX_TABLE_PAGES || (int64_t)n_slots * max_pages > ((int64_t)1 << 26)) return SPARK_ERR_UNSUPPORTED;
  if (!table || !new_table || !aligned4(table) || !aligned4(new_table)) return SPARK_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      workspace_bytes < pages::ws_layout(pools[0].n_pages, n_slots).total)
    return SPARK_ERR_WORKSPACE;
  c->n_pools = n_pools;
  c->n_pages = pools[0].n_pages;
  c->page_size = pools[0].page_size;
  c->row_bytes = (int64_t)g->n_kv * kHeadDim * (pools[0].dtype == SPARK_BF16 ? 2 : 4);
  c->table = table;
  c->new_table = new_table;
  c->n_slots = n_slots;
  c->max_pages = max_pages;
  c->workspace = workspace;
  return SPARK_OK;
}

}  // namespace

int spark_pages_remap(const spark_geom* g, const spark_page_pool* pools, int32_t n_pools, const int32_t* table,
                      int32_t n_slots, int32_t max_pages, const int32_t* parent, const int32_t* keep_len,
                      const int32_t* new_len, int32_t* new_table, void* workspace, size_t workspace_bytes,
                      void* stream) {
  pages::Call c = {};
  const int s = pages_call(&c, g, pools, n_pools, table, n_slots, max_pages, new_table, workspace, workspace_bytes);
  if (s != SPARK_OK) return s;
  if (!parent || !keep_len || !new_len || !aligned4(parent) || !aligned4(keep_len) || !aligned4(new_len))
    return SPARK_ERR_INVALID_ARG;
  const int64_t n = (int64_t)n_slots * max_pages;  // the old table is read while the new one is written
  if (table < new_table + n && new_table < table + n) return SPARK_ERR_INVALID_ARG;
  c.parent = parent;
  c.keep = keep_len;
  c.grow = new_len;
  return cuda_status(launch_pages(c, (cudaStream_t)stream));
}

int spark_pages_compact(const spark_geom* g, const spark_page_pool* pools, int32_t n_pools, const int32_t* table,
                        int32_t n_slots, int32_t max_pages, int32_t* new_table, int32_t* n_live, void* workspace,
                        size_t workspace_bytes, void* stream) {
  pages::Call c = {};
  const int s = pages_call(&c, g, pools, n_pools, table, n_slots, max_pages, new_table, workspace, workspace_bytes);
  if (s != SPARK_OK) return s;
  if (!n_live || !aligned4(n_live)) return SPARK_ERR_INVALID_ARG;
  const int64_t n = (int64_t)n_slots * max_pages;  // in place, entry by entry, or apart
  if (table != new_table && table < new_table + n && new_table < table + n) return SPARK_ERR_INVALID_ARG;
  c.n_live = n_live;
  return cuda_status(launch_pages(c, (cudaStream_t)stream));
}

size_t spark_logprobs_workspace_bytes(int32_t n_rows, int32_t top_k) {
  if (n_rows < 1 || n_rows > kMaxScoreRows || top_k < 0 || top_k > SPARK_MAX_TOP) return 0;
  return score::kTotal;
}

int spark_token_logprobs(const void* logits, int64_t ld, int32_t dtype, int32_t n_rows, int32_t vocab,
                         const int32_t* targets, int32_t top_k, float* logprob, float* entropy, int32_t* top_ids,
                         float* top_logprobs, void* workspace, size_t workspace_bytes, void* stream) {
  if (check_dtype(dtype) != SPARK_OK || !logits || n_rows < 1 || n_rows > kMaxScoreRows || vocab < 1 ||
      vocab > (1 << 24) || top_k < 0 || top_k > SPARK_MAX_TOP || top_k > vocab || ld < vocab ||
      ld > ((int64_t)1 << 40))
    return SPARK_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(logits) & (dtype == SPARK_BF16 ? 1u : 3u)) != 0) return SPARK_ERR_INVALID_ARG;
  if (!targets || !logprob || !entropy || !aligned4(targets) || !aligned4(logprob) || !aligned4(entropy))
    return SPARK_ERR_INVALID_ARG;
  if (top_k > 0 && (!top_ids || !top_logprobs || !aligned4(top_ids) || !aligned4(top_logprobs)))
    return SPARK_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < score::kTotal)
    return SPARK_ERR_WORKSPACE;
  return cuda_status(launch_score(logits, ld, dtype, n_rows, vocab, targets, top_k, logprob, entropy, top_ids,
                                  top_logprobs, workspace, (cudaStream_t)stream));
}

}  // extern "C"
