// paged_launch.h -- host launchers of the paged cache's attention and append
// kernels (internal to the library).
#pragma once

#include "paged_parts.cuh"

namespace spark {
namespace paged {

// Rows of tokens on their way into pages: queries and keys rotated by the
// first `half` pairs of a table's row (0: not at all; q null: no queries).
struct RopeRows {
  const void *q, *k, *v;
  int64_t ld;
  const float* rope;
  int half, n_positions;
  void* q_out;
  int64_t q_out_ld;
  void *pk, *pv;
};

}  // namespace paged

// Attention of every new token over its pages.
cudaError_t launch_paged_attention(const paged::Args& p, int qdtype, int cdtype, const void* k, const void* v,
                                   cudaStream_t st);

// The same for chunks on a bf16 pool, on the tensor cores, 32 tokens at a time.
cudaError_t launch_paged_chunk(const paged::Args& p, int qdtype, const void* k, const void* v, cudaStream_t st);

// The same on pairs of CTAs, 64 tokens at a time.
cudaError_t launch_paged_pair(const paged::Args& p, int qdtype, const void* k, const void* v, cudaStream_t st);

// Attention over 4-bit pages.
cudaError_t launch_paged4_attention(const paged::Args& p, int qdtype, const void* k, const void* v, cudaStream_t st);

// The same for chunks, on the tensor cores, 32 tokens at a time.
cudaError_t launch_paged4_chunk(const paged::Args& p, int qdtype, const void* k, const void* v, cudaStream_t st);

// The same on pairs of CTAs, 64 tokens at a time.
cudaError_t launch_paged4_pair(const paged::Args& p, int qdtype, const void* k, const void* v, cudaStream_t st);

// The new tokens' rows into their pages, rotated on the way; any pool.
cudaError_t launch_paged_rope(const paged::Args& p, int xdtype, int cdtype, const paged::RopeRows& a, cudaStream_t st);

// The tokens' rows out of their pages; any pool.
cudaError_t launch_paged_read(const paged::Args& p, int xdtype, int cdtype, const void* pk, const void* pv, void* k,
                              void* v, int64_t ld, cudaStream_t st);

// (cos, sin) of the rope angles of positions 0 .. n_positions - 1.
cudaError_t launch_rope_table(float* rope, int n_positions, int rotary_dim, double theta, cudaStream_t st);

// The new tokens' k and v rows into their pages.
cudaError_t launch_paged_append(const paged::Args& p, int xdtype, int cdtype, const void* k, const void* v, int64_t ld,
                                void* pk, void* pv, cudaStream_t st);

}  // namespace spark
