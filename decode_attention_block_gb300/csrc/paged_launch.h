// paged_launch.h -- host launchers of the paged cache's attention and append
// kernels (internal to the library).
#pragma once

#include "paged_parts.cuh"

namespace spark {

// Attention of every new token over its pages.
cudaError_t launch_paged_attention(const paged::Args& p, int qdtype, int cdtype, const void* k, const void* v,
                                   cudaStream_t st);

// The same for chunks on a bf16 pool, on the tensor cores, 32 tokens at a time.
cudaError_t launch_paged_chunk(const paged::Args& p, int qdtype, const void* k, const void* v, cudaStream_t st);

// The same on pairs of CTAs, 64 tokens at a time.
cudaError_t launch_paged_pair(const paged::Args& p, int qdtype, const void* k, const void* v, cudaStream_t st);

// The new tokens' k and v rows into their pages.
cudaError_t launch_paged_append(const paged::Args& p, int xdtype, int cdtype, const void* k, const void* v, int64_t ld,
                                void* pk, void* pv, cudaStream_t st);

}  // namespace spark
