// paged_parts.cuh -- device pieces shared by the kernels of the paged cache:
// the arguments of a call, the prefix sums of its work list, and a cursor
// over a CTA's share of it (index arithmetic: paged.h).
#pragma once

#include "common.cuh"
#include "paged.h"

namespace spark {
namespace paged {

// CTAs of an attention launch at most (two partial slots each)
constexpr int kMaxCtas = 320;
// the chunk kernel: tokens of a group, CTAs at most, floats of a partial
// state (128 rows of 256 dims, their maxima, their sums)
constexpr int kChunkTokens = 32;
constexpr int kMaxChunkCtas = 160;
constexpr int kChunkPart = kGroup * kChunkTokens * (kHeadDim + 2);
// bytes of the partial states of either kernel
constexpr size_t kTokenPartBytes = sizeof(float) * 2 * kMaxCtas * kPartFloats;
constexpr size_t kChunkPartBytes = sizeof(float) * 2 * kMaxChunkCtas * kChunkPart;
constexpr size_t kPartBytes = kTokenPartBytes > kChunkPartBytes ? kTokenPartBytes : kChunkPartBytes;

// A group of the chunk kernel that begins in a CTA's share and goes on behind
// it: what the join needs.  n_rows 0: there is none.
struct Join {
  int32_t row0, n_rows;  // first token's row, rows (4 per token)
  int32_t head, last;    // KV head, last CTA
  int64_t begin, total;  // the group's first unit, units of the call
  int32_t G, unused;     // CTAs that share them
};

struct Args {
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* seq_len;
  int32_t n_seqs, max_pages, n_tokens, max_q;
  int32_t from, to;  // a launch takes the sequences of from .. to new tokens
  int32_t n_pages, page_size;
  uint64_t page_mul;  // of page_size (paged.h)
  int32_t n_kv, window;  // window 0: the whole history
  const void* q;
  int64_t q_ld;
  void* a;
  float scale_log2;
  uint32_t* err;
  uint32_t* tickets;  // [kMaxCtas], zero between launches
  Join* joins;        // [kMaxChunkCtas]
  float* part;        // partial states, two slots per CTA
};

#if defined(__CUDACC__)

__device__ __forceinline__ Seq load_seq(const Args& p, int s) {
  Seq q = seq_of(__ldcg(p.q_start + s), __ldcg(p.q_start + s + 1), __ldcg(p.seq_len + s), p.n_tokens, p.max_q,
                 (int64_t)p.max_pages * p.page_size);
  if (q.n < p.from || q.n > p.to) q.n = 0;
  return q;
}

// prefix[s] = units of the sequences before s (all KV heads), s <= n_seqs, in
// shared memory; every thread of the block calls this and `sums` has room for
// one value per warp.  CTA 0 reports sequences that make no sense.
template <int NT>
__device__ __forceinline__ void work_prefix(const Args& p, const Shape& sh, int64_t* prefix, int64_t* sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kPer = (SPARK_MAX_BATCH + NT - 1) / NT;
  const int per = (p.n_seqs + NT - 1) / NT;
  int64_t u[kPer], mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = tid * per + i;
    u[i] = 0;
    if (i < per && s < p.n_seqs) {
      const Seq q = load_seq(p, s);
      if (q.bad && blockIdx.x == 0) atomicOr(p.err, kErrIndex);
      if (q.n > 0) u[i] = (int64_t)p.n_kv * units_of(q, sh);
    }
    mine += u[i];
  }
  int64_t run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += up;
  }
  if (lane == 31) sums[warp] = run;
  __syncthreads();
  int64_t before = run - mine;
  for (int w = 0; w < warp; ++w) before += sums[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = tid * per + i;
    if (i < per && s < p.n_seqs) prefix[s] = before;
    before += u[i];
    if (i < per && s == p.n_seqs - 1) prefix[p.n_seqs] = before;
  }
  __syncthreads();
}

// A walk over the groups a share of the work list meets.
struct Cursor {
  int s, j, i;      // sequence, KV head, group
  int groups;       // groups of the sequence
  Seq seq;
  Group g;
  int64_t begin, end;  // the group's units in the list

  __device__ __forceinline__ void set_group(const Shape& sh, int64_t at) {
    g = group_of(seq, sh, i);
    begin = at;
    end = at + (g.tile1 - g.tile0);
  }
  // the group that holds unit u (u < total)
  __device__ __forceinline__ void seek(const Args& p, const Shape& sh, const int64_t* prefix, int64_t u) {
    int lo = 0, hi = p.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= u) lo = mid; else hi = mid - 1;
    }
    s = lo;
    seq = load_seq(p, s);
    groups = groups_of(seq, sh);
    const int64_t per_head = (prefix[s + 1] - prefix[s]) / p.n_kv;
    j = (int)((u - prefix[s]) / per_head);
    const int64_t at = prefix[s] + j * per_head;
    i = group_at(seq, sh, u - at);
    set_group(sh, at + units_before(seq, sh, i));
  }
  // the next group (there is one: end < total)
  __device__ __forceinline__ void next(const Args& p, const Shape& sh) {
    if (++i >= groups) {
      i = 0;
      if (++j >= p.n_kv) {
        j = 0;
        do {
          ++s;
          seq = load_seq(p, s);
        } while (seq.n == 0 && s + 1 < p.n_seqs);
        groups = groups_of(seq, sh);
      }
    }
    set_group(sh, end);
  }
};

__device__ __forceinline__ int page_col(const Args& p, int pos) { return page_col(pos, p.page_mul); }
__device__ __forceinline__ int page_row(const Args& p, int pos) {
  return page_row(pos, page_col(p, pos), p.page_size);
}

// The table's entry for column `col` of sequence s ...
__device__ __forceinline__ int page_entry(const Args& p, int s, int col) {
  return __ldcg(p.table + (int64_t)s * p.max_pages + col);
}
// ... as a page: an entry outside the pool is reported and read as page 0.
__device__ __forceinline__ int page_of(const Args& p, int entry) {
  if (entry >= 0 && entry < p.n_pages) return entry;
  atomicOr(p.err, kErrIndex);
  return 0;
}

#endif  // __CUDACC__

}  // namespace paged
}  // namespace spark
