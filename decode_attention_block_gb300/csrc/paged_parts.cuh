// paged_parts.cuh -- device pieces shared by the kernels of the paged cache:
// the arguments of a call, the prefix sums of its work list, and a cursor
// over a CTA's share of it (index arithmetic: paged.h).
#pragma once

#include "common.cuh"
#include "paged.h"

namespace spark {
namespace paged {

// CTAs of an attention launch at most (two partial slots each)
constexpr int kMaxCtas = 480;
// the chunk kernel: tokens of a group, CTAs at most, floats of a partial
// state (128 rows of 256 dims, their maxima, their sums)
constexpr int kChunkTokens = 32;
constexpr int kMaxChunkCtas = 160;
constexpr int kChunkPart = kGroup * kChunkTokens * (kHeadDim + 2);
// bytes of the partial states of either kernel; behind the token kernel's what a
// warp over 4-bit pages sums up beside its registers (4 warps a CTA, 8 rows, two
// values a lane)
constexpr size_t kTokenPartBytes = sizeof(float) * 2 * kMaxCtas * kPartFloats;
constexpr int kWarpSums = 8 * kHeadDim + 64;
constexpr size_t kChunkPartBytes = sizeof(float) * 2 * kMaxChunkCtas * kChunkPart;
constexpr size_t kPartBytes = kTokenPartBytes > kChunkPartBytes ? kTokenPartBytes : kChunkPartBytes;
static_assert(kTokenPartBytes % 16 == 0 && kTokenPartBytes + sizeof(float) * 4 * kMaxCtas * kWarpSums <= kPartBytes, "room for both");

// A group of the chunk kernel that begins in a CTA's share and goes on behind
// it: what the join needs.  n_rows 0: there is none.
struct alignas(16) Join {
  int32_t row0, n_rows;  // first token's row, rows (4 per token)
  int32_t head, last;    // KV head, last CTA
  int64_t begin, total;  // the group's first unit, units of the call
  int32_t G, unused[3];  // CTAs that share them
};

struct Args {
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* seq_len;
  int32_t n_seqs, max_pages, n_tokens, max_q;
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
  return seq_of(__ldcg(p.q_start + s), __ldcg(p.q_start + s + 1), __ldcg(p.seq_len + s), p.n_tokens, p.max_q,
                (int64_t)p.max_pages * p.page_size);
}

// prefix[s] = units of the sequences before s (all KV heads), s <= n_seqs, in
// shared memory; every thread of the block calls this and `sums` has room for
// two values per warp.  Returns the number of groups.  CTA 0 reports sequences
// that make no sense.
template <int NT>
__device__ __forceinline__ int64_t work_prefix(const Args& p, const Shape& sh, int64_t* prefix, int64_t* sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kPer = (SPARK_MAX_BATCH + NT - 1) / NT;
  const int per = (p.n_seqs + NT - 1) / NT;
  int64_t u[kPer], mine = 0;
  int groups = 0;  // (a call's tokens are at most 2^17)
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = tid * per + i;
    u[i] = 0;
    if (i < per && s < p.n_seqs) {
      const Seq q = load_seq(p, s);
      if (q.bad && blockIdx.x == 0) atomicOr(p.err, kErrIndex);
      if (q.n > 0) u[i] = (int64_t)p.n_kv * units_of(q, sh);
      groups += groups_of(q, sh);
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
  groups = __reduce_add_sync(0xffffffffu, groups);
  if (lane == 0) sums[NT / 32 + warp] = groups;
  __syncthreads();
  int64_t all = 0;
  for (int w = 0; w < NT / 32; ++w) all += sums[NT / 32 + w];
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
  return all * p.n_kv;
}

// A walk over the groups a share of the work list meets.
struct Cursor {
  int s, j, i;      // sequence, KV head, group
  int groups;       // groups of the sequence
  Seq seq;
  Group g;
  int64_t begin, end;  // the units of the group's tiles in the list

  __device__ __forceinline__ void set_group(const Shape& sh, int64_t at) {
    g = group_of(seq, sh, i);
    begin = at + sh.lead;
    end = begin + (g.tile1 - g.tile0);
  }
  // the group that holds unit u, in sequence `s`, `seq`, whose units begin at
  // `first`, per_head for each KV head
  __device__ __forceinline__ void seek(const Shape& sh, int64_t u, int64_t first, int64_t per_head) {
    groups = groups_of(seq, sh);
    j = (int)quotient(u - first, per_head);
    const int64_t at = first + j * per_head;
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
  // the next group, if it has a tile before unit u1
  __device__ __forceinline__ bool advance(const Args& p, const Shape& sh, int64_t u1) {
    if (end >= u1) return false;
    next(p, sh);
    return begin < u1;
  }
};

// What a group of U units is split into at most is sqrt(kSpread U) parts.  One
// token at 12000 with one KV head: 33 us with as many parts as there are CTAs,
// 19.1 at 2.5, 19.8 at 5, 21.6 at 10; at 700 9.2 at 5, 10.0 at 2.5.  And a
// whole number of parts a group, where they fit the grid (ctas_for): one token
// at 100 with 4 KV heads took 12.9 us on 7 CTAs that met two groups each, 7.6
// on one a group.
constexpr float kSpread = 4.f;

// A CTA's share of the list: the units [u0, u1) of `total`, shared by G CTAs,
// and the group it begins with.  Without a tile (c >= G, or a share that is
// all lead): no more is set.
struct Share {
  int64_t total, u0, u1;
  int G;
  Cursor cur;
  __device__ __forceinline__ bool cut(int c, int64_t groups, int least, int most) {
    G = total > 0 ? ctas_for(total, groups, least, kSpread, most) : 0;
    if (c >= G) return false;
    u0 = share_begin(total, G, c);
    u1 = share_begin(total, G, c + 1);
    return true;
  }
};

// Every thread of the block calls this, with room for SPARK_MAX_BATCH + 2 +
// NT / 16 values in shared memory; the block is in step afterwards.  Up to 32
// sequences (the common decode and prefill calls) each warp keeps one per
// lane and finds its share without another thread: 900 cycles against 4000
// by way of the prefix sums in shared memory.
template <int NT>
__device__ __forceinline__ bool find_share(const Args& p, const Shape& sh, int c, int least, int most, int64_t* room,
                                           Share& share) {
  const int lane = threadIdx.x & 31;
  Cursor& cur = share.cur;
  if (p.n_seqs <= 32) {
    Seq q = {0, 0, 0, false};
    if (lane < p.n_seqs) q = load_seq(p, lane);
    if (q.bad && blockIdx.x == 0 && threadIdx.x < 32) atomicOr(p.err, kErrIndex);
    // (a single token's units are its one group's; groups of one are of calls
    // with max_q 1, but not asked for that the compiler spills registers here)
    const Group only = group_of(q, sh, 0);
    const int64_t per_head = q.n == 0 ? 0 : sh.gt == 1 && p.max_q == 1 ? only.tile1 - only.tile0 : units_of(q, sh);
    int64_t run = per_head * p.n_kv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += up;
    }
    const int64_t first = run - per_head * p.n_kv;
    share.total = __shfl_sync(0xffffffffu, run, 31);
    const int groups = sh.gt == 1 && p.max_q == 1 ? __popc(__ballot_sync(0xffffffffu, q.n != 0))
                                                  : __reduce_add_sync(0xffffffffu, groups_of(q, sh));
    const bool any = share.cut(c, (int64_t)groups * p.n_kv, least, most);
    __syncthreads();
    if (!any) return false;
    // the last sequence that begins at or before u0 (one without units shares its beginning with the next)
    cur.s = 31 - __clz(__ballot_sync(0xffffffffu, first <= share.u0));
    cur.seq.q0 = __shfl_sync(0xffffffffu, q.q0, cur.s);
    cur.seq.n = __shfl_sync(0xffffffffu, q.n, cur.s);
    cur.seq.p0 = __shfl_sync(0xffffffffu, q.p0, cur.s);
    cur.seq.bad = false;
    const int64_t at = __shfl_sync(0xffffffffu, first, cur.s), each = __shfl_sync(0xffffffffu, per_head, cur.s);
    if (sh.gt == 1 && p.max_q == 1) {
      cur.groups = 1;
      cur.i = 0;
      cur.j = (int)quotient(share.u0 - at, each);
      cur.set_group(sh, at + cur.j * each);
    } else {
      cur.seek(sh, share.u0, at, each);
    }
    return cur.begin < share.u1;
  }
  const int64_t groups = work_prefix<NT>(p, sh, room, room + SPARK_MAX_BATCH + 2);
  share.total = room[p.n_seqs];
  if (!share.cut(c, groups, least, most)) return false;
  int lo = 0, hi = p.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (room[mid] <= share.u0) lo = mid; else hi = mid - 1;
  }
  cur.s = lo;
  cur.seq = load_seq(p, lo);
  cur.seek(sh, share.u0, room[lo], (room[lo + 1] - room[lo]) / p.n_kv);
  return cur.begin < share.u1;
}

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
