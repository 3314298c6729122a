// score.cu -- log probabilities of given tokens, entropy and the highest
// alternatives of rows of logits (spark_token_logprobs).
//
// One pass over the logits: each thread keeps a running maximum m, the sum
// z = sum e^(x - m) and u = sum (x - m) e^(x - m), which a higher maximum
// m + d turns into z e^-d and (u - d z) e^-d; then logprob = x_t - m - ln z
// and entropy = ln z - u / z.  Bound by the logits' bytes: 4 (or 2) per
// element against about eight operations.  Few rows are split over the
// vocabulary; the last CTA of a row to arrive joins the parts in order.
// Measured: 511 rows of 131072 fp32 logits, 5 alternatives, 49 us, 5.5 TB/s;
// one row, 20 alternatives, 10 us, the chain of a part and of the join.
//
// The alternatives ride along.  A logit and its index form one 64-bit key
// (value order first, then the lower index), so all keys differ and the
// outcome does not depend on any order of arrival.  Each warp holds its best k
// keys, lane i the i-th, and publishes a value that c = ceil(k / 8) of its
// logits reach: the least of the eight warps' values is a floor that k logits
// of the block reach, whenever it is read (the published values only rise).
// Only what reaches the floor is offered to the lists, and a tile in which no
// lane's maximum does costs one vote.  The lists meet in shared memory at the
// end.  (511 rows masked down to a few logits, or constant ones, cost 57 to 60 us
// with 20 alternatives, random ones 57; rows that ascend with the index offer
// every logit, one after another, and take 1.7 ms, 1.1 ms with 5.)
#include <math.h>

#include "launch.h"
#include "score.h"
#include "score_parts.cuh"

namespace spark {
namespace {

using namespace score;

// CTA (row, part)
template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
    k_score(const T* logits, int64_t ld, int vocab, const int32_t* targets, int k, int parts,
            float* logprob, float* entropy, int32_t* top_ids, float* top_logprobs, uint32_t* err, uint32_t* tickets,
            score::Part* part) {
  __shared__ Smem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / parts, c = blockIdx.x % parts;
  if (tid == 0) {
    sm.last = 0;
    sm.count = 0;
  }
  const int share = (k + kWarps - 1) / kWarps;  // of the k, a warp's
  WarpTop top;
  top.reset();
  pdl_wait();
  pdl_trigger();
  const T* x = logits + row * ld;
  Stat st = row_pass<T, true>(x, vocab, k, share, c, parts, sm, top);
  if (k > 0) join_tops(sm, top, k);
  st = warp_join(st);
  if (lane == 0) sm.stat[warp] = st;
  __syncthreads();
  st = sm.stat[0];
  for (int w = 1; w < kThreads / 32; ++w) st = join(st, sm.stat[w]);
  if (parts > 1) {
    score::Part* mine = part + (int64_t)row * parts + c;
    if (tid == 0) {
      mine->m = st.m;
      mine->z = st.z;
      mine->u = st.u;
      mine->bad = st.bad;
    }
    if (tid < k) mine->key[tid] = sm.best[tid];
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      sm.last = atomicAdd(&tickets[row], 1u) == (uint32_t)(parts - 1);
      if (sm.last) tickets[row] = 0;
    }
    __syncthreads();
    if (!sm.last) return;
    __threadfence();
    const score::Part* all = part + (int64_t)row * parts;
    // (every warp for itself: two parts a lane, then the tree over the lanes)
    static_assert(score::kMaxParts <= 64, "two parts a lane");
    Stat s2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int q = lane + 32 * i;
      s2[i] = Stat{-INFINITY, 0.f, 0.f, 0};
      if (q < parts) {
        const int4 w = __ldcg(reinterpret_cast<const int4*>(&all[q]));
        s2[i] = Stat{__int_as_float(w.x), __int_as_float(w.y), __int_as_float(w.z), w.w};
      }
    }
    st = warp_join(join(s2[0], s2[1]));
    if (k > 0) {
      top.reset();
      constexpr int kN = score::kMaxParts * kMaxK / kThreads;
      Key key[kN];
      Key mine = 0;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int e = tid + i * kThreads, q = e / kMaxK;  // (kMaxK keys of room a part, k of them in use)
        key[i] = q < parts && e % kMaxK < k ? __ldcg(&all[q].key[e % kMaxK]) : 0;
        mine = key[i] > mine ? key[i] : mine;
      }
      const uint32_t o = warp_kth(mine != 0 ? key_value(mine) : -INFINITY, share, lane);
      if (lane == 0) sm.reached[warp] = o;
      if (tid == 0) sm.count = 0;
      __syncthreads();
      const float floor = floor_now(sm, lane);
      uint32_t mask = 0;
#pragma unroll
      for (int i = 0; i < kN; ++i) mask |= key[i] == 0 || key_value(key[i]) < floor ? 0u : 1u << i;
#pragma unroll 1
      while (__any_sync(0xffffffffu, mask != 0)) {
        const int bit = mask != 0 ? __ffs(mask) - 1 : 0;
        Key y = key[0];
#pragma unroll
        for (int i = 1; i < kN; ++i) y = bit == i ? key[i] : y;
        top.offer(mask != 0 ? y : 0, k, lane);
        mask &= mask - 1;
      }
      publish(sm, top, share, lane, warp);
      join_tops(sm, top, k);
    }
  }
  const float lz = logf(st.z);
  const bool none = st.bad != 0 || st.m == -INFINITY;
  const float nan = __uint_as_float(0x7FC00000u);
  if (tid == 0) {
    const int32_t tg = __ldcg(targets + row);
    float lp = 0.f;
    if (tg != -1) {
      const bool in = tg >= 0 && tg < vocab;
      if (!in) atomicOr(err, kErrIndex);
      lp = in && !none ? load1(x + tg) - st.m - lz : nan;
    }
    logprob[row] = lp;
    entropy[row] = none ? nan : lz - st.u / st.z;
  }
  if (tid < k) {
    const Key key = sm.best[tid];
    top_ids[(int64_t)row * k + tid] = key_index(key);
    top_logprobs[(int64_t)row * k + tid] = none ? nan : key_value(key) - st.m - lz;
  }
}

}  // namespace

cudaError_t launch_score(const void* logits, int64_t ld, int dtype, int n_rows, int vocab, const int32_t* targets, int k,
                         float* logprob, float* entropy, int32_t* top_ids, float* top_logprobs, void* workspace,
                         cudaStream_t st) {
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  uint32_t* err = reinterpret_cast<uint32_t*>(ws);
  uint32_t* tickets = reinterpret_cast<uint32_t*>(ws + score::kTickets);
  score::Part* part = reinterpret_cast<score::Part*>(ws + score::kParts);
  const int parts = score::parts_for(n_rows, vocab);
  const dim3 grid((unsigned)n_rows * (unsigned)parts);
  if (dtype == SPARK_BF16)
    return launch_pdl(k_score<__nv_bfloat16>, grid, dim3(kThreads), 0, st, static_cast<const __nv_bfloat16*>(logits), ld,
                      vocab, targets, k, parts, logprob, entropy, top_ids, top_logprobs, err, tickets, part);
  return launch_pdl(k_score<float>, grid, dim3(kThreads), 0, st, static_cast<const float*>(logits), ld, vocab, targets,
                    k, parts, logprob, entropy, top_ids, top_logprobs, err, tickets, part);
}

}  // namespace spark
