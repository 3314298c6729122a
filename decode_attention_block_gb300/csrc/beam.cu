// beam.cu -- a step of beam search (spark_beam_select) and the beams' states in
// their new order (spark_beam_reorder).
//
// One pass over the logits of the live beams leaves for each part of a row its
// maximum, its sum of exponentials and its best n_beams logits (score_parts.cuh):
// within a row the offers are ordered as the logits are, so no other can be
// chosen.  The last CTA of a group to arrive joins them: an offer's score is
// (score - ln z) + (x - m) in 64 bits, and the order (score, then the
// lower beam, then the lower token) of which no two offers are equal.  Lists are
// sorted, so the n_beams best offers are in the n_beams lists of highest heads:
// a floor that n_beams heads reach (a few reductions in a warp), the exact
// ranks of the heads above it, then the ranks of at most n_beams^2 offers.
#include <math.h>

#include "beam.h"
#include "launch.h"
#include "score_parts.cuh"

namespace spark {
namespace {

using namespace score;
using beam::Part;
using beam::Select;

constexpr int kMaxBeams = SPARK_MAX_BEAMS;
constexpr int kLists = beam::kMaxPairs;  // of a group at most

struct Offers {
  double value[kLists];
  uint32_t id[kLists];     // beam * vocab + token
  uint16_t list[kLists];
  double base[kMaxBeams];  // score - ln z; -inf: the beam offers nothing
  float top[kMaxBeams];    // m
  int ended[kMaxBeams];
  double t_value;          // the least head that counts
  uint32_t t_id;
  int count, n_lists;
  uint16_t lists[kMaxBeams];
  double best[kMaxBeams];
  uint32_t best_id[kMaxBeams];
};
static_assert(kLists >= kMaxBeams * kMaxBeams, "room for the offers of the lists that count");

__device__ __forceinline__ bool above(double v, uint32_t i, double w, uint32_t j) { return v > w || (v == w && i < j); }

__device__ __forceinline__ double warp_sum_double(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// the rank of offer (v, i) among the n in sm, all different
__device__ __forceinline__ int rank_of(const Offers& sm, int n, double v, uint32_t i) {
  int r = 0;
  for (int j = 0; j < n; ++j) r += above(sm.value[j], sm.id[j], v, i);
  return r;
}

// whether a slot offers continuations of its own row
__device__ __forceinline__ bool is_live(float score, int done) { return done == 0 && fabsf(score) < INFINITY; }

// The last CTA of group `group`: its offers joined, the best written.
__device__ __forceinline__ void join_group(const Select& a, int group, int k, int parts, Offers& sm, Smem& reach) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int W = a.n_beams, slot0 = group * W;
  // the rows' bases: a warp each in turn
  for (int b = warp; b < W; b += kWarps) {
    const float score = __ldcg(a.score + slot0 + b);
    const int done = a.done ? __ldcg(a.done + slot0 + b) : 0;
    const bool live = is_live(score, done);
    double base = -INFINITY;
    float top = -INFINITY;
    if (live) {
      float m[beam::kMaxParts / 32];
      double z[beam::kMaxParts / 32];
      bool bad = false;
#pragma unroll
      for (int i = 0; i < beam::kMaxParts / 32; ++i) {
        const int c = lane + 32 * i;
        m[i] = -INFINITY;
        z[i] = 0.0;
        if (c < parts) {
          const Part* q = a.part + (int64_t)(slot0 + b) * parts + c;
          m[i] = __ldcg(&q->m);
          z[i] = __ldcg(&q->z);
          bad = bad || __ldcg(&q->bad) != 0;
        }
        top = fmaxf(top, m[i]);
      }
      top = warp_max(top);
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < beam::kMaxParts / 32; ++i)
        if (m[i] > -INFINITY) sum += z[i] * exp((double)(m[i] - top));
      sum = warp_sum_double(sum);
      if (!__any_sync(0xffffffffu, bad) && top > -INFINITY) base = (double)score - log(sum);
    } else if (done != 0 && fabsf(score) < INFINITY) {
      base = (double)score;
    }
    if (lane == 0) {
      sm.base[b] = base;
      sm.top[b] = top;
      sm.ended[b] = done != 0;
    }
  }
  if (tid == 0) {
    sm.count = 0;
    sm.n_lists = 0;
    sm.t_value = -INFINITY;
    sm.t_id = 0xFFFFFFFFu;
  }
  __syncthreads();
  // list l: part l % parts of beam l / parts; an ended beam has one, of one offer
  const int lists = W * parts;
  auto entry = [&](int l, int i, double& v, uint32_t& id) {
    const int b = l / parts, c = l - b * parts;
    const double base = sm.base[b];
    v = -INFINITY;
    id = 0xFFFFFFFFu;
    if (!(base > -INFINITY)) return;
    if (sm.ended[b]) {
      if (c == 0 && i == 0) {
        v = base;
        id = (uint32_t)b * (uint32_t)a.vocab + (uint32_t)a.eos;
      }
      return;
    }
    const Key key = __ldcg(&a.part[(int64_t)(slot0 + b) * parts + c].key[i]);
    if (key == 0) return;
    // (x - m first: logits may be far larger than the scores; -inf: no offer)
    v = base + ((double)key_value(key) - (double)sm.top[b]);
    id = (uint32_t)b * (uint32_t)a.vocab + (uint32_t)key_index(key);
  };
  constexpr int kHeads = kLists / kThreads;
  double v[kHeads];
  uint32_t id[kHeads];
  float mine = -INFINITY;
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int l = tid + i * kThreads;
    v[i] = -INFINITY;
    id[i] = 0xFFFFFFFFu;
    if (l < lists) entry(l, 0, v[i], id[i]);
    mine = fmaxf(mine, (float)v[i]);
  }
  // a floor that W heads reach, in fp32 (rounding keeps the order)
  const uint32_t o = warp_kth(mine, (W + kWarps - 1) / kWarps, lane);
  if (lane == 0) reach.reached[warp] = o;
  __syncthreads();
  const float floor = floor_now(reach, lane);
#pragma unroll
  for (int i = 0; i < kHeads; ++i)
    if (v[i] > -INFINITY && !((float)v[i] < floor)) {
      const int at = atomicAdd(&sm.count, 1);
      sm.value[at] = v[i];
      sm.id[at] = id[i];
      sm.list[at] = (uint16_t)(tid + i * kThreads);
    }
  __syncthreads();
  const int heads = sm.count;
  for (int e = tid; e < heads; e += kThreads)
    if (rank_of(sm, heads, sm.value[e], sm.id[e]) < W) sm.lists[atomicAdd(&sm.n_lists, 1)] = sm.list[e];
  __syncthreads();
  // the offers of these lists
  const int n_lists = sm.n_lists;
  if (tid == 0) sm.count = 0;
  __syncthreads();
  for (int e = tid; e < n_lists * k; e += kThreads) {
    double x;
    uint32_t xi;
    entry(sm.lists[e / k], e % k, x, xi);
    if (x > -INFINITY) {
      const int at = atomicAdd(&sm.count, 1);
      sm.value[at] = x;
      sm.id[at] = xi;
    }
  }
  __syncthreads();
  const int n = sm.count;
  for (int e = tid; e < n; e += kThreads) {
    const double x = sm.value[e];
    const uint32_t xi = sm.id[e];
    const int r = rank_of(sm, n, x, xi);
    if (r < W) {
      sm.best[r] = x;
      sm.best_id[r] = xi;
    }
  }
  __syncthreads();
  // (what the parents were is read before any slot of the group is written)
  int parent = -1, token = -1, done = 1, keep = 0, grow = 0;
  float score = -INFINITY;
  if (tid < W && tid < n) {
    const int b = (int)(sm.best_id[tid] / (uint32_t)a.vocab);
    token = (int)(sm.best_id[tid] - (uint32_t)b * (uint32_t)a.vocab);
    parent = slot0 + b;
    score = (float)sm.best[tid];
    const bool was = sm.ended[b] != 0;
    done = was || token == a.eos;
    if (a.length) {
      keep = __ldcg(a.length + parent);
      grow = keep + (was ? 0 : 1);
    }
  }
  __syncthreads();
  if (tid < W) {
    const int s = slot0 + tid;
    a.new_score[s] = score;
    a.token[s] = token;
    a.parent[s] = parent;
    if (a.new_done) a.new_done[s] = done;
    if (a.length) {
      a.keep_len[s] = keep;
      a.new_len[s] = grow;
    }
  }
}

// CTA (row, part)
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_beam_select(const __grid_constant__ Select a, int k, int parts) {
  __shared__ Smem sm;
  __shared__ Offers offers;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / parts, c = blockIdx.x % parts, group = row / a.n_beams;
  if (tid == 0) sm.count = 0;
  pdl_wait();
  pdl_trigger();
  if (is_live(__ldcg(a.score + row), a.done ? __ldcg(a.done + row) : 0)) {
    const int share = (k + kWarps - 1) / kWarps;  // of the k, a warp's
    WarpTop top;
    top.reset();
    const Stat st = row_pass<T, false>(static_cast<const T*>(a.logits) + row * a.ld, a.vocab, k, share, c, parts, sm, top);
    join_tops(sm, top, k);
    // the block's sum in 64 bits: scores of different beams are compared
    const float wm = warp_max(st.m);
    const double wz = warp_sum_double(st.m > -INFINITY ? (double)st.z * (double)expf(st.m - wm) : 0.0);
    const bool wbad = __any_sync(0xffffffffu, st.bad != 0);
    if (lane == 0) {
      sm.stat[warp].m = wm;
      sm.stat[warp].bad = wbad;
      offers.value[warp] = wz;
    }
    __syncthreads();
    Part* mine = a.part + (int64_t)row * parts + c;
    if (warp == 0) {
      const float m = lane < kWarps ? sm.stat[lane].m : -INFINITY, bm = warp_max(m);
      const double z = warp_sum_double(m > -INFINITY ? offers.value[lane] * exp((double)(m - bm)) : 0.0);
      const bool bad = __any_sync(0xffffffffu, lane < kWarps && sm.stat[lane].bad != 0);
      if (lane == 0) {
        mine->m = bm;
        mine->bad = bad;
        mine->z = z;
      }
    }
    if (tid < k) mine->key[tid] = tid < sm.count ? sm.best[tid] : 0;
    __threadfence();
  }
  __syncthreads();
  if (tid == 0) {
    sm.last = atomicAdd(&a.tickets[group], 1u) == (uint32_t)(a.n_beams * parts - 1);
    if (sm.last) a.tickets[group] = 0;
  }
  __syncthreads();
  if (!sm.last) return;
  __threadfence();
  join_group(a, group, k, parts, offers, sm);
}

constexpr int kMoveThreads = 256;
constexpr int64_t kMovePiece = 32768;  // bytes of a row a CTA copies

// CTA (slot, state, piece of its row)
__global__ void __launch_bounds__(kMoveThreads)
    k_beam_reorder(const int32_t* parent, const int32_t* keep_len, const int32_t* new_len, int n_slots,
                   const __grid_constant__ beam::States states, uint32_t* err) {
  const int s = blockIdx.x;
  const spark_beam_state& st = states.s[blockIdx.y];
  pdl_wait();
  const int par = __ldcg(parent + s);
  if (par == -1) return;
  bool ok = par >= 0 && par < n_slots;
  int64_t bytes = st.pitch;
  int keep = 0, grow = 0;
  if (st.elem > 0) {
    keep = __ldcg(keep_len + s);
    grow = __ldcg(new_len + s);
    const int64_t room = st.pitch / st.elem;
    ok = ok && keep >= 0 && keep <= grow && keep <= room && (st.push == nullptr || grow == keep || keep < room);
    bytes = (int64_t)keep * st.elem;
  }
  if (!ok) {
    if (threadIdx.x == 0 && blockIdx.z == 0) atomicOr(err, kErrIndex);
    return;
  }
  const unsigned char* src = static_cast<const unsigned char*>(st.src) + par * st.pitch;
  unsigned char* dst = static_cast<unsigned char*>(st.dst) + s * st.pitch;
  const bool wide = ((reinterpret_cast<uintptr_t>(st.src) | reinterpret_cast<uintptr_t>(st.dst) | (uintptr_t)st.pitch) & 15u) == 0;
  for (int64_t at = blockIdx.z * kMovePiece; at < bytes; at += gridDim.z * kMovePiece) {
    const int n = (int)(bytes - at < kMovePiece ? bytes - at : kMovePiece);
    const int n16 = wide ? n / 16 : 0;
    for (int i = threadIdx.x; i < n16; i += kMoveThreads)
      reinterpret_cast<uint4*>(dst + at)[i] = __ldcg(reinterpret_cast<const uint4*>(src + at) + i);
    for (int i = 4 * n16 + threadIdx.x; i < n / 4; i += kMoveThreads)
      reinterpret_cast<uint32_t*>(dst + at)[i] = __ldcg(reinterpret_cast<const uint32_t*>(src + at) + i);
  }
  if (st.push != nullptr && grow > keep && blockIdx.z == 0 && threadIdx.x == 0)
    reinterpret_cast<int32_t*>(dst)[keep] = __ldcg(st.push + s);
}

}  // namespace

cudaError_t launch_beam_select(const Select& a, int dtype, cudaStream_t st) {
  const int rows = a.n_groups * a.n_beams, parts = beam::parts_for(rows, a.vocab);
  const int k = a.n_beams < a.vocab ? a.n_beams : a.vocab;
  auto kern = dtype == SPARK_BF16 ? k_beam_select<__nv_bfloat16> : k_beam_select<float>;
  return launch_pdl(kern, dim3((unsigned)(rows * parts)), dim3(kThreads), 0, st, a, k, parts);
}

cudaError_t launch_beam_reorder(const int32_t* parent, const int32_t* keep, const int32_t* grow, int n_slots,
                                const beam::States& states, int n_states, uint32_t* err, cudaStream_t st) {
  int64_t most = 0;
  for (int i = 0; i < n_states; ++i) most = states.s[i].pitch > most ? states.s[i].pitch : most;
  int64_t pieces = (most + kMovePiece - 1) / kMovePiece;
  pieces = pieces < 1 ? 1 : pieces > 64 ? 64 : pieces;
  return launch_pdl(k_beam_reorder, dim3(n_slots, n_states, (unsigned)pieces), dim3(kMoveThreads), 0, st, parent, keep, grow,
                    n_slots, states, err);
}

}  // namespace spark
