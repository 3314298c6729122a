// beam.cu -- a step of beam search (spark_beam_select) and the beams' states in
// their new order (spark_beam_reorder).
//
// One pass over the logits of the live beams leaves for each part of a row its
// maximum, its sum of exponentials and its best n_beams logits (score_parts.cuh):
// within a row the offers are ordered as the logits are, so no other can be
// chosen.  The last CTA of a group to arrive joins them: an offer's score is
// (score - ln z) + (x - m), and the order (score, then the lower beam, then the
// lower token) of which no two offers are equal.  Lists are sorted, so the n_beams
// best offers are in the n_beams lists of highest heads: a floor that n_beams
// heads reach (a few reductions in a warp), the exact ranks of the heads above it,
// then the ranks of their offers that reach the last of these n_beams.
//
// Sums and scores are pairs of fp32 numbers (a number and what it leaves: 48
// bits), so that the order of offers of different beams is not left to fp32, whose
// steps at a score of -30 are 2e-6; an offer's pair is one 64-bit integer to
// compare.  (fp64 runs at a 64th of fp32's rate here: one group of 4 beams took 30
// us with the reorder when it joined in fp64, now 17.)  The one logarithm of each
// row is fp64, a row a lane.
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

// x + y, exactly where |x_lo|, |y_lo| are what their parts leave, to 2^-48
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
  return Two{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z))};
}
__device__ __forceinline__ Two add(Two x, Two y) {
  const Two s = two_sum(x.hi, y.hi);
  return Two{s.hi, __fadd_rn(s.lo, __fadd_rn(x.lo, y.lo))};
}
// so that hi is the sum rounded
__device__ __forceinline__ Two settle(Two x) {
  const float s = __fadd_rn(x.hi, x.lo);
  return Two{s, __fsub_rn(x.lo, __fsub_rn(s, x.hi))};
}
__device__ __forceinline__ Two scaled(Two x, float f) {
  const float p = __fmul_rn(x.hi, f);
  return Two{p, __fmaf_rn(x.lo, f, __fmaf_rn(x.hi, f, -p))};
}
__device__ __forceinline__ Two warp_sum(Two x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    x = add(x, Two{__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)});
  return x;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// An offer: its score in the order of integers (a settled pair, the first
// number's order above the second's), and beam * vocab + token.  Value 0: none.
struct Offer {
  unsigned long long value;
  uint32_t id;
};
__device__ __forceinline__ unsigned long long value_key(Two v) {
  return ((unsigned long long)order_of(v.hi) << 32) | order_of(v.lo);
}
__device__ __forceinline__ float offer_score(unsigned long long value) { return value_of((uint32_t)(value >> 32)); }
__device__ __forceinline__ bool above(unsigned long long v, uint32_t i, unsigned long long w, uint32_t j) {
  return v > w || (v == w && i < j);
}

struct Offers {
  unsigned long long value[kLists];
  uint32_t id[kLists];     // beam * vocab + token
  uint16_t list[kLists];
  Two base[kMaxBeams];     // score - ln z; hi -inf: the beam offers nothing
  Two z[kMaxBeams];
  float top[kMaxBeams];    // m
  int ended[kMaxBeams];
  int count, n_lists;
  unsigned long long least;  // the head that n_beams - 1 others are above, if there are as many
  uint32_t least_id;
  uint16_t lists[kMaxBeams];
  unsigned long long best[kMaxBeams];
  uint32_t best_id[kMaxBeams];
};
static_assert(kLists >= kMaxBeams * kMaxBeams, "room for the offers of the lists that count");

// the rank of offer (v, i) among the n in sm, all different
__device__ __forceinline__ int rank_of(const Offers& sm, int n, unsigned long long v, uint32_t i) {
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
  // the lists' heads, asked for while the rows' sums are joined: list l is part l %
  // parts of beam l / parts; an ended beam has one, of one offer
  const int lists = W * parts;
  constexpr int kHeads = kLists / kThreads;
  auto key_of = [&](int l, int i) { return __ldcg(&a.part[(int64_t)slot0 * parts + l].key[i]); };
  Key first[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) first[i] = tid + i * kThreads < lists ? key_of(tid + i * kThreads, 0) : 0;
  // the rows' sums, a warp each in turn
  for (int b = warp; b < W; b += kWarps) {
    const float score = __ldcg(a.score + slot0 + b);
    const int done = a.done ? __ldcg(a.done + slot0 + b) : 0;
    const bool live = is_live(score, done);
    float top = -INFINITY;
    Two z = {0.f, 0.f};
    bool bad = false;
    if (live) {
      constexpr int kEach = beam::kMaxParts / 32;
      float m[kEach];
      Two part[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int c = lane + 32 * i;
        m[i] = -INFINITY;
        part[i] = Two{0.f, 0.f};
        if (c < parts) {
          const float4 q = __ldcg(reinterpret_cast<const float4*>(a.part + (int64_t)(slot0 + b) * parts + c));
          m[i] = q.x;
          bad = bad || __float_as_int(q.y) != 0;
          part[i] = Two{q.z, q.w};
        }
        top = fmaxf(top, m[i]);
      }
      top = warp_max(top);
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (m[i] > -INFINITY) z = add(z, scaled(part[i], expf(m[i] - top)));
      z = warp_sum(z);
      bad = __any_sync(0xffffffffu, bad);
    }
    if (lane == 0) {
      const bool any = live ? !bad && top > -INFINITY : done != 0 && fabsf(score) < INFINITY;
      sm.base[b] = Two{any ? score + 0.f : -INFINITY, 0.f};  // (-0 is 0: equal scores have equal keys)
      sm.z[b] = z;
      sm.top[b] = top;
      sm.ended[b] = done != 0;
    }
  }
  if (tid == 0) {
    sm.count = 0;
    sm.n_lists = 0;
    sm.least = 0;
    sm.least_id = 0xFFFFFFFFu;
  }
  __syncthreads();
  if (tid < W && sm.base[tid].hi > -INFINITY && !sm.ended[tid]) {
    const double base = (double)sm.base[tid].hi - log((double)sm.z[tid].hi + (double)sm.z[tid].lo);
    const float hi = (float)base;
    sm.base[tid] = Two{hi, (float)(base - (double)hi)};
  }
  __syncthreads();
  // offer i of list l, whose key it is (a beam that offers none left stale ones)
  auto entry = [&](int l, int i, Key key) {
    const int b = l / parts, c = l - b * parts;
    const Two base = sm.base[b];
    if (!(base.hi > -INFINITY)) return Offer{0, 0};
    if (sm.ended[b]) {
      if (c != 0 || i != 0) return Offer{0, 0};
      return Offer{value_key(base), (uint32_t)b * (uint32_t)a.vocab + (uint32_t)a.eos};
    }
    const float x = key_value(key);
    if (key == 0 || !(x > -INFINITY)) return Offer{0, 0};
    // (x - m first: logits may be far larger than the scores)
    const Two v = settle(add(settle(two_sum(x, -sm.top[b])), base));
    if (!(fabsf(v.hi) < INFINITY)) return Offer{0, 0};  // below what fp32 holds
    return Offer{value_key(v), (uint32_t)b * (uint32_t)a.vocab + (uint32_t)key_index(key)};
  };
  Offer head[kHeads];
  float mine = -INFINITY;
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int l = tid + i * kThreads;
    head[i] = l < lists ? entry(l, 0, first[i]) : Offer{0, 0};
    if (head[i].value != 0) mine = fmaxf(mine, offer_score(head[i].value));
  }
  // a floor that W heads reach, in fp32 (rounding keeps the order)
  const uint32_t o = warp_kth(mine, (W + kWarps - 1) / kWarps, lane);
  if (lane == 0) reach.reached[warp] = o;
  __syncthreads();
  const float floor = floor_now(reach, lane);
#pragma unroll
  for (int i = 0; i < kHeads; ++i)
    if (head[i].value != 0 && !(offer_score(head[i].value) < floor)) {
      const int at = atomicAdd(&sm.count, 1);
      sm.value[at] = head[i].value;
      sm.id[at] = head[i].id;
      sm.list[at] = (uint16_t)(tid + i * kThreads);
    }
  __syncthreads();
  const int heads = sm.count;
  for (int e = tid; e < heads; e += kThreads) {
    const int r = rank_of(sm, heads, sm.value[e], sm.id[e]);
    if (r < W) sm.lists[atomicAdd(&sm.n_lists, 1)] = sm.list[e];
    if (r == W - 1) {
      sm.least = sm.value[e];
      sm.least_id = sm.id[e];
    }
  }
  __syncthreads();
  // the offers of these lists that are not below all n_beams heads
  const int n_lists = sm.n_lists;
  if (tid == 0) sm.count = 0;
  __syncthreads();
  for (int e = tid; e < n_lists * k; e += kThreads) {
    const int l = sm.lists[e / k], i = e % k;
    const Offer x = entry(l, i, key_of(l, i));
    if (x.value != 0 && !above(sm.least, sm.least_id, x.value, x.id)) {
      const int at = atomicAdd(&sm.count, 1);
      sm.value[at] = x.value;
      sm.id[at] = x.id;
    }
  }
  __syncthreads();
  const int n = sm.count;
  for (int e = tid; e < n; e += kThreads) {
    const unsigned long long x = sm.value[e];
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
    score = offer_score(sm.best[tid]);
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
    const float wm = warp_max(st.m);
    const Two wz = warp_sum(scaled(Two{st.z, 0.f}, st.m > -INFINITY ? expf(st.m - wm) : 0.f));
    const bool wbad = __any_sync(0xffffffffu, st.bad != 0);
    if (lane == 0) sm.stat[warp] = Stat{wm, wz.hi, wz.lo, wbad};
    __syncthreads();
    Part* mine = a.part + (int64_t)row * parts + c;
    if (warp == 0) {
      const Stat w = lane < kWarps ? sm.stat[lane] : Stat{-INFINITY, 0.f, 0.f, 0};
      const float m = warp_max(w.m);
      const Two z = warp_sum(scaled(Two{w.z, w.u}, w.m > -INFINITY ? expf(w.m - m) : 0.f));
      const bool bad = __any_sync(0xffffffffu, w.bad != 0);
      if (lane == 0) *reinterpret_cast<float4*>(mine) = make_float4(m, __int_as_float(bad), z.hi, z.lo);
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
