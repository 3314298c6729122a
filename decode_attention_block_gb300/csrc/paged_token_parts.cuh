// paged_token_parts.cuh -- what the kernels of single new tokens share
// (paged_attn.cu: fp32 and bf16 pages; paged4_attn.cu: 4-bit ones): which CTAs
// share a group, the merge of its partial states and its output.
#pragma once

#include <math.h>

#include "attn_parts.cuh"
#include "paged_parts.cuh"

namespace spark {
namespace token {

using paged::Args;

// eight output dims of one head
__device__ __forceinline__ void store8(float* dst, const float (&o)[8], float inv) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
  reinterpret_cast<float4*>(dst)[1] = make_float4(o[4] * inv, o[5] * inv, o[6] * inv, o[7] * inv);
}
__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float (&o)[8], float inv) {
  *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                                              pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
}

// The CTAs of a group, first and last, the slots of this CTA's partial state
// and of the first's (the others' are their CTAs' first).
struct Parts {
  int first, last, slot, slot0;
  __device__ __forceinline__ Parts(int64_t begin, int64_t end, int64_t total, int G, int c)
      : first(paged::cta_at(begin, total, G)),
        last(paged::cta_at(end - 1, total, G)),
        slot(paged::partial_slot(c, begin, total, G)),
        slot0(paged::partial_slot(first, begin, total, G)) {}
};

// Where dim d of a head lies in a warp's state in shared memory, PAD floats
// behind each 32, and the floats of a head.
template <int PAD>
__device__ __forceinline__ constexpr int state_at(int d) { return d + (d >> 5) * PAD; }
template <int PAD>
constexpr int kStateFloats = kHeadDim + kHeadDim / 32 * PAD;

// The group's state from the consumer warps' states in `sm`: finished if
// whole, else this CTA's partial; the last of the group's CTAs to arrive
// merges them in CTA order.  Warp h takes query head h, lane l its dims
// [8 l, 8 l + 8); the warps' states are WARP floats apart.  (Over fp32 and bf16
// pages the parts are worked out before the tiles arrive: their divisions took up to
// 2000 cycles here.  Over 4-bit ones, where registers are short, they are not.)
template <typename QT, int PAD = 0, int WARP = 4 * kStateFloats<PAD>>
__device__ __forceinline__ void finish_group(const MergeSmem& sm, volatile int* flags, const Args& p, QT* a_head0,
                                             const Parts& parts) {
  const int tid = threadIdx.x, h = tid >> 5, lane = tid & 31;
  named_bar_sync(kBarConsumers, kConsumerThreads);
  float M = -INFINITY;
#pragma unroll
  for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, sm.ms[w * 4 + h]);
  float L = 0.f, O[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) O[i] = 0.f;
#pragma unroll
  for (int w = 0; w < kConsumers; ++w) {
    const float mw = sm.ms[w * 4 + h];
    const float scl = mw == -INFINITY ? 0.f : exp2f(mw - M);
    L = fmaf(sm.ls[w * 4 + h], scl, L);
    const float4* src = reinterpret_cast<const float4*>(sm.os + w * WARP + h * kStateFloats<PAD> + state_at<PAD>(8 * lane));
    const float4 x0 = src[0], x1 = src[1];
    O[0] = fmaf(x0.x, scl, O[0]); O[1] = fmaf(x0.y, scl, O[1]);
    O[2] = fmaf(x0.z, scl, O[2]); O[3] = fmaf(x0.w, scl, O[3]);
    O[4] = fmaf(x1.x, scl, O[4]); O[5] = fmaf(x1.y, scl, O[5]);
    O[6] = fmaf(x1.z, scl, O[6]); O[7] = fmaf(x1.w, scl, O[7]);
  }
  QT* dst = a_head0 + h * kHeadDim + 8 * lane;
  const int c_first = parts.first, c_last = parts.last;
  if (c_first == c_last) {
    if (!flags[0]) store8(dst, O, 1.0f / L);
    return;
  }
  float* P = p.part + (int64_t)parts.slot * kPartFloats;
  float4* po = reinterpret_cast<float4*>(P + 8 + h * kHeadDim + 8 * lane);
  po[0] = make_float4(O[0], O[1], O[2], O[3]);
  po[1] = make_float4(O[4], O[5], O[6], O[7]);
  if (lane == 0) {
    P[h] = M;
    P[4 + h] = L;
  }
  named_bar_sync(kBarMerge, kConsumerThreads);
  if (tid == 0) {
    __threadfence();  // the block's partial, ordered before this thread by the barrier, before the ticket
    // the group's ticket is that of its first CTA, where no other split group
    // begins; every arrival counts, so the ticket is back at zero after it
    const int last = atomicAdd(&p.tickets[c_first], 1u) == (uint32_t)(c_last - c_first);
    if (last) p.tickets[c_first] = 0;
    flags[1] = last && !flags[0];
    if (last) __threadfence();  // the ticket before the others' partials
  }
  named_bar_sync(kBarMerge, kConsumerThreads);
  if (!flags[1]) return;
  float M2 = -INFINITY, L2 = 0.f, O2[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) O2[i] = 0.f;
  constexpr int kBatch = 8;  // partials loaded per round trip
  for (int q0 = c_first; q0 <= c_last; q0 += kBatch) {
    float mq[kBatch], lq[kBatch];
    float4 x0[kBatch], x1[kBatch];
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      // (behind the last part the last once more, at weight 0: loads without
      // a condition stay in flight together)
      const int q = min(q0 + t, c_last);
      const float* Pq = p.part + (int64_t)(q == c_first ? parts.slot0 : 2 * q) * kPartFloats;
      mq[t] = __ldcg(Pq + h);
      lq[t] = __ldcg(Pq + 4 + h);
      x0[t] = __ldcg(reinterpret_cast<const float4*>(Pq + 8 + h * kHeadDim + 8 * lane));
      x1[t] = __ldcg(reinterpret_cast<const float4*>(Pq + 8 + h * kHeadDim + 8 * lane + 4));
      if (q0 + t > c_last) mq[t] = -INFINITY;
    }
    float mb = M2;
#pragma unroll
    for (int t = 0; t < kBatch; ++t) mb = fmaxf(mb, mq[t]);
    const float rs = M2 == -INFINITY ? 0.f : exp2f(M2 - mb);
    L2 *= rs;
#pragma unroll
    for (int i = 0; i < 8; ++i) O2[i] *= rs;
    M2 = mb;
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      const float scl = mq[t] == -INFINITY ? 0.f : exp2f(mq[t] - M2);
      L2 = fmaf(lq[t], scl, L2);
      O2[0] = fmaf(x0[t].x, scl, O2[0]); O2[1] = fmaf(x0[t].y, scl, O2[1]);
      O2[2] = fmaf(x0[t].z, scl, O2[2]); O2[3] = fmaf(x0[t].w, scl, O2[3]);
      O2[4] = fmaf(x1[t].x, scl, O2[4]); O2[5] = fmaf(x1[t].y, scl, O2[5]);
      O2[6] = fmaf(x1[t].z, scl, O2[6]); O2[7] = fmaf(x1[t].w, scl, O2[7]);
    }
  }
  store8(dst, O2, 1.0f / L2);
}

}  // namespace token
}  // namespace spark
