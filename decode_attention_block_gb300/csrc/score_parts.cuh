// score_parts.cuh -- one pass over rows of logits, shared by the token scores
// (score.cu) and beam search (beam.cu): a row's maximum and sums, and its
// highest logits (the scheme: score.cu).
#pragma once

#include <math.h>

#include "common.cuh"
#include "../../include/spark_score.h"

namespace spark {
namespace score {

constexpr int kThreads = 256;
constexpr int kVecs = 4;            // 16-byte words per thread and tile
constexpr int kMaxK = SPARK_MAX_TOP;
constexpr int kWarps = kThreads / 32;

using Key = unsigned long long;

// the order of floats as that of integers: NaN lowest, -0 and 0 equal
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return x != x ? 0u : (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return o == 0u ? __uint_as_float(0x7FC00000u) : __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ Key make_key(float x, uint32_t idx) {
  return ((Key)order_of(x) << 32) | (0xFFFFFFFFu - idx);
}
__device__ __forceinline__ float key_value(Key k) { return value_of((uint32_t)(k >> 32)); }
__device__ __forceinline__ int32_t key_index(Key k) { return (int32_t)(0xFFFFFFFFu - (uint32_t)k); }

struct Stat {
  float m, z, u;
  int bad;  // a NaN or +inf among the logits
};

__device__ __forceinline__ Stat join(const Stat& a, const Stat& b) {
  Stat r;
  r.m = fmaxf(a.m, b.m);
  r.bad = a.bad | b.bad;
  const float ref = r.m == -INFINITY ? 0.f : r.m;
  const float da = a.m == -INFINITY ? 0.f : a.m - ref, db = b.m == -INFINITY ? 0.f : b.m - ref;
  const float ea = expf(da), eb = expf(db);
  r.z = fmaf(a.z, ea, b.z * eb);
  // (a mask of the type's lowest value: e = 0, and d z may overflow)
  r.u = (ea > 0.f ? (a.u + da * a.z) * ea : 0.f) + (eb > 0.f ? (b.u + db * b.z) * eb : 0.f);
  return r;
}

__device__ __forceinline__ Stat warp_join(Stat s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat t;
    t.m = __shfl_xor_sync(0xffffffffu, s.m, o);
    t.z = __shfl_xor_sync(0xffffffffu, s.z, o);
    t.u = __shfl_xor_sync(0xffffffffu, s.u, o);
    t.bad = __shfl_xor_sync(0xffffffffu, s.bad, o);
    s = join(s, t);
  }
  return s;
}

struct Smem {
  Stat stat[kWarps];
  Key list[kWarps * kMaxK];  // the warps' keys at the end
  Key best[kMaxK];
  uint32_t reached[kWarps];  // c logits of the warp reach this (order_of)
  int count;
  int last;
};

constexpr uint32_t kLowest = 0x007FFFFFu;  // -inf

// The c-th largest of the lanes' values (NaN: none).
__device__ __forceinline__ uint32_t warp_kth(float mine, int c, int lane) {
  uint32_t x = order_of(mine), top = 0;
  for (int i = 0; i < c; ++i) {
    top = __reduce_max_sync(0xffffffffu, x);
    if (lane == __ffs(__ballot_sync(0xffffffffu, x == top)) - 1) x = 0;
  }
  return top;
}

__device__ __forceinline__ float floor_now(const Smem& sm, int lane) {
  const uint32_t o = lane < kWarps ? *(const volatile uint32_t*)&sm.reached[lane] : 0xFFFFFFFFu;
  const uint32_t least = __reduce_min_sync(0xffffffffu, o);
  return value_of(least < kLowest ? kLowest : least);
}

// A warp's best k keys: lane i holds the i-th (0: none), every lane the k-th.
struct WarpTop {
  Key key, least;
  __device__ __forceinline__ void reset() { key = least = 0; }
  // one candidate per lane (0: none)
  __device__ __forceinline__ void offer(Key cand, int k, int lane) {
    unsigned m = __ballot_sync(0xffffffffu, cand > least);
    while (m != 0) {
      const int src = __ffs(m) - 1;
      const Key c = __shfl_sync(0xffffffffu, cand, src);
      const int pos = __popc(__ballot_sync(0xffffffffu, key > c));
      const Key up = __shfl_up_sync(0xffffffffu, key, 1);
      key = lane == pos ? c : lane > pos ? up : key;
      least = __shfl_sync(0xffffffffu, key, k - 1);
      m &= m - 1;
      m &= __ballot_sync(0xffffffffu, cand > least);
    }
  }
};

// Publish the c-th of a warp's list, if it has as many.
__device__ __forceinline__ void publish(Smem& sm, const WarpTop& top, int c, int lane, int warp) {
  if (lane == c - 1 && top.key != 0) *(volatile uint32_t*)&sm.reached[warp] = (uint32_t)(top.key >> 32);
}

// The best k of the warps' lists into sm.best, in descending order; every
// thread of the block, the lists published, sm.count 0 (behind a barrier).
// What reaches the floor is gathered; a key's rank is the number of larger ones.
__device__ __forceinline__ void join_tops(Smem& sm, const WarpTop& top, int k) {
  const int tid = threadIdx.x, lane = tid & 31;
  __syncthreads();
  const float floor = floor_now(sm, lane);
  const bool in = lane < k && top.key != 0 && !(key_value(top.key) < floor);
  const unsigned m = __ballot_sync(0xffffffffu, in);
  int at = 0;
  if (lane == 0) at = atomicAdd(&sm.count, __popc(m));
  at = __shfl_sync(0xffffffffu, at, 0) + __popc(m & ((1u << lane) - 1u));
  if (in) sm.list[at] = top.key;
  __syncthreads();
  const int n = sm.count;
  if (tid < n) {
    const Key x = sm.list[tid];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += sm.list[j] > x;
    if (rank < k) sm.best[rank] = x;
  }
  __syncthreads();
}

// (loads that stay behind the wait on the kernel before, whose output the
// logits may be)
__device__ __forceinline__ uint4 load_word(const void* p) { return __ldcs(static_cast<const uint4*>(p)); }
__device__ __forceinline__ void unpack(uint4 w, float (&x)[4]) {
  x[0] = __uint_as_float(w.x);
  x[1] = __uint_as_float(w.y);
  x[2] = __uint_as_float(w.z);
  x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void unpack(uint4 w, float (&x)[8]) {
  const float2 a = bf16x2_to_f32x2(w.x), b = bf16x2_to_f32x2(w.y), c = bf16x2_to_f32x2(w.z), d = bf16x2_to_f32x2(w.w);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y; x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
}
__device__ __forceinline__ uint32_t bits_of(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }
// the larger of two or three, a NaN if one is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float load1(const float* p) { return __ldcg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(__ldcg(p)); }

// Part c of `parts` of a row: the 16-byte words [W c / parts, W (c + 1) / parts)
// of its W aligned words (the first and last may belong to it in part).  The
// thread's share of the statistics (u only with ENTROPY), its warp's best k keys
// in `top` (reset by the caller), `share` of them published in `sm`.
template <typename T, bool ENTROPY>
__device__ __forceinline__ Stat row_pass(const T* x, int vocab, int k, int share, int c, int parts, Smem& sm, WarpTop& top) {
  constexpr int kE = 16 / sizeof(T);  // elements of a 16-byte word
  constexpr int kPer = kVecs * 4;     // elements of a thread's tile: 16 either way
  static_assert(kPer == 16, "the maximum below");
  constexpr int kWords = kPer / kE;   // 16-byte words of it
  const int shift = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));  // elements before the row in its first word
  const T* base = x - shift;
  const int words = (shift + vocab + kE - 1) / kE;
  const int w0 = (int)((int64_t)words * c / parts), w1 = (int)((int64_t)words * (c + 1) / parts);
  constexpr int kTileWords = kThreads * kWords;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Stat st = {-INFINITY, 0.f, 0.f, 0};
  float least = -INFINITY;  // nothing below it is an alternative
  // a tile wholly inside the row and the part
  auto inner = [&](int t) { return t + kTileWords <= w1 && t * kE >= shift && (t + kTileWords) * kE <= shift + vocab; };
  // the words of a tile; an edge of the row, or what lies behind the part, as
  // the bits of -inf
  auto fetch = [&](int t, uint4 (&w)[kWords]) {
    if (inner(t)) {
      const T* src = base + (int64_t)(t + tid) * kE;
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = load_word(src + i * kThreads * kE);
      return;
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int at = t + tid + i * kThreads;
      const int e0 = at * kE - shift;  // index of the word's first element
      if (at < w1 && e0 >= 0 && e0 + kE <= vocab) {
        w[i] = load_word(base + (int64_t)at * kE);
      } else {
        constexpr uint32_t kNone = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
        uint32_t b[4] = {kNone, kNone, kNone, kNone};
        if (at < w1) {
#pragma unroll
          for (int j = 0; j < kE; ++j)
            if (e0 + j >= 0 && e0 + j < vocab) {
              const uint32_t v = bits_of(__ldcg(x + e0 + j));
              if (sizeof(T) == 4)
                b[j % 4] = v;
              else
                b[j / 2 % 4] = (j & 1) ? (b[j / 2 % 4] & 0xFFFFu) | (v << 16) : (b[j / 2 % 4] & 0xFFFF0000u) | v;
            }
        }
        w[i] = make_uint4(b[0], b[1], b[2], b[3]);
      }
    }
  };
  uint4 word[kWords];
  if (w0 < w1) fetch(w0, word);
  for (int t = w0; t < w1; t += kTileWords) {
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      float y[kE];
      unpack(word[i], y);
#pragma unroll
      for (int j = 0; j < kE; ++j) v[i * kE + j] = y[j];
    }
    // the next tile's loads run while this one is folded in
    if (t + kTileWords < w1) fetch(t + kTileWords, word);
    float mx[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) mx[i] = max_nan(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
    const float tm = max_nan(max_nan(mx[0], mx[1], mx[2]), mx[3], max_nan(mx[4], v[15]));
    st.bad |= !(tm < INFINITY);
    if (tm > st.m) {
      const float d = st.m == -INFINITY ? 0.f : st.m - tm, e = expf(d);
      if (ENTROPY) st.u = e > 0.f ? (st.u + d * st.z) * e : 0.f;
      st.z *= e;
      st.m = tm;
    }
    const float ref = st.m == -INFINITY ? 0.f : st.m;
    float2 z = make_float2(0.f, 0.f), u = z;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      // e^-200 is 0 in fp32: what lies lower (-inf, a mask's value) adds the same
      // nothing, but its d e would be a NaN
      float2 d = ffma2(make_float2(v[i], v[i + 1]), make_float2(1.f, 1.f), make_float2(-ref, -ref));
      if (ENTROPY) d = make_float2(fmaxf(d.x, -200.f), fmaxf(d.y, -200.f));
      const float2 x2 = ffma2(d, make_float2(1.4426950408889634f, 1.4426950408889634f), make_float2(0.f, 0.f));
      const float2 e = make_float2(ex2(x2.x), ex2(x2.y));
      z = ffma2(e, make_float2(1.f, 1.f), z);
      if (ENTROPY) u = ffma2(d, e, u);
    }
    st.z += z.x + z.y;
    if (ENTROPY) st.u += u.x + u.y;
    if (k > 0) {
      if (t == w0) {
        // (a NaN hides the thread's other logits: the floor is only lower)
        const uint32_t o = warp_kth(tm, share, lane);
        if (lane == 0) sm.reached[warp] = o;
        __syncthreads();
      }
      least = fmaxf(least, floor_now(sm, lane));
    }
    // (a NaN hides the others: then all of the tile is looked at)
    if (k > 0 && __any_sync(0xffffffffu, !(tm < least))) {
      // the lane's candidates, one a round
      uint32_t mask = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) mask |= v[i] < least ? 0u : 1u << i;
#pragma unroll 1
      while (__any_sync(0xffffffffu, mask != 0)) {
        const int bit = mask != 0 ? __ffs(mask) - 1 : 0;
        float y = v[0];
#pragma unroll
        for (int i = 1; i < kPer; ++i) y = bit == i ? v[i] : y;
        const int at = t + tid + bit / kE * kThreads, e = at * kE - shift + bit % kE;
        top.offer(mask != 0 && at < w1 && e >= 0 && e < vocab ? make_key(y, (uint32_t)e) : 0, k, lane);
        mask &= mask - 1;
      }
      // the next value above the list's last, once it is full: the tiles to
      // come have higher indices, so what equals it stays out (a row masked
      // down to fewer than k logits would offer every -inf otherwise)
      if (top.least != 0) least = fmaxf(least, value_of((uint32_t)(top.least >> 32) + 1));
      publish(sm, top, share, lane, warp);
    }
  }
  return st;
}

}  // namespace score
}  // namespace spark
