// paged_attn.cu -- attention of single new tokens over a paged cache, of chunks
// over an fp32 one, and the write of new rows into pages.
//
// a[t, h] = sum_x softmax_x(scale q[t, h] . k[x, h / 4]) v[x, h / 4] over the
// positions x the token attends to.  A group is one token's four query heads
// of one KV head: each row it reads serves all four.  The work is bound by
// the rows read from HBM; it is split evenly over the GPU whatever the
// lengths are (paged.h: tiles of 16 positions, equal shares, the last CTA of
// a split group merges the partial softmax states in CTA order), and inside a
// CTA one producer warp streams tiles through a shared-memory ring (one TMA
// box per K or V tile, the page number from the table) to four consumer warps
// holding the softmax states: the schedule and the tile of the contiguous
// cache's decode attention (attn.cu, attn_parts.cuh).
//
// Measured on the GPU (calls in a graph): 64 sequences at 512-32768 (4.92 GB of
// rows) 0.71 ms, 6.95 TB/s, 1.04 of the measured copy bandwidth; the same with
// a window of 512 (136 MB) 35 us, 3.9 TB/s, every group cut by a share's border
// and merged; 16 at 400-3000 28 us; one at 700 9.0 us with bf16 queries, 9.6
// with fp32 ones, all of it latency (share 1.6 us, first tile 1.2, one tile a
// warp 1.1, merge 2.2).
// fp32 pools run the same schedule on the CUDA cores, and chunks over them with
// a warp for each of eight tokens (k_paged_rows).
#include <math.h>

#include <type_traits>

#include "attn_parts.cuh"
#include "launch.h"
#include "paged_launch.h"
#include "paged_parts.cuh"

namespace spark {
namespace {

using paged::Args;
using paged::Cursor;
using paged::Shape;

constexpr int kTokThreads = (kConsumers + 1) * 32;
constexpr int kStages = 4;    // 16-row K + V tiles in flight per CTA
constexpr int kMinUnits = 4;  // tiles per CTA at least: one per consumer warp

template <typename CT>
struct TokSmem {
  static constexpr int kHalf = kv_half_bytes<CT>();
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kQ = kStages * kStage;
  static constexpr int kP = kQ + 4 * kQStride * 4;
  static constexpr int kM = kP + kConsumers * kTile * 16;
  static constexpr int kL = kM + kConsumers * 16;
  static constexpr int kO = kL + kConsumers * 16;
  static constexpr int kBars = kO + kConsumers * 4 * kHeadDim * 4;
  static constexpr int kFlags = kBars + 2 * kStages * 8;
  static constexpr int kPrefix = kFlags + 16;
  static constexpr int kBytes = kPrefix + 8 * (SPARK_MAX_BATCH + 2 + kTokThreads / 16);
  static constexpr int kAlloc = kBytes + 1024;  // slack to align the base to 1024 (128B swizzle)
};

// the four heads' queries of one (token, KV head), as attn_load_q lays them
// out (fp32 in 64-dim slices); consumer threads only
__device__ __forceinline__ void load_q(float* q_s, const float* qg, int tid) { attn_load_q<kConsumerThreads>(q_s, qg, tid); }
__device__ __forceinline__ void load_q(float* q_s, const __nv_bfloat16* qg, int tid) {
  const uint4 w = __ldcg(reinterpret_cast<const uint4*>(qg) + tid);  // 8 elements of 4 x 256
  const int e = 8 * tid, h = e >> 8, d = e & 255;
  float* dst = q_s + (d >> 6) * kQStride + h * 64 + (d & 63);
  const float2 a = bf16x2_to_f32x2(w.x), b = bf16x2_to_f32x2(w.y), c = bf16x2_to_f32x2(w.z), f = bf16x2_to_f32x2(w.w);
  reinterpret_cast<float4*>(dst)[0] = make_float4(a.x, a.y, b.x, b.y);
  reinterpret_cast<float4*>(dst)[1] = make_float4(c.x, c.y, f.x, f.y);
}

// The tensor-core tile's query fragments (attn_parts.cuh, MmaQ) straight from
// global memory, all loads in flight together: column g & 3 the head, hi
// halves for g < 4, lo halves after.  By way of shared memory the block's
// barrier and the bank conflicts of four heads 256 bytes apart cost 1200
// cycles more.
__device__ __forceinline__ void load_fragments(MmaQ& Q, const float* qg, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const bool lo = g >= 4;
  const float2* src = reinterpret_cast<const float2*>(qg + (g & 3) * kHeadDim + 2 * t);
  float2 x[kHeadDim / 16][2];
#pragma unroll
  for (int ks = 0; ks < kHeadDim / 16; ++ks) {
    x[ks][0] = __ldcg(src + 8 * ks);
    x[ks][1] = __ldcg(src + 8 * ks + 4);
  }
#pragma unroll
  for (int ks = 0; ks < kHeadDim / 16; ++ks)
#pragma unroll
    for (int i = 0; i < 2; ++i) Q.b[ks][i] = pack_bf16x2(split_part(x[ks][i].x, lo), split_part(x[ks][i].y, lo));
}
__device__ __forceinline__ void load_fragments(MmaQ& Q, const __nv_bfloat16* qg, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const uint32_t* src = reinterpret_cast<const uint32_t*>(qg + (g & 3) * kHeadDim + 2 * t);
#pragma unroll
  for (int ks = 0; ks < kHeadDim / 16; ++ks)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w = __ldcg(src + 8 * ks + 4 * i);
      Q.b[ks][i] = g < 4 ? w : 0u;
    }
}

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

// The group's state from the consumer warps' states in `sm`: finished if
// whole, else this CTA's partial; the last of the group's CTAs to arrive
// merges them in CTA order.  Warp h takes query head h, lane l its dims
// [8 l, 8 l + 8).  (The parts are worked out before the tiles arrive: their
// divisions took up to 2000 cycles here.)
template <typename QT>
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
    const float4* src = reinterpret_cast<const float4*>(sm.os + (w * 4 + h) * kHeadDim + 8 * lane);
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

// The producer warp: the tiles of a share, K and V of each in a stage of the
// ring, one TMA box each.
template <typename S>
__device__ __forceinline__ void fill_ring(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Args& p, const Shape& sh,
                                          Cursor& cur, int64_t u0, int64_t u1, unsigned char* base, uint64_t* full_bar,
                                          uint64_t* empty_bar, volatile int* flags) {
  const int lane = threadIdx.x & 31;
  uint32_t k = 0;
  bool ok = true;
  for (;;) {
    const int64_t t1 = cur.end < u1 ? cur.end : u1;
    for (int64_t u = cur.begin > u0 ? cur.begin : u0; u < t1; u += 32) {
      // the pages of the next 32 tiles, one per lane
      const int n = t1 - u < 32 ? (int)(t1 - u) : 32;
      const int pos = (cur.g.tile0 + (int)(u - cur.begin) + lane) * kTile;
      int z = 0;
      if (lane < n)
        z = paged::page_of(p, paged::page_entry(p, cur.s, paged::page_col(p, pos))) * p.page_size +
            paged::page_row(p, pos);
      for (int i = 0; i < n; ++i, ++k) {
        const int zi = __shfl_sync(0xffffffffu, z, i);
        if (lane == 0) {
          const int s = (int)(k % kStages);
          const uint32_t r = k / kStages;
          if (ok && r > 0 && !mbar_wait_bounded(&empty_bar[s], (r - 1) & 1, flags, kWaitLimitNs)) {
            ok = false;
            flags[0] = 1;
            atomicOr(p.err, kErrWaitTimeout);
          }
          if (ok) {
            mbar_arrive_expect_tx(&full_bar[s], S::kStage);
            unsigned char* kd = base + s * S::kStage;
            tma_load_4d(kd, &tm_k, &full_bar[s], 0, zi, 0, cur.j);
            tma_load_4d(kd + S::kHalf, &tm_v, &full_bar[s], 0, zi, 0, cur.j);
          }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        if (!ok) break;
      }
      if (!ok) break;
    }
    if (!ok || cur.end >= u1) break;
    cur.next(p, sh);
  }
  if (lane == 0 && flags[0]) {
    // let the copies in flight land before the CTA can exit
    int never = 0;
    for (uint32_t i = k > kStages ? k - kStages : 0; i < k; ++i)
      mbar_wait_bounded(&full_bar[i % kStages], (i / kStages) & 1, &never, kWaitLimitNs);
  }
}

template <typename CT, typename QT, int MINB>
__global__ void __launch_bounds__(kTokThreads, MINB)
    k_paged_token(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ Args p) {
  using S = TokSmem<CT>;
  constexpr bool kMma = std::is_same<CT, __nv_bfloat16>::value;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* q_s = reinterpret_cast<float*>(base + S::kQ);
  float4* p_s = reinterpret_cast<float4*>(base + S::kP);
  const MergeSmem msm{reinterpret_cast<float*>(base + S::kM), reinterpret_cast<float*>(base + S::kL),
                      reinterpret_cast<float*>(base + S::kO)};
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(base + S::kBars);
  uint64_t* empty_bar = full_bar + kStages;
  volatile int* flags = reinterpret_cast<volatile int*>(base + S::kFlags);  // [0] abort, [1] last
  int64_t* prefix = reinterpret_cast<int64_t*>(base + S::kPrefix);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    flags[0] = 0;
    flags[1] = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  // tables, lengths, rows and queries may come from the kernel before
  pdl_wait();
  pdl_trigger();
  const Shape sh{1, kTile, p.window};
  const int c = blockIdx.x;
  paged::Share share;
  if (!paged::find_share<kTokThreads>(p, sh, c, kMinUnits, gridDim.x, prefix, share)) return;
  const int64_t total = share.total, u0 = share.u0, u1 = share.u1;
  const int G = share.G;
  Cursor cur = share.cur;
  if (warp == kConsumers) {
    fill_ring<S>(tm_k, tm_v, p, sh, cur, u0, u1, base, full_bar, empty_bar, flags);
    return;
  }
  // ---- consumers
  uint32_t k = 0;
  AttnState st;
  MmaQ mq;
  MmaState mst;
  const QT* q = static_cast<const QT*>(p.q);
  QT* a = static_cast<QT*>(p.a);
  for (;;) {
    const int64_t t1 = cur.end < u1 ? cur.end : u1;
    const int64_t row = cur.seq.q0 + cur.g.tok;
    named_bar_sync(kBarConsumers, kConsumerThreads);  // the previous group's merge is done
    const QT* qg = q + row * p.q_ld + (int64_t)cur.j * kGroup * kHeadDim;
    if constexpr (kMma) {
      load_fragments(mq, qg, lane);
      mst.reset();
    } else {
      load_q(q_s, qg, tid);
      named_bar_sync(kBarConsumers, kConsumerThreads);
      st.reset();
    }
    const Parts parts(cur.begin, cur.end, total, G, c);
    for (int64_t u = cur.begin > u0 ? cur.begin : u0; u < t1; ++u, ++k) {
      if ((int)(k % kConsumers) != warp) continue;
      const int s = (int)(k % kStages);
      const bool ok =
          __all_sync(0xffffffffu, !flags[0] && mbar_wait_bounded(&full_bar[s], (k / kStages) & 1, flags, kWaitLimitNs));
      if (!ok) {
        if (lane == 0 && !flags[0]) {
          flags[0] = 1;
          atomicOr(p.err, kErrWaitTimeout);
        }
      } else {
        const int pos = (cur.g.tile0 + (int)(u - cur.begin)) * kTile;
        const int r0 = cur.g.lo > pos ? cur.g.lo - pos : 0;
        const int r1 = cur.g.hi + 1 - pos < kTile ? cur.g.hi + 1 - pos : kTile;
        unsigned char* kst = base + s * S::kStage;
        if constexpr (kMma)
          attn_tile_mma_rows<true>(kst, kst + S::kHalf, r0, r1, mq, reinterpret_cast<float*>(p_s + warp * kTile),
                                   p.scale_log2, mst);
        else
          attn_tile_rows<CT>(kst, kst + S::kHalf, r0, r1, q_s, p_s + warp * kTile, p.scale_log2, st);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_bar[s]);
    }
    if constexpr (kMma)
      attn_store_state_mma(mst, msm);
    else
      attn_store_state(st, msm);
    finish_group(msm, flags, p, a + (row * p.n_kv + cur.j) * kGroup * kHeadDim, parts);
    if (cur.end >= u1) break;
    cur.next(p, sh);
  }
}

template <typename CT, typename QT>
cudaError_t launch_token(const Args& p, const void* k, const void* v, cudaStream_t st) {
  using S = TokSmem<CT>;
  constexpr int kMinB = CacheT<CT>::kDeepBlocks;
  CUtensorMap mk, mv;
  const bool bf16 = std::is_same<CT, __nv_bfloat16>::value;
  const int64_t rows = (int64_t)p.n_pages * p.page_size;
  if (!make_kv_tile_map(&mk, k, bf16, p.n_kv, rows) || !make_kv_tile_map(&mv, v, bf16, p.n_kv, rows))
    return cudaErrorInvalidValue;
  auto kern = k_paged_token<CT, QT, kMinB>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kAlloc);
  if (e != cudaSuccess) return e;
  // two CTAs per SM, and no more than the tables' rows could give work to
  const int64_t parts = ((int64_t)p.max_pages * (p.page_size / kTile) + kMinUnits - 1) / kMinUnits;
  const int64_t most = (int64_t)p.n_seqs * p.n_kv * p.max_q * parts;
  int grid = kMinB * device_sm_count();
  if (grid > paged::kMaxCtas) grid = paged::kMaxCtas;
  if (grid > most) grid = (int)most;
  return launch_pdl(kern, dim3(grid), dim3(kTokThreads), S::kAlloc, st, mk, mv, p);
}

// ---------------------------------------------------------------------------
// chunks of new tokens over an fp32 pool
// ---------------------------------------------------------------------------

// Groups of eight consecutive tokens with one KV head, a consumer warp for
// each token: every tile that lands serves all of them, where a token at a
// time took each tile in for every token and was bound by that.  fp32
// arithmetic throughout, on the CUDA cores.  A token's state stays in its
// warp; a group that a share's border cuts leaves one partial per token.
// Measured, 1500 tokens at 1500, 4 KV heads: 1465 us a token at a time, 962 for
// groups of four, 754 for eight, 24.5 TFLOP/s: bound by the warps' own chains
// (a tile's dot products, their shuffles, the softmax), two warps a scheduler.
// 16 sequences of 16 tokens at 1500: 453, 321 and 256 us.
constexpr int kRowTokens = 8;
constexpr int kRowThreads = (kRowTokens + 1) * 32;
struct RowsSmem {
  static constexpr int kHalf = kv_half_bytes<float>();
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kQ = kStages * kStage;
  static constexpr int kQToken = 4 * kQStride * 4;
  static constexpr int kP = kQ + kRowTokens * kQToken;
  static constexpr int kBars = kP + kRowTokens * kTile * 16;
  static constexpr int kFlags = kBars + 2 * kStages * 8;
  static constexpr int kPrefix = kFlags + 16;
  static constexpr int kBytes = kPrefix + 8 * (SPARK_MAX_BATCH + 2 + kRowThreads / 16);
  static constexpr int kAlloc = kBytes + 1024;  // slack to align the base to 1024 (128B swizzle)
};
static_assert(sizeof(float) * 2 * paged::kMaxCtas * kRowTokens * kPartFloats <= paged::kPartBytes, "a partial per token");

// a token's four heads' queries by its warp, as attn_load_q lays them out
__device__ __forceinline__ void load_token(float* q_s, const float* qg, int lane) {
  float4 v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = __ldcg(reinterpret_cast<const float4*>(qg) + lane + 32 * k);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int e = 4 * (lane + 32 * k), h = e >> 8, d = e & 255;
    *reinterpret_cast<float4*>(q_s + (d >> 6) * kQStride + h * 64 + (d & 63)) = v[k];
  }
}
__device__ __forceinline__ void load_token(float* q_s, const __nv_bfloat16* qg, int lane) {
  uint2 v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = __ldcg(reinterpret_cast<const uint2*>(qg) + lane + 32 * k);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int e = 4 * (lane + 32 * k), h = e >> 8, d = e & 255;
    const float2 a = bf16x2_to_f32x2(v[k].x), b = bf16x2_to_f32x2(v[k].y);
    *reinterpret_cast<float4*>(q_s + (d >> 6) * kQStride + h * 64 + (d & 63)) = make_float4(a.x, a.y, b.x, b.y);
  }
}

template <typename QT>
__global__ void __launch_bounds__(kRowThreads, 1)
    k_paged_rows(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ Args p) {
  using S = RowsSmem;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(base + S::kBars);
  uint64_t* empty_bar = full_bar + kStages;
  volatile int* flags = reinterpret_cast<volatile int*>(base + S::kFlags);  // [0] abort, [1] last
  int64_t* prefix = reinterpret_cast<int64_t*>(base + S::kPrefix);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], kRowTokens);
    }
    flags[0] = 0;
    flags[1] = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  // tables, lengths, rows and queries may come from the kernel before
  pdl_wait();
  pdl_trigger();
  const Shape sh{kRowTokens, kTile, p.window};
  const int c = blockIdx.x;
  paged::Share share;
  if (!paged::find_share<kRowThreads>(p, sh, c, kMinUnits, gridDim.x, prefix, share)) return;
  const int64_t total = share.total, u0 = share.u0, u1 = share.u1;
  const int G = share.G;
  Cursor cur = share.cur;
  if (warp == kRowTokens) {
    fill_ring<S>(tm_k, tm_v, p, sh, cur, u0, u1, base, full_bar, empty_bar, flags);
    return;
  }
  // ---- consumers: warp w has the group's token w
  float* q_s = reinterpret_cast<float*>(base + S::kQ + warp * S::kQToken);
  float4* p_s = reinterpret_cast<float4*>(base + S::kP) + warp * kTile;
  const QT* q = static_cast<const QT*>(p.q);
  QT* a = static_cast<QT*>(p.a);
  uint32_t k = 0;
  AttnState st;
  for (;;) {
    const int64_t t1 = cur.end < u1 ? cur.end : u1;
    const bool mine = warp < cur.g.n_tok;
    const int64_t row = cur.seq.q0 + cur.g.tok + warp;
    // positions the token sees
    const int hi = cur.seq.p0 + cur.g.tok + warp, lo = p.window > 0 && hi + 1 > p.window ? hi + 1 - p.window : 0;
    if (mine) load_token(q_s, q + row * p.q_ld + (int64_t)cur.j * kGroup * kHeadDim, lane);
    __syncwarp();
    st.reset();
    const Parts parts(cur.begin, cur.end, total, G, c);
    for (int64_t u = cur.begin > u0 ? cur.begin : u0; u < t1; ++u, ++k) {
      const int s = (int)(k % kStages);
      const bool ok =
          __all_sync(0xffffffffu, !flags[0] && mbar_wait_bounded(&full_bar[s], (k / kStages) & 1, flags, kWaitLimitNs));
      if (!ok) {
        if (lane == 0 && !flags[0]) {
          flags[0] = 1;
          atomicOr(p.err, kErrWaitTimeout);
        }
      } else if (mine) {
        const int pos = (cur.g.tile0 + (int)(u - cur.begin)) * kTile;
        const int r0 = lo > pos ? lo - pos : 0, r1 = hi + 1 - pos < kTile ? hi + 1 - pos : kTile;
        unsigned char* kst = base + s * S::kStage;
        if (r0 < r1) attn_tile_rows<float>(kst, kst + S::kHalf, r0, r1, q_s, p_s, p.scale_log2, st);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_bar[s]);
    }
    QT* dst = a + (row * p.n_kv + cur.j) * (kGroup * kHeadDim) + 8 * lane;
    float O[4][8], L[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      L[h] = warp_sum(st.l[h]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        O[h][2 * i] = st.o[h][i].x;
        O[h][2 * i + 1] = st.o[h][i].y;
      }
    }
    if (parts.first == parts.last) {
      if (mine && !flags[0])
#pragma unroll
        for (int h = 0; h < 4; ++h) store8(dst + h * kHeadDim, O[h], 1.0f / L[h]);
    } else {
      float* P = p.part + ((int64_t)parts.slot * kRowTokens + warp) * kPartFloats;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        store8(P + 8 + h * kHeadDim + 8 * lane, O[h], 1.0f);
        if (lane == 0) {
          P[h] = st.m[h];
          P[4 + h] = L[h];
        }
      }
      named_bar_sync(kBarMerge, 32 * kRowTokens);
      if (tid == 0) {
        __threadfence();  // the block's partials, ordered before this thread by the barrier, before the ticket
        const int last = atomicAdd(&p.tickets[parts.first], 1u) == (uint32_t)(parts.last - parts.first);
        if (last) p.tickets[parts.first] = 0;  // every arrival counts: back at zero
        flags[1] = last && !flags[0];
        if (last) __threadfence();  // the ticket before the others' partials
      }
      named_bar_sync(kBarMerge, 32 * kRowTokens);
      if (flags[1] && mine) {
        // the parts in CTA order, a head at a time
#pragma unroll 1
        for (int h = 0; h < 4; ++h) {
          constexpr int kBatch = 4;  // loaded per round trip
          float M = -INFINITY, sum = 0.f, o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = 0.f;
          for (int q0 = parts.first; q0 <= parts.last; q0 += kBatch) {
            float m[kBatch], l[kBatch];
            float4 x[kBatch], y[kBatch];
#pragma unroll
            for (int t = 0; t < kBatch; ++t) {
              // (behind the last part the last once more, at weight 0)
              const int r = min(q0 + t, parts.last);
              const float* Pr = p.part + ((int64_t)(r == parts.first ? parts.slot0 : 2 * r) * kRowTokens + warp) * kPartFloats;
              m[t] = __ldcg(Pr + h);
              l[t] = __ldcg(Pr + 4 + h);
              x[t] = __ldcg(reinterpret_cast<const float4*>(Pr + 8 + h * kHeadDim + 8 * lane));
              y[t] = __ldcg(reinterpret_cast<const float4*>(Pr + 8 + h * kHeadDim + 8 * lane + 4));
              if (q0 + t > parts.last) m[t] = -INFINITY;
            }
#pragma unroll
            for (int t = 0; t < kBatch; ++t) {
              const float mn = fmaxf(M, m[t]);
              // (a part in which the token saw nothing holds no state)
              const float e0 = M == -INFINITY ? 0.f : exp2f(M - mn), e1 = m[t] == -INFINITY ? 0.f : exp2f(m[t] - mn);
              M = mn;
              sum = sum * e0 + l[t] * e1;
              o[0] = o[0] * e0 + x[t].x * e1; o[1] = o[1] * e0 + x[t].y * e1;
              o[2] = o[2] * e0 + x[t].z * e1; o[3] = o[3] * e0 + x[t].w * e1;
              o[4] = o[4] * e0 + y[t].x * e1; o[5] = o[5] * e0 + y[t].y * e1;
              o[6] = o[6] * e0 + y[t].z * e1; o[7] = o[7] * e0 + y[t].w * e1;
            }
          }
          store8(dst + h * kHeadDim, o, 1.0f / sum);
        }
      }
    }
    if (cur.end >= u1) break;
    cur.next(p, sh);
  }
}

template <typename QT>
cudaError_t launch_rows(const Args& p, const void* k, const void* v, cudaStream_t st) {
  using S = RowsSmem;
  CUtensorMap mk, mv;
  const int64_t rows = (int64_t)p.n_pages * p.page_size;
  if (!make_kv_tile_map(&mk, k, false, p.n_kv, rows) || !make_kv_tile_map(&mv, v, false, p.n_kv, rows))
    return cudaErrorInvalidValue;
  auto kern = k_paged_rows<QT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kAlloc);
  if (e != cudaSuccess) return e;
  int grid = device_sm_count();
  if (grid > paged::kMaxCtas) grid = paged::kMaxCtas;
  return launch_pdl(kern, dim3(grid), dim3(kRowThreads), S::kAlloc, st, mk, mv, p);
}

// ---------------------------------------------------------------------------
// the write of new rows
// ---------------------------------------------------------------------------

// four elements in the pool's type, rounded once
__device__ __forceinline__ float4 load4(const float* p) { return __ldcg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = __ldcg(reinterpret_cast<const uint2*>(p));
  const float2 a = bf16x2_to_f32x2(w.x), b = bf16x2_to_f32x2(w.y);
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// A CTA takes up to kAppendTokens consecutive tokens: their page rows first,
// one thread each (a binary search in q_start, then the table), then the
// rows' words four at a time per thread, whatever rows they are of.  Bound by
// the rows' bytes where there are many (8370 tokens, 103 MB: 16.5 to 19 us, 5.4
// to 6.2 TB/s; one CTA per token took 80 us, its dependent loads exposed), by
// the chain of dependent loads where there are few (64 tokens: 3.2 us).
constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 16;
constexpr int kAppendUnroll = 4;

template <typename XT, typename CT>
__global__ void __launch_bounds__(kAppendThreads)
    k_paged_append(const XT* k, const XT* v, int64_t ld, CT* pk, CT* pv, int per, const __grid_constant__ Args p) {
  __shared__ int64_t to[kAppendTokens];
  pdl_wait();
  // no early trigger: a kernel that reads pages before its own wait must not
  // start before these rows are written
  const int t0 = blockIdx.x * per;
  const int row4 = p.n_kv * kHeadDim / 4;  // words of four elements in a row
  if (threadIdx.x < per) {
    const int t = t0 + threadIdx.x;
    int64_t at = -1;
    if (t < p.n_tokens) {
      int lo = 0, hi = p.n_seqs - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldcg(p.q_start + mid) <= t) lo = mid; else hi = mid - 1;
      }
      const paged::Seq s = paged::load_seq(p, lo);
      if (t >= s.q0 && t < s.q0 + s.n) {  // else: behind the last sequence, or a sequence that makes no sense
        const int pos = s.p0 + (t - s.q0);
        const int pg = paged::page_entry(p, lo, paged::page_col(p, pos));
        if (pg >= 0 && pg < p.n_pages)
          at = ((int64_t)pg * p.page_size + paged::page_row(p, pos)) * row4;
        else
          atomicOr(p.err, kErrIndex);
      }
    }
    to[threadIdx.x] = at;
  }
  // every sequence is looked at, also one that no token's search ends in, by
  // the threads that have no token first
  for (int s = blockIdx.x * kAppendThreads + kAppendThreads - 1 - (int)threadIdx.x; s < p.n_seqs;
       s += gridDim.x * kAppendThreads)
    if (paged::load_seq(p, s).bad) atomicOr(p.err, kErrIndex);
  __syncthreads();
  const int words = per * row4;
  for (int w0 = threadIdx.x; w0 < words; w0 += kAppendThreads * kAppendUnroll) {
    float4 x[kAppendUnroll], y[kAppendUnroll];
    int64_t dst[kAppendUnroll];
#pragma unroll
    for (int i = 0; i < kAppendUnroll; ++i) {
      const int w = w0 + i * kAppendThreads;
      const int t = w < words ? w / row4 : 0, e = w - t * row4;
      dst[i] = w < words && to[t] >= 0 ? to[t] + e : -1;
      if (dst[i] >= 0) {
        const int64_t src = (int64_t)(t0 + t) * ld + 4 * e;
        x[i] = load4(k + src);
        y[i] = load4(v + src);
      }
    }
#pragma unroll
    for (int i = 0; i < kAppendUnroll; ++i)
      if (dst[i] >= 0) {
        store4(pk + 4 * dst[i], x[i]);
        store4(pv + 4 * dst[i], y[i]);
      }
  }
}

template <typename XT, typename CT>
cudaError_t launch_append_t(const Args& p, const void* k, const void* v, int64_t ld, void* pk, void* pv,
                            cudaStream_t st) {
  // one token per CTA until the CTAs that run at once (eight an SM) have one each
  const int at_once = 8 * device_sm_count();
  int per = (p.n_tokens + at_once - 1) / at_once;
  if (per > kAppendTokens) per = kAppendTokens;
  return launch_pdl(k_paged_append<XT, CT>, dim3((p.n_tokens + per - 1) / per), dim3(kAppendThreads), 0, st,
                    static_cast<const XT*>(k), static_cast<const XT*>(v), ld, static_cast<CT*>(pk),
                    static_cast<CT*>(pv), per, p);
}

// single tokens (max_q 1)
cudaError_t launch_tokens(const paged::Args& p, int qdtype, int cdtype, const void* k, const void* v,
                          cudaStream_t st) {
  if (cdtype == SPARK_BF16)
    return qdtype == SPARK_BF16 ? launch_token<__nv_bfloat16, __nv_bfloat16>(p, k, v, st)
                                : launch_token<__nv_bfloat16, float>(p, k, v, st);
  return qdtype == SPARK_BF16 ? launch_token<float, __nv_bfloat16>(p, k, v, st)
                              : launch_token<float, float>(p, k, v, st);
}

}  // namespace

cudaError_t launch_paged_attention(const paged::Args& p, int qdtype, int cdtype, const void* k, const void* v,
                                   cudaStream_t st) {
  if (p.max_q == 1) return launch_tokens(p, qdtype, cdtype, k, v, st);
  if (cdtype != SPARK_BF16)
    return qdtype == SPARK_BF16 ? launch_rows<__nv_bfloat16>(p, k, v, st) : launch_rows<float>(p, k, v, st);
  if (p.max_q <= paged::kChunkTokens) return launch_paged_chunk(p, qdtype, k, v, st);
  // Longer chunks take pairs of CTAs, which read 64 tokens' rows once: where
  // most sequences are long (the average above half of the longest: 32 of 33
  // tokens at 4096-8192, bf16 queries, 166 us against 261 on single CTAs), or
  // where the long ones are most of the work (above 128 tokens a sequence on
  // average: 16 sequences, 3 of them with chunks of ~3000 tokens, 402 against
  // 446 us).  In other batches the short sequences would leave most of a
  // pair's rows empty, and single CTAs take them all (32 sequences, 4 of them
  // with chunks of ~400 tokens: 107 against 118 us; fp32 queries 132 against
  // 172).  Each kind on the kernel that suits it, one after the other, was
  // slower than either: the two kernels' starts and ends add up.
  const int64_t T = p.n_tokens, S = p.n_seqs;
  if (2 * T > S * p.max_q || T > 128 * S) return launch_paged_pair(p, qdtype, k, v, st);
  return launch_paged_chunk(p, qdtype, k, v, st);
}

cudaError_t launch_paged_append(const paged::Args& p, int xdtype, int cdtype, const void* k, const void* v, int64_t ld,
                                void* pk, void* pv, cudaStream_t st) {
  if (cdtype == SPARK_BF16)
    return xdtype == SPARK_BF16 ? launch_append_t<__nv_bfloat16, __nv_bfloat16>(p, k, v, ld, pk, pv, st)
                                : launch_append_t<float, __nv_bfloat16>(p, k, v, ld, pk, pv, st);
  return xdtype == SPARK_BF16 ? launch_append_t<__nv_bfloat16, float>(p, k, v, ld, pk, pv, st)
                              : launch_append_t<float, float>(p, k, v, ld, pk, pv, st);
}

}  // namespace spark
