// paged4_attn.cu -- attention of single new tokens over pages held in 4 bits.
//
// The schedule is that of paged_attn.cu: a group is one token's four query
// heads of one KV head, the work list of 16-position tiles is split evenly
// over the CTAs, the last CTA of a split group merges its partial states.  A
// tile of one head is one block of K and one of V (fp4.cuh), 2304 contiguous
// bytes each: a plain bulk copy, no tensor map.
//
// A warp folds a block by itself, codes to fp16 in registers, straight into
// the fragments of mma.m16n8k16 (fp16 in, fp32 sums):
//   s = K q^T      A = K (16 positions x 16 dims), B = [q_hi | q_lo]^T, the four
//                  heads' queries as two fp16 halves
//   o^T += V^T p^T A = V^T (16 dims x 16 positions), B = [p_hi | p_lo]^T
// An element code * scale has at most 6 significant bits: its fp16 product is
// exact.  A contraction may take its K dimension, and an output its M one, in
// any order, so that each lane's share of a row is contiguous: of K the 64 dims
// from 64 t of positions g and g + 8, of V the 32 dims from 32 g of positions 4
// t .. 4 t + 3 (lane 4 g + t), eight 16-byte reads a block in all.  Two rows of
// V make pairs along the positions by exchanging halves of their bytes, before
// the conversion: four operations for 16 elements.
//
// Queries are scaled by a power of two into fp16's range; scores take it back
// in fp32.  The running maximum is raised once a score passes it by 2^8 (as in
// the chunk kernels): most tiles cost one vote for it.
#include <math.h>

#include <type_traits>

#include "attn_parts.cuh"
#include "fp4.cuh"
#include "launch.h"
#include "paged_launch.h"
#include "paged_parts.cuh"
#include "paged_token_parts.cuh"

namespace spark {
namespace {

using namespace token;
using paged::Cursor;
using paged::Shape;

constexpr int kThreads4 = (kConsumers + 1) * 32;
constexpr int kBlocks4 = 2;      // CTAs per SM
constexpr int kStages4 = 16;     // tiles in flight per CTA
constexpr int kMinUnits4 = 4;    // tiles per CTA at least: one per consumer warp
constexpr int kPad = 4;          // floats behind each 32 of a state in shared memory
constexpr int kPRow = 20;        // floats of a head's probabilities of a tile (16, and a shift of banks)
constexpr float kRaise4 = 8.0f;
static_assert(kStages4 % kConsumers == 0, "a stage serves one warp: no wait aliases an older phase");

struct Smem4 {
  static constexpr int kStage = 2 * fp4::kBlock;
  static constexpr int kP = kStages4 * kStage;
  static constexpr int kM = kP + kConsumers * 4 * kPRow * 4;
  static constexpr int kL = kM + kConsumers * 16;
  static constexpr int kO = kL + kConsumers * 16;
  static constexpr int kBars = kO + kConsumers * 4 * kStateFloats<kPad> * 4;
  static constexpr int kFlags = kBars + 2 * kStages4 * 8;
  static constexpr int kPrefix = kFlags + 16;
  static constexpr int kBytes = kPrefix + 8 * (SPARK_MAX_BATCH + 2 + kThreads4 / 16);
};

// the queries of a KV head as the B fragments of all 16-dim steps: step s holds
// dims 64 t + 4 s .. + 3, column g head g & 3, its high half for g < 4
struct Queries {
  uint32_t b[kHeadDim / 16][2];
  float scale[2];  // of the scores of heads 2 (t & 1) + j
};

__device__ __forceinline__ void load64(float (&x)[64], const float* q) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(q) + i);
    x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
  }
}
__device__ __forceinline__ void load64(float (&x)[64], const __nv_bfloat16* q) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(q) + i);
    const float2 a = bf16x2_to_f32x2(v.x), b = bf16x2_to_f32x2(v.y), c = bf16x2_to_f32x2(v.z), d = bf16x2_to_f32x2(v.w);
    x[8 * i] = a.x; x[8 * i + 1] = a.y; x[8 * i + 2] = b.x; x[8 * i + 3] = b.y;
    x[8 * i + 4] = c.x; x[8 * i + 5] = c.y; x[8 * i + 6] = d.x; x[8 * i + 7] = d.y;
  }
}

template <typename QT>
__device__ __forceinline__ void load_queries(Queries& Q, const QT* qg, float scale_log2, int lane) {
  const int g = lane >> 2, t = lane & 3;
  float x[64];
  load64(x, qg + (g & 3) * kHeadDim + 64 * t);
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 64; ++i) m = fmaxf(m, fabsf(x[i]));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const float2 unit = fp4::unit_of(m);
#pragma unroll
  for (int s = 0; s < kHeadDim / 16; ++s)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      Q.b[s][i] = fp4::pack(fp4::split_part(x[4 * s + 2 * i] * unit.x, g >= 4),
                            fp4::split_part(x[4 * s + 2 * i + 1] * unit.x, g >= 4));
#pragma unroll
  for (int j = 0; j < 2; ++j) Q.scale[j] = scale_log2 * __shfl_sync(0xffffffffu, unit.y, 4 * (2 * (t & 1) + j));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte `i` of a word of scales as an fp16 pair of it.
__device__ __forceinline__ uint32_t scale2(uint32_t w, int i) { return __byte_perm(w, 0u, 0x4040u | (uint32_t)(i | (i << 8))) << 7; }

// One warp folds rows [r0, r1) of a block of K and V into its state (o[i]: dims
// 32 g + 2 i in [0], [1], the next in [2], [3], columns 2 t and 2 t + 1; l: this
// lane's rows only).  p_w: the warp's 4 x kPRow probability scratch.
__device__ __forceinline__ void fold_block(const unsigned char* kst, const unsigned char* vst, int r0, int r1,
                                           const Queries& Q, float* p_w, MmaState& st) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const bool whole = r0 == 0 && r1 == fp4::kRows;
  // s = K q^T, even and odd steps in two chains
  float c[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};
  {
    const uint32_t sa = *reinterpret_cast<const uint32_t*>(kst + fp4::scale_at(g, 64 * t));
    const uint32_t sb = *reinterpret_cast<const uint32_t*>(kst + fp4::scale_at(g + 8, 64 * t));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 ka = *reinterpret_cast<const uint4*>(kst + fp4::code_at(g, 64 * t + 32 * i));
      const uint4 kb = *reinterpret_cast<const uint4*>(kst + fp4::code_at(g + 8, 64 * t + 32 * i));
      const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t fa = scale2(sa, 2 * i + (w >> 1)), fb = scale2(sb, 2 * i + (w >> 1));
        uint32_t ha[4], hb[4];
        fp4::halves8(wa[w], ha);
        fp4::halves8(wb[w], hb);
        const uint32_t a0[4] = {fp4::mul2(ha[0], fa), fp4::mul2(hb[0], fb), fp4::mul2(ha[1], fa), fp4::mul2(hb[1], fb)};
        const uint32_t a1[4] = {fp4::mul2(ha[2], fa), fp4::mul2(hb[2], fb), fp4::mul2(ha[3], fa), fp4::mul2(hb[3], fb)};
        const int s = 8 * i + 2 * w;
        mma_f16(c, a0, Q.b[s][0], Q.b[s][1]);
        mma_f16(c2, a1, Q.b[s + 1][0], Q.b[s + 1][1]);
      }
    }
  }
  // hi and lo columns, scale, mask: sc[r][j] = row g + 8 r, head 2 (t & 1) + j
  float sc[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] += c2[i];
    c[i] += __shfl_xor_sync(0xffffffffu, c[i], 2);
    sc[i >> 1][i & 1] = c[i] * Q.scale[i & 1];
  }
  if (!whole) {
    if (g < r0 || g >= r1) sc[0][0] = sc[0][1] = -INFINITY;
    if (g + 8 < r0 || g + 8 >= r1) sc[1][0] = sc[1][1] = -INFINITY;
  }
  const float m0 = fmaxf(sc[0][0], sc[1][0]), m1 = fmaxf(sc[0][1], sc[1][1]);
  if (__any_sync(0xffffffffu, m0 > st.m[0] + kRaise4 || m1 > st.m[1] + kRaise4)) {
    float mx[2] = {m0, m1}, corr[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 4));
      mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 8));
      mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 16));
      const float mn = fmaxf(st.m[j], mx[j]);
      corr[j] = st.m[j] == -INFINITY ? 0.f : exp2f(st.m[j] - mn);
      st.m[j] = mn;
      st.l[j] *= corr[j];
    }
#pragma unroll
    for (int i = 0; i < kHeadDim / 16; ++i) {
      st.o[i][0] *= corr[0];
      st.o[i][1] *= corr[1];
      st.o[i][2] *= corr[0];
      st.o[i][3] *= corr[1];
    }
  }
  // (a row that is masked, or a maximum of -inf under it, is a probability of 0)
  float pr[2][2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float ref = st.m[j] == -INFINITY ? 0.f : st.m[j];
    pr[0][j] = ex2(sc[0][j] - ref);
    pr[1][j] = ex2(sc[1][j] - ref);
    st.l[j] += pr[0][j] + pr[1][j];
  }
  __syncwarp();
  if (t < 2) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      p_w[(2 * t + j) * kPRow + g] = pr[0][j];
      p_w[(2 * t + j) * kPRow + g + 8] = pr[1][j];
    }
  }
  __syncwarp();
  // B fragments of [p_hi | p_lo]^T: the MMA's steps 2 t, 2 t + 1, 2 t + 8, 2 t +
  // 9 are positions 4 t .. 4 t + 3
  const float4 p4 = *reinterpret_cast<const float4*>(p_w + (g & 3) * kPRow + 4 * t);
  const uint32_t pb0 = fp4::pack(fp4::split_part(p4.x, g >= 4), fp4::split_part(p4.y, g >= 4));
  const uint32_t pb1 = fp4::pack(fp4::split_part(p4.z, g >= 4), fp4::split_part(p4.w, g >= 4));
  // o^T += V^T p^T
  uint32_t v[4][4], f01[2], f23[2];
  {
    uint32_t s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 4 * t + j;
      const uint4 x = *reinterpret_cast<const uint4*>(vst + fp4::code_at(row, 32 * g));
      v[j][0] = x.x; v[j][1] = x.y; v[j][2] = x.z; v[j][3] = x.w;
      s[j] = *reinterpret_cast<const uint16_t*>(vst + fp4::scale_at(row, 32 * g));
      // (0 times whatever a row outside holds, a NaN's scale included)
      if (!whole && (row < r0 || row >= r1)) s[j] = 0;
    }
    const uint32_t s01 = s[0] | (s[1] << 16), s23 = s[2] | (s[3] << 16);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f01[u] = ((s01 >> (8 * u)) & 0x00FF00FFu) << 7;
      f23[u] = ((s23 >> (8 * u)) & 0x00FF00FFu) << 7;
    }
  }
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    // bytes of one dim of two rows: even dims, odd dims
    constexpr uint32_t kLow = 0x0F0F0F0Fu;
    uint32_t e01[4], d01[4], e23[4], d23[4];
    fp4::halves8((v[0][w] & kLow) | ((v[1][w] << 4) & ~kLow), e01);
    fp4::halves8(((v[0][w] >> 4) & kLow) | (v[1][w] & ~kLow), d01);
    fp4::halves8((v[2][w] & kLow) | ((v[3][w] << 4) & ~kLow), e23);
    fp4::halves8(((v[2][w] >> 4) & kLow) | (v[3][w] & ~kLow), d23);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t a[4] = {fp4::mul2(e01[b], f01[w >> 1]), fp4::mul2(d01[b], f01[w >> 1]),
                             fp4::mul2(e23[b], f23[w >> 1]), fp4::mul2(d23[b], f23[w >> 1])};
      mma_f16(st.o[4 * w + b], a, pb0, pb1);
    }
  }
}

// Put one warp's state into the merge scratch: the hi and lo columns and the
// lanes' sums added.
__device__ __forceinline__ void store_state4(MmaState& st, const MergeSmem& sm) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < kHeadDim / 16; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) st.o[i][k] += __shfl_xor_sync(0xffffffffu, st.o[i][k], 2);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    st.l[j] += __shfl_xor_sync(0xffffffffu, st.l[j], 4);
    st.l[j] += __shfl_xor_sync(0xffffffffu, st.l[j], 8);
    st.l[j] += __shfl_xor_sync(0xffffffffu, st.l[j], 16);
  }
  if (t < 2) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int h = 2 * t + j;
      float* os = sm.os + (warp * 4 + h) * kStateFloats<kPad> + state_at<kPad>(32 * g);
#pragma unroll
      for (int i = 0; i < kHeadDim / 16; i += 2)
        *reinterpret_cast<float4*>(os + 2 * i) = make_float4(st.o[i][j], st.o[i][2 + j], st.o[i + 1][j], st.o[i + 1][2 + j]);
      if (g == 0) {
        sm.ms[warp * 4 + h] = st.m[j];
        sm.ls[warp * 4 + h] = st.l[j];
      }
    }
  }
}

template <typename QT>
__global__ void __launch_bounds__(kThreads4, kBlocks4)
    k_paged4_token(const unsigned char* pk, const unsigned char* pv, const __grid_constant__ Args p) {
  using S = Smem4;
  extern __shared__ __align__(128) unsigned char base[];
  float* p_s = reinterpret_cast<float*>(base + S::kP);
  const MergeSmem msm{reinterpret_cast<float*>(base + S::kM), reinterpret_cast<float*>(base + S::kL),
                      reinterpret_cast<float*>(base + S::kO)};
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(base + S::kBars);
  uint64_t* empty_bar = full_bar + kStages4;
  volatile int* flags = reinterpret_cast<volatile int*>(base + S::kFlags);  // [0] abort, [1] last
  int64_t* prefix = reinterpret_cast<int64_t*>(base + S::kPrefix);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages4; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    flags[0] = 0;
    flags[1] = 0;
    fence_mbar_init();
  }
  // tables, lengths, rows and queries may come from the kernel before
  pdl_wait();
  pdl_trigger();
  const Shape sh{1, kTile, p.window};
  const int c = blockIdx.x;
  paged::Share share;
  if (!paged::find_share<kThreads4>(p, sh, c, kMinUnits4, gridDim.x, prefix, share)) return;
  const int64_t total = share.total, u0 = share.u0, u1 = share.u1;
  const int G = share.G;
  Cursor cur = share.cur;
  if (warp == kConsumers) {
    // ---- the producer: the tiles of the share, a stage of the ring each
    uint32_t k = 0;
    bool ok = true;
    for (;;) {
      const int64_t t1 = cur.end < u1 ? cur.end : u1;
      for (int64_t u = cur.begin > u0 ? cur.begin : u0; ok && u < t1; u += 32) {
        // the blocks of the next 32 tiles, one per lane
        const int n = t1 - u < 32 ? (int)(t1 - u) : 32;
        const int pos = (cur.g.tile0 + (int)(u - cur.begin) + lane) * kTile;
        int64_t at = 0;
        if (lane < n)
          at = fp4::block_at(paged::page_of(p, paged::page_entry(p, cur.s, paged::page_col(p, pos))),
                             paged::page_row(p, pos), cur.j, p.page_size, p.n_kv);
        for (int i = 0; i < n; ++i, ++k) {
          const int64_t from = __shfl_sync(0xffffffffu, at, i);
          if (lane == 0) {
            const int s = (int)(k % kStages4);
            const uint32_t r = k / kStages4;
            if (r > 0 && !mbar_wait_bounded(&empty_bar[s], (r - 1) & 1, flags, kWaitLimitNs)) {
              ok = false;
              flags[0] = 1;
              atomicOr(p.err, kErrWaitTimeout);
            }
            if (ok) {
              mbar_arrive_expect_tx(&full_bar[s], S::kStage);
              bulk_load(base + s * S::kStage, pk + from, fp4::kBlock, &full_bar[s]);
              bulk_load(base + s * S::kStage + fp4::kBlock, pv + from, fp4::kBlock, &full_bar[s]);
            }
          }
          ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
          if (!ok) break;
        }
      }
      if (!ok || cur.end >= u1) break;
      cur.next(p, sh);
    }
    if (lane == 0 && flags[0]) {
      // let the copies in flight land before the CTA can exit
      int never = 0;
      for (uint32_t i = k > kStages4 ? k - kStages4 : 0; i < k; ++i)
        mbar_wait_bounded(&full_bar[i % kStages4], (i / kStages4) & 1, &never, kWaitLimitNs);
    }
    return;
  }
  // ---- consumers
  uint32_t k = 0;
  Queries Q;
  MmaState st;
  const QT* q = static_cast<const QT*>(p.q);
  QT* a = static_cast<QT*>(p.a);
  for (;;) {
    const int64_t t1 = cur.end < u1 ? cur.end : u1;
    const int64_t row = cur.seq.q0 + cur.g.tok;
    named_bar_sync(kBarConsumers, kConsumerThreads);  // the previous group's merge is done
    load_queries(Q, q + row * p.q_ld + (int64_t)cur.j * kGroup * kHeadDim, p.scale_log2, lane);
    st.reset();
    const Parts parts(cur.begin, cur.end, total, G, c);
    for (int64_t u = cur.begin > u0 ? cur.begin : u0; u < t1; ++u, ++k) {
      if ((int)(k % kConsumers) != warp) continue;
      const int s = (int)(k % kStages4);
      const bool ok =
          __all_sync(0xffffffffu, !flags[0] && mbar_wait_bounded(&full_bar[s], (k / kStages4) & 1, flags, kWaitLimitNs));
      if (!ok) {
        if (lane == 0 && !flags[0]) {
          flags[0] = 1;
          atomicOr(p.err, kErrWaitTimeout);
        }
      } else {
        const int pos = (cur.g.tile0 + (int)(u - cur.begin)) * kTile;
        const int r0 = cur.g.lo > pos ? cur.g.lo - pos : 0;
        const int r1 = cur.g.hi + 1 - pos < kTile ? cur.g.hi + 1 - pos : kTile;
        const unsigned char* kst = base + s * S::kStage;
        fold_block(kst, kst + fp4::kBlock, r0, r1, Q, p_s + warp * 4 * kPRow, st);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_bar[s]);
    }
    store_state4(st, msm);
    finish_group<QT, kPad>(msm, flags, p, a + (row * p.n_kv + cur.j) * kGroup * kHeadDim, parts);
    if (cur.end >= u1) break;
    cur.next(p, sh);
  }
}

template <typename QT>
cudaError_t launch_token4(const Args& p, const void* k, const void* v, cudaStream_t st) {
  auto kern = k_paged4_token<QT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem4::kBytes);
  if (e != cudaSuccess) return e;
  // no more CTAs than the tables' rows could give work to
  const int64_t parts = ((int64_t)p.max_pages * (p.page_size / kTile) + kMinUnits4 - 1) / kMinUnits4;
  const int64_t most = (int64_t)p.n_seqs * p.n_kv * p.max_q * parts;
  int grid = kBlocks4 * device_sm_count();
  if (grid > paged::kMaxCtas) grid = paged::kMaxCtas;
  if (grid > most) grid = (int)most;
  return launch_pdl(kern, dim3(grid), dim3(kThreads4), Smem4::kBytes, st, static_cast<const unsigned char*>(k),
                    static_cast<const unsigned char*>(v), p);
}

}  // namespace

cudaError_t launch_paged4_attention(const paged::Args& p, int qdtype, const void* k, const void* v, cudaStream_t st) {
  if (p.max_q > paged::kChunkTokens && (2 * (int64_t)p.n_tokens > (int64_t)p.n_seqs * p.max_q || p.n_tokens > 128 * p.n_seqs))
    return launch_paged4_pair(p, qdtype, k, v, st);
  if (p.max_q > 1) return launch_paged4_chunk(p, qdtype, k, v, st);
  return qdtype == SPARK_BF16 ? launch_token4<__nv_bfloat16>(p, k, v, st) : launch_token4<float>(p, k, v, st);
}

}  // namespace spark
