// paged4_attn.cu -- attention of single new tokens over pages held in 4 bits.
//
// A group is one token's four query heads of one KV head, as in paged_attn.cu:
// the work list of tiles (32 positions here: two blocks of K, two of V) is split
// evenly over the CTAs, the last CTA of a split group merges its partial states.
// A block (fp4.cuh) is 2304 contiguous bytes: a plain bulk copy, no tensor map.
//
// A warp folds a tile by itself, codes to fp16 in registers, straight into
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
// in fp32.  Probabilities are relative to a reference below the running maximum
// (fp4::kBelow), raised once a score passes it by 2^15 (as in the chunk kernels):
// most tiles cost one vote for it.
//
// With a quarter of the bytes of bf16 pages the instructions count: a tile costs
// a warp some 1200, 256 conversions and 256 products among them, each two cycles
// of its pipe.  So everything is done for 12 folding warps an SM at 168
// registers, three a scheduler: no producer warp (each warp asks for its own
// tiles, K and V by turns, three halves ahead), the walk over the groups in shared
// memory, the queries' fragments too, and loops short enough for the instruction
// cache.  64 sequences at 512-32768 (1.2 GB of pages): 338 us with a producer
// warp, 16-position tiles and 8 folding warps an SM, 288 with 12 (of 128
// registers), 275 with 8 and 32-position tiles, 245 with loops over their blocks,
// 230 as it is: 5.24 TB/s, 0.78 of the measured copy bandwidth (128 sequences at
// 130000 0.87).  A pair of warps a tile, each half of the output's dims, took 268.  One
// sequence at 700: 11 us, latency.
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

constexpr int kThreads4 = kConsumerThreads;
constexpr int kTileBlocks = 2;   // of K and of V in a tile
constexpr int kTile4 = kTileBlocks * fp4::kRows;  // positions of a tile
constexpr int kCtas4 = 3;        // CTAs per SM
constexpr int kSlots4 = 3;       // halves of tiles (K or V) a warp has room for
constexpr int kMinUnits4 = 4;    // tiles per CTA at least: one per warp
// Tiles of a warp after which its output (of fp32 queries the probabilities' sum
// too) is added to a sum in memory: the MMAs cut off towards zero, of a sum what lies
// 2^-23 below it a step of 16 positions, of a product 2^-25 (paged_chunk_parts.cuh:
// kFoldTiles).  fp32 queries: at most 1.25 * 2^-15 of the output.  Beside one dominant
// position 2.0e-5 of it (64 tiles 3.8e-5, 16 1.3e-5); values alike, 32000 positions a
// warp, never 2.5e-5, 64 tiles 1.6e-6.  128 sequences at 130000: 3340 us, 64 tiles
// 3310, 16 3400.
template <typename QT>
constexpr int kFoldTiles4 = std::is_same<QT, float>::value ? 32 : 64;
constexpr int kPad = 4;          // floats behind each 32 of a state in shared memory
constexpr int kPRow = kTile4 + 4;  // floats of a head's scores of a tile, and a shift of banks
constexpr uint32_t kNoBlock = 0xFFFFFFFFu;

// The walk over the groups waits in shared memory, a copy for each warp, while
// tiles are folded.
constexpr int kWalkBytes = 128;
static_assert(sizeof(paged::Share) <= kWalkBytes, "room for it");

struct Smem4 {
  static constexpr int kSlot = kTileBlocks * fp4::kBlock;
  static constexpr int kWarp = kSlots4 * kSlot;  // a warp's slots
  static constexpr int kQ = kConsumers * kWarp;
  static constexpr int kP = kQ + kHeadDim / 32 * 32 * 16;
  static constexpr int kM = kP + kConsumers * 4 * kPRow * 4;
  static constexpr int kL = kM + kConsumers * 16;
  static constexpr int kBars = kL + kConsumers * 16;
  static constexpr int kFlags = kBars + kConsumers * kSlots4 * 8;
  static constexpr int kWalk = kFlags + 16;
  static constexpr int kBytes = kWalk + kConsumers * kWalkBytes;
  // the prefix sums, before the first copy
  static_assert(8 * (SPARK_MAX_BATCH + 2 + kThreads4 / 16) <= kQ, "room in the slots");
  static_assert(4 * kStateFloats<kPad> * 4 <= kSlot, "a warp's state in a slot");
};

// The queries of a KV head as the B fragments of all 16-dim steps, in shared
// memory for all warps: step s holds dims 64 t + 4 s .. + 3, column g head g & 3,
// its high half for g < 4; steps 2 i and 2 i + 1 of a lane are 16 bytes.
struct Queries {
  uint32_t b;      // [8][32] of 16 bytes, the lane's
  float scale[2];  // of the scores of heads 2 (t & 1) + j
};

__device__ __forceinline__ void load16(float (&x)[16], const float* q) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(q) + i);
    x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
  }
}
__device__ __forceinline__ void load16(float (&x)[16], const __nv_bfloat16* q) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(q) + i);
    const float2 a = bf16x2_to_f32x2(v.x), b = bf16x2_to_f32x2(v.y), c = bf16x2_to_f32x2(v.z), d = bf16x2_to_f32x2(v.w);
    x[8 * i] = a.x; x[8 * i + 1] = a.y; x[8 * i + 2] = b.x; x[8 * i + 3] = b.y;
    x[8 * i + 4] = c.x; x[8 * i + 5] = c.y; x[8 * i + 6] = d.x; x[8 * i + 7] = d.y;
  }
}

// Every warp finds the heads' units, and puts a quarter of the steps down.
template <typename QT>
__device__ __forceinline__ void load_queries(Queries& Q, uint4* q_s, const QT* qg, float scale_log2, int warp, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const QT* mine = qg + (g & 3) * kHeadDim + 64 * t;
  float m = 0.f, y[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[16];
    load16(x, mine + 16 * i);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      m = fmaxf(m, fabsf(x[e]));
      y[e] = i == warp ? x[e] : y[e];
    }
  }
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const float2 unit = fp4::unit_of(m);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      h[j] = fp4::pack(fp4::split_part(y[8 * i + 2 * j] * unit.x, g >= 4), fp4::split_part(y[8 * i + 2 * j + 1] * unit.x, g >= 4));
    q_s[32 * (2 * warp + i) + lane] = make_uint4(h[0], h[1], h[2], h[3]);
  }
  Q.b = smem_u32(q_s + lane);
#pragma unroll
  for (int j = 0; j < 2; ++j) Q.scale[j] = scale_log2 * __shfl_sync(0xffffffffu, unit.y, 4 * (2 * (t & 1) + j));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Shared memory by its own addresses.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint32_t v;
  asm volatile("{\n\t.reg .u16 h;\n\tld.shared.u16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }

// A lane's places in a block: its first chunk of rows g and g + 8 of K and their
// scales, its chunk of row 4 t of V (of row 4 t + j at ^ 16 (j & 1), 128 j behind)
// and its scales.
struct Places {
  uint32_t ka, kb, ks, v, vs;
  __device__ __forceinline__ explicit Places(int lane) {
    const int g = lane >> 2, t = lane & 3;
    ka = (uint32_t)fp4::code_at(g, 64 * t);
    kb = (uint32_t)fp4::code_at(g + 8, 64 * t);
    ks = (uint32_t)fp4::scale_at(g, 64 * t);
    v = (uint32_t)fp4::code_at(4 * t, 32 * g);
    vs = (uint32_t)fp4::scale_at(4 * t, 32 * g);
  }
};

// Byte `i` of a word of scales as an fp16 pair of it.
__device__ __forceinline__ uint32_t scale2(uint32_t w, int i) { return __byte_perm(w, 0u, 0x4040u | (uint32_t)(i | (i << 8))) << 7; }

// One warp's running state: o[i] holds dims 32 g + 2 i in [0], [1], the next in
// [2], [3], of columns 2 t and 2 t + 1; m the references (base 2) of the columns'
// heads 2 (t & 1) + j, mg of head g & 3, l the sum of head g & 3 over positions 4
// t .. 4 t + 3 of every block.
struct State4 {
  float o[kHeadDim / 16][4];
  float m[2], mg, l;
  float m_sum[2];  // references of the sum in memory, -inf while there is none
  __device__ __forceinline__ void reset() {
    clear();
    m[0] = m[1] = mg = m_sum[0] = m_sum[1] = -INFINITY;
    l = 0.f;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kHeadDim / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }
  // o and (L) l += the lane's part of the sums in memory, under the references of now
  template <bool L>
  __device__ __forceinline__ void add(const float* sums, int lane) {
    const float4* sum = reinterpret_cast<const float4*>(sums) + lane;
    const float* sum_l = sums + 8 * kHeadDim + lane;
    if (L && sum_l[32] != -INFINITY) l = fmaf(sum_l[0], ex2(sum_l[32] - mg), l);
    float f[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) f[j] = m_sum[j] == -INFINITY ? 0.f : ex2(m_sum[j] - m[j]);
#pragma unroll
    for (int i = 0; i < kHeadDim / 16; ++i) {
      const float4 x = sum[32 * i];
      o[i][0] = fmaf(f[0], x.x, o[i][0]);
      o[i][1] = fmaf(f[1], x.y, o[i][1]);
      o[i][2] = fmaf(f[0], x.z, o[i][2]);
      o[i][3] = fmaf(f[1], x.w, o[i][3]);
    }
  }
  template <bool L>
  __device__ __forceinline__ void put(float* sums, int lane) {
    float4* sum = reinterpret_cast<float4*>(sums) + lane;
    float* sum_l = sums + 8 * kHeadDim + lane;
    if (L) {
      sum_l[0] = l;
      sum_l[32] = mg;
      l = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kHeadDim / 16; ++i) sum[32 * i] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
    m_sum[0] = m[0];
    m_sum[1] = m[1];
    clear();
  }
};

// One warp folds rows [r0, r1) of a tile into its state: first K's blocks, their
// scores into the warp's 4 x kPRow scratch and the lane's maxima, then V's.  Rows
// outside may hold anything.  (The loops over blocks are not unrolled, see above.)
__device__ __forceinline__ void fold_keys(uint32_t kst, int r0, int r1, const Queries& Q, const Places& at, uint32_t p_w,
                                          float (&mx)[2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const bool whole = r0 == 0 && r1 == kTile4;
  mx[0] = mx[1] = -INFINITY;
  __syncwarp();  // the scratch is free
#pragma unroll 1
  for (int blk = 0; blk < kTileBlocks; ++blk) {
    const uint32_t kb = kst + blk * fp4::kBlock;
    // s = K q^T, even and odd steps in two chains
    float c[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t sa = lds32(kb + at.ks), sb = lds32(kb + at.ks + 8 * fp4::kScales);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 xa = lds128(kb + (at.ka ^ (uint32_t)(16 * i))), xb = lds128(kb + (at.kb ^ (uint32_t)(16 * i)));
      const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t fa = scale2(sa, w >> 1), fb = scale2(sb, w >> 1);
        uint32_t ha[4], hb[4];
        fp4::halves8(wa[w], ha);
        fp4::halves8(wb[w], hb);
        const uint32_t a0[4] = {fp4::mul2(ha[0], fa), fp4::mul2(hb[0], fb), fp4::mul2(ha[1], fa), fp4::mul2(hb[1], fb)};
        const uint32_t a1[4] = {fp4::mul2(ha[2], fa), fp4::mul2(hb[2], fb), fp4::mul2(ha[3], fa), fp4::mul2(hb[3], fb)};
        const uint4 qb = lds128(Q.b + 512 * (4 * i + w));
        mma_f16(c, a0, qb.x, qb.y);
        mma_f16(c2, a1, qb.z, qb.w);
      }
      sa >>= 16;
      sb >>= 16;
    }
    // hi and lo columns, scale, mask: c[2 r + j] is row g + 8 r, head 2 (t & 1) + j
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[e] += c2[e];
      c[e] += __shfl_xor_sync(0xffffffffu, c[e], 2);
      c[e] *= Q.scale[e & 1];
    }
    if (!whole) {
      const int row = 16 * blk + g;
      if (row < r0 || row >= r1) c[0] = c[1] = -INFINITY;
      if (row + 8 < r0 || row + 8 >= r1) c[2] = c[3] = -INFINITY;
    }
    mx[0] = fmaxf(mx[0], fmaxf(c[0], c[2]));
    mx[1] = fmaxf(mx[1], fmaxf(c[1], c[3]));
    if (t < 2) {
      const uint32_t to = p_w + 4 * (2 * t * kPRow + 16 * blk + g);
      sts32(to, c[0]);
      sts32(to + 4 * kPRow, c[1]);
      sts32(to + 32, c[2]);
      sts32(to + 4 * kPRow + 32, c[3]);
    }
  }
}

__device__ __forceinline__ void fold_values(uint32_t vst, int r0, int r1, const Places& at, uint32_t p_w, float (&mx)[2], State4& st) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const bool whole = r0 == 0 && r1 == kTile4;
  if (__any_sync(0xffffffffu, fp4::past(mx[0], st.m[0]) || fp4::past(mx[1], st.m[1]))) {
    float corr[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 4));
      mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 8));
      mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 16));
      const float mn = fmaxf(st.m[j], fp4::below(mx[j]));
      corr[j] = st.m[j] == -INFINITY ? 0.f : exp2f(st.m[j] - mn);
      st.m[j] = mn;
    }
    // of head g & 3: the lane t = (g & 3) / 2 has it
    const float m0 = __shfl_sync(0xffffffffu, st.m[0], (g & 3) >> 1), m1 = __shfl_sync(0xffffffffu, st.m[1], (g & 3) >> 1);
    const float mn = (g & 1) ? m1 : m0;
    st.l *= st.mg == -INFINITY ? 0.f : exp2f(st.mg - mn);
    st.mg = mn;
#pragma unroll
    for (int i = 0; i < kHeadDim / 16; ++i) {
      st.o[i][0] *= corr[0];
      st.o[i][1] *= corr[1];
      st.o[i][2] *= corr[0];
      st.o[i][3] *= corr[1];
    }
  }
  const float ref = st.mg == -INFINITY ? 0.f : st.mg;
  __syncwarp();
  // p, and o^T += V^T p^T
#pragma unroll 1
  for (int blk = 0; blk < kTileBlocks; ++blk) {
    const uint32_t vb = vst + blk * fp4::kBlock;
    uint32_t v[4][4], f01[2], f23[2], s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 4 * t + j;
      const uint4 x = lds128(vb + (at.v ^ (uint32_t)(16 * (j & 1))) + j * fp4::kCodes);
      v[j][0] = x.x; v[j][1] = x.y; v[j][2] = x.z; v[j][3] = x.w;
      s[j] = lds16(vb + at.vs + j * fp4::kScales);
      // (0 times whatever a row outside holds, a NaN's scale included)
      if (!whole && (16 * blk + row < r0 || 16 * blk + row >= r1)) s[j] = 0;
    }
    // B fragments of [p_hi | p_lo]^T: the MMA's steps 2 t, 2 t + 1, 2 t + 8, 2 t +
    // 9 are positions 4 t .. 4 t + 3 (a masked one's probability is 0, also
    // under a reference of -inf)
    const uint4 s4 = lds128(p_w + 4 * ((g & 3) * kPRow + 16 * blk + 4 * t));
    const float4 p4 = make_float4(ex2(__uint_as_float(s4.x) - ref), ex2(__uint_as_float(s4.y) - ref),
                                  ex2(__uint_as_float(s4.z) - ref), ex2(__uint_as_float(s4.w) - ref));
    st.l += (p4.x + p4.y) + (p4.z + p4.w);
    const uint32_t pb0 = fp4::pack(fp4::split_part(p4.x, g >= 4), fp4::split_part(p4.y, g >= 4));
    const uint32_t pb1 = fp4::pack(fp4::split_part(p4.z, g >= 4), fp4::split_part(p4.w, g >= 4));
    const uint32_t s01 = s[0] | (s[1] << 16), s23 = s[2] | (s[3] << 16);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f01[u] = ((s01 >> (8 * u)) & 0x00FF00FFu) << 7;
      f23[u] = ((s23 >> (8 * u)) & 0x00FF00FFu) << 7;
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
}

// Put one warp's state into the merge scratch: the hi and lo columns and the
// lanes' sums added.
__device__ __forceinline__ void store_state4(State4& st, const MergeSmem& sm) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < kHeadDim / 16; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) st.o[i][k] += __shfl_xor_sync(0xffffffffu, st.o[i][k], 2);
  st.l += __shfl_xor_sync(0xffffffffu, st.l, 1);
  st.l += __shfl_xor_sync(0xffffffffu, st.l, 2);
  if (lane < 16 && t == 0) {
    sm.ms[warp * 4 + g] = st.mg;
    sm.ls[warp * 4 + g] = st.l;
  }
  if (t < 2) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int h = 2 * t + j;
      float* os = sm.os + warp * (Smem4::kWarp / 4) + h * kStateFloats<kPad> + state_at<kPad>(32 * g);
#pragma unroll
      for (int i = 0; i < kHeadDim / 16; i += 2)
        *reinterpret_cast<float4*>(os + 2 * i) = make_float4(st.o[i][j], st.o[i][2 + j], st.o[i + 1][j], st.o[i + 1][2 + j]);
    }
  }
}

// A warp's way through its tiles of a group (every kConsumers-th of the CTA's):
// item 2 j is K of its tile j, 2 j + 1 V; the copies run kSlots4 items ahead.  A
// warp fills its own slots, lanes 0 and 1 a block each, so nothing but the copies'
// own barriers is waited for.
struct Stream {
  uint32_t slots, bars;  // shared addresses
  uint32_t fill, use;    // slots filled and used next
  uint32_t phase;        // of the slot used next
  uint32_t block;        // of lane 2 i + b: block b of tile i of the 16 looked up
  int issued, items;     // of this group
  int x0;                // first position of the group's first tile of the warp

  __device__ __forceinline__ void begin(int x, int tiles) {
    x0 = x;
    issued = 0;
    items = 2 * tiles;
  }
  __device__ __forceinline__ uint32_t slot() const { return slots + use * Smem4::kSlot; }
  __device__ __forceinline__ void issue(const Args& p, const Cursor& cur, const unsigned char* pk, const unsigned char* pv,
                                        int lane) {
    if (issued >= items) return;
    if ((issued & 31) == 0) {
      const int tile = (issued >> 1) + (lane >> 1), x = x0 + tile * (kConsumers * kTile4) + (lane & 1) * fp4::kRows;
      block = kNoBlock;
      if (2 * tile < items && x <= cur.g.hi && x + fp4::kRows > cur.g.lo) {
        const int col = paged::page_col(p, x), in_page = (x - col * p.page_size) / fp4::kRows;
        const int page = paged::page_of(p, paged::page_entry(p, cur.s, col));
        // (pages * page_size < 2^31: the blocks of all heads are below 2^30)
        block = ((uint32_t)page * (uint32_t)(p.page_size / fp4::kRows) + (uint32_t)in_page) * (uint32_t)p.n_kv + (uint32_t)cur.j;
      }
    }
    const uint32_t mine = __shfl_sync(0xffffffffu, block, (issued & 30) | (lane & 1));
    if (lane < 2) {
      const uint32_t bar = bars + 8 * fill;
      if (mine != kNoBlock) {
        const unsigned char* from = ((issued & 1) ? pv : pk) + (uint64_t)mine * fp4::kBlock;
        asm volatile(
            "{\n\t.reg .b64 st;\n\t"
            "mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 st, [%0], %1;\n\t"
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%2], [%3], %1, [%0];\n\t}" ::"r"(bar),
            "r"(fp4::kBlock), "r"(slots + fill * Smem4::kSlot + lane * fp4::kBlock), "l"(reinterpret_cast<uint64_t>(from))
            : "memory");
      } else {
        asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.release.cta.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar) : "memory");
      }
    }
    ++issued;
    fill = fill + 1 == kSlots4 ? 0 : fill + 1;
  }
  __device__ __forceinline__ bool wait(volatile int* abort) const {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 q, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(done)
        : "r"(bars + 8 * use), "r"(phase)
        : "memory");
    if (__all_sync(0xffffffffu, done != 0)) return true;
    uint64_t* bar = reinterpret_cast<uint64_t*>(__cvta_shared_to_generic(bars + 8 * use));
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, phase, abort, kWaitLimitNs));
  }
  __device__ __forceinline__ void advance() {
    const bool last = use + 1 == kSlots4;
    use = last ? 0 : use + 1;
    phase ^= last ? 1u : 0u;
  }
};

template <typename QT>
__global__ void __launch_bounds__(kThreads4, kCtas4)
    k_paged4_token(const unsigned char* pk, const unsigned char* pv, const __grid_constant__ Args p) {
  using S = Smem4;
  extern __shared__ __align__(128) unsigned char base[];
  volatile int* flags = reinterpret_cast<volatile int*>(base + S::kFlags);  // [0] abort, [1] last
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t p_w = smem_u32(base + S::kP) + warp * 16 * kPRow;
  const Places places(lane);
  if (tid == 0) {
    for (int s = 0; s < kConsumers * kSlots4; ++s) mbar_init(reinterpret_cast<uint64_t*>(base + S::kBars) + s, 2);
    flags[0] = 0;
    flags[1] = 0;
    fence_mbar_init();
  }
  // tables, lengths, rows and queries may come from the kernel before
  pdl_wait();
  pdl_trigger();
  const Shape sh{1, kTile4, p.window};
  const int c = blockIdx.x;
  paged::Share share;
  if (!paged::find_share<kThreads4>(p, sh, c, kMinUnits4, gridDim.x, reinterpret_cast<int64_t*>(base), share)) return;
  paged::Share& walk = *reinterpret_cast<paged::Share*>(base + S::kWalk + warp * kWalkBytes);
  if (lane == 0) walk = share;
  __syncthreads();  // the prefix sums have been read
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // and make way for the copies
  Stream in;
  in.slots = smem_u32(base) + warp * S::kWarp;
  in.bars = smem_u32(base + S::kBars) + warp * kSlots4 * 8;
  in.fill = in.use = in.phase = 0;
  int skip = warp;  // the CTA's tiles before the warp's next one
  Queries Q;
  State4 st;
  constexpr int kFold = kFoldTiles4<QT>;
  constexpr bool kFoldL = std::is_same<QT, float>::value;
  auto sums = [&] {
    return p.part + paged::kTokenPartBytes / sizeof(float) + (int64_t)(c * kConsumers + warp) * paged::kWarpSums;
  };
  bool ok = true;
  for (;;) {
    int n, tiles, pos, lo, hi;
    {
      const paged::Share w = walk;
      const int64_t t0 = w.cur.begin > w.u0 ? w.cur.begin : w.u0, t1 = w.cur.end < w.u1 ? w.cur.end : w.u1;
      n = (int)(t1 - t0);
      tiles = skip < n ? (n - skip + kConsumers - 1) / kConsumers : 0;
      pos = (w.cur.g.tile0 + (int)(t0 - w.cur.begin) + skip) * kTile4;
      lo = w.cur.g.lo;
      hi = w.cur.g.hi;
    }
    in.begin(pos, tiles);
    skip += tiles * kConsumers - n;
#pragma unroll 1
    for (int i = 0; i < kSlots4; ++i) in.issue(p, walk.cur, pk, pv, lane);
    load_queries(Q, reinterpret_cast<uint4*>(base + S::kQ),
                 static_cast<const QT*>(p.q) + (int64_t)(walk.cur.seq.q0 + walk.cur.g.tok) * p.q_ld + walk.cur.j * (kGroup * kHeadDim),
                 p.scale_log2, warp, lane);
    st.reset();
    named_bar_sync(kBarConsumers, kConsumerThreads);  // the queries are there
    int done = 0;  // items
    auto landed = [&] {
      ok = ok && in.wait(flags);
      return ok;
    };
    auto used = [&] {
      ++done;
      in.advance();
      __syncwarp();  // the slot has been read
      in.issue(p, walk.cur, pk, pv, lane);
    };
#pragma unroll 1
    for (int i = 0; i < tiles; ++i, pos += kConsumers * kTile4) {
      if (i % kFold == 0 && i > 0) {
        if (i > kFold) st.add<kFoldL>(sums(), lane);
        st.put<kFoldL>(sums(), lane);
      }
      const int r0 = lo > pos ? lo - pos : 0, r1 = hi + 1 - pos < kTile4 ? hi + 1 - pos : kTile4;
      float mx[2];
      if (!landed()) break;
      fold_keys(in.slot(), r0, r1, Q, places, p_w, mx);
      used();
      if (!landed()) break;
      fold_values(in.slot(), r0, r1, places, p_w, mx, st);
      used();
    }
    if (!ok) {
      if (lane == 0) {
        if (!flags[0]) atomicOr(p.err, kErrWaitTimeout);
        flags[0] = 1;
      }
      // let the copies in flight land before the CTA can exit
      for (; done < in.issued; ++done) {
        int never = 0;
        mbar_wait_bounded(reinterpret_cast<uint64_t*>(__cvta_shared_to_generic(in.bars + 8 * in.use)), in.phase, &never, kWaitLimitNs);
        in.advance();
      }
    }
    if (ok && tiles > kFold) st.add<kFoldL>(sums(), lane);
    // the warps' states lie in a slot of each: the slots are all free now
    const MergeSmem msm{reinterpret_cast<float*>(base + S::kM), reinterpret_cast<float*>(base + S::kL),
                        reinterpret_cast<float*>(base)};
    store_state4(st, msm);
    Cursor cur = walk.cur;
    finish_group<QT, kPad, S::kWarp / 4>(
        msm, flags, p, static_cast<QT*>(p.a) + ((int64_t)(cur.seq.q0 + cur.g.tok) * p.n_kv + cur.j) * (kGroup * kHeadDim),
        Parts(cur.begin, cur.end, walk.total, walk.G, c));
    if (cur.end >= walk.u1) break;
    cur.next(p, sh);
    __syncwarp();
    if (lane == 0) walk.cur = cur;
    named_bar_sync(kBarConsumers, kConsumerThreads);  // the states have been read
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // and make way for the copies
  }
}

template <typename QT>
cudaError_t launch_token4(const Args& p, const void* k, const void* v, cudaStream_t st) {
  auto kern = k_paged4_token<QT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem4::kBytes);
  if (e != cudaSuccess) return e;
  // CTAs for sqrt(2 U) parts a group of as many tiles U as the tables have room for
  // (where a group has fewer, ctas_for takes fewer): with 456 always, parts that
  // were fewer lay two on an SM beside SMs without (one sequence at 8000 18.8 us, now
  // 16.7; at 32768 30.9 and 29.4).  sqrt(4 U), the limit of bf16 pages, 17.7 and
  // 30.3; sqrt(U) 18.6 and 26.7.  These tables were as wide as the sequence; with room
  // for 131072 positions 20.3 and 31.6.
  int64_t tiles = ((int64_t)p.max_pages * p.page_size + kTile4 - 1) / kTile4;
  if (p.window > 0 && tiles > p.window / kTile4 + 2) tiles = p.window / kTile4 + 2;
  int64_t parts = tiles / kMinUnits4;
  const int64_t cap = (int64_t)sqrt(2.0 * (double)tiles);
  if (parts > cap) parts = cap;
  if (parts < 1) parts = 1;
  const int groups = p.n_seqs * p.n_kv;
  int grid = kCtas4 * device_sm_count();
  if (grid > paged::kMaxCtas) grid = paged::kMaxCtas;
  // Where groups have parts for more, a whole number of CTAs each if that leaves an
  // eighth of them at most: 16 sequences at 2000, 64 groups on 448 CTAs 18.9 us, cut
  // by all 456 22.8.
  const int whole = grid / groups * groups;
  if (groups * parts <= grid)
    grid = (int)(groups * parts);
  else if ((grid - whole) * 8 <= grid)
    grid = whole;
  return launch_pdl(kern, dim3(grid), dim3(kThreads4), Smem4::kBytes, st, static_cast<const unsigned char*>(k),
                    static_cast<const unsigned char*>(v), p);
}

}  // namespace

cudaError_t launch_paged4_attention(const paged::Args& p, int qdtype, const void* k, const void* v, cudaStream_t st) {
  if (p.max_q == 1) return qdtype == SPARK_BF16 ? launch_token4<__nv_bfloat16>(p, k, v, st) : launch_token4<float>(p, k, v, st);
  // Pairs of CTAs or single ones by the rule of launch_paged_attention, for its
  // reasons (bf16 queries: 32 sequences of 33 tokens at 4096-8192 165 us on pairs,
  // 184 on single CTAs, a chunk of 4096 264 and 328; 4 tokens each 150 and 98, 32 of
  // them 4 with chunks of ~400 tokens 155 and 135, fp32 queries 265 and 224).
  if (p.max_q > paged::kChunkTokens && (2 * (int64_t)p.n_tokens > (int64_t)p.n_seqs * p.max_q || p.n_tokens > 128 * p.n_seqs))
    return launch_paged4_pair(p, qdtype, k, v, st);
  return launch_paged4_chunk(p, qdtype, k, v, st);
}

}  // namespace spark
