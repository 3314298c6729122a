// paged_chunk_parts.cuh -- what the chunk attention kernels share
// (paged_chunk.cu: one CTA and 32 tokens a group; paged_pair.cu: two CTAs and
// 64): the queries' layout in shared memory, the softmax warps, the join of
// partial states, the tensor map of a pool.
#pragma once

#include <math.h>

#include <type_traits>

#include "launch.h"
#include "paged_launch.h"
#include "paged_parts.cuh"
#include "tmem.cuh"

namespace spark {
namespace chunk {

using paged::Args;
using paged::Cursor;
using paged::Shape;

constexpr int kRows = 128;                      // rows of a group: 32 tokens x 4 heads
constexpr int kPos = 128;                       // positions of a tile
constexpr int kThreads = 192;
constexpr int kSoft = 128;                      // softmax threads, one row each (an arrival per warp)
constexpr uint32_t kLineBytes = kPos * 128;     // 64 dims of 128 rows or positions
constexpr uint32_t kSlot = 2 * kLineBytes;      // 128 dims
constexpr uint32_t kQBytes = 4 * kLineBytes;
// K and V lie in a slot as groups of 8 rows, each group line by line: [row /
// 8][line][8 rows][128 bytes].  So one TMA box holds all the slot's lines of
// its rows, and groups and lines are a fixed stride apart, as an MMA's operand
// wants them.  TMA spends about 100 cycles on a request whatever its size:
// line by line, pages of 16 rows bound a tile by its 64 requests (a mixed
// batch of 32, bf16 queries: 135 against 107 us; a chunk of 4096 345 against
// 240), and longer pages gained nothing (109 and 225 us either way).
constexpr uint32_t kAtom = 8 * 128;
template <int LINES>  // of a slot
constexpr uint32_t kGroupBytes = LINES * kAtom;
constexpr uint32_t kCols = 512;
constexpr uint32_t kColS = 256;                 // first column of S buffer 0; O starts at 0
constexpr float kRaise = 8.0f;                  // m is raised once a score passes it by 2^8

// L2 policies of the pool's rows.  A sequence of one group reads its rows
// once: they make room first, or they would drive out the rows of longer
// chunks, which every group of the sequence reads, up to a whole call later (28
// sequences with up to 7 new tokens, 0.37 GB: 79 -> 74 us).
__device__ __forceinline__ uint64_t policy_once() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t policy_again() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// A TMA load of a box of rows from row `row` (a multiple of 8), lines `line` ..,
// of a head, under a policy.
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* map, uint64_t* bar, int row, int line,
                                              int head, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(line), "r"(row >> 3), "r"(head), "l"(policy)
      : "memory");
}

// A warp clears the rows outside [r0, r1) of a slot of two lines of 128 rows.
// (Kept small: a loop over the rows, unrolled, cost a mixed batch 18 of 123
// us, the MMA warp's code missing the instruction cache.)
__device__ __forceinline__ void clear_rows(unsigned char* v, int r0, int r1, int lane) {
#pragma unroll 1
  for (int g = 0; g < kPos / 8; ++g) {
    if (8 * g >= r0 && 8 * g + 8 <= r1) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * (i & 1) + (lane >> 3);
      if (8 * g + r < r0 || 8 * g + r >= r1)
        *reinterpret_cast<uint4*>(v + g * kGroupBytes<2> + (i >> 1) * kAtom + r * 128 + (lane & 7) * 16) =
            make_uint4(0u, 0u, 0u, 0u);
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) { return ffma2(a, make_float2(1.f, 1.f), b); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// eight elements of a query row as bf16 and the remainders
__device__ __forceinline__ void split8(const float (&x)[8], uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack2(x[2 * i], x[2 * i + 1]);
    const float2 f = bf16x2_to_f32x2(h[i]);
    l[i] = pack2(x[2 * i] - f.x, x[2 * i + 1] - f.y);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Queries in shared memory: 64-dim lines of 128 rows, 16-byte chunk c of row r
// at c ^ (r % 8) (the 128-byte swizzle).  TMA brings them, bf16 as they are
// used, fp32 in 32-dim lines, which the softmax warps turn into a line of bf16
// halves and a line of remainders in the same place.  (Read by the warps 8
// rows at a time instead, they took 5 us at the start and 3 to 6 at each later
// group.)  More than 16 tokens come in one request of 32 with all lines, fewer
// in requests of a line of 8.  Rows behind the group's last token are other
// tokens', zero or what they were: their scores reach no other row, and
// nothing is written for them.
constexpr int kQueryBoxTokens = 8;
constexpr int kQueryBoxes = paged::kChunkTokens / kQueryBoxTokens;
constexpr uint32_t kQueryBox = kQueryBoxTokens * kGroup * 128;  // bytes
template <typename QT>
constexpr int kQueryLines = kHeadDim * sizeof(QT) / 128;

// 8-token boxes of a line that hold tokens of the group, of the 32 from `tok0`
__device__ __forceinline__ int query_boxes(int n_tok, int tok0) {
  return min(kQueryBoxes, max(0, (n_tok - tok0 + kQueryBoxTokens - 1) / kQueryBoxTokens));
}
template <typename QT>
__device__ __forceinline__ uint32_t query_bytes(int n_tok, int tok0) {
  const int n = query_boxes(n_tok, tok0);
  return (n > kQueryBoxes / 2 ? kQueryBoxes : n) * (kQueryLines<QT> * kQueryBox);
}
// a warp loads them: load(map, to, head, token, line)
template <typename QT, typename Load>
__device__ __forceinline__ void load_queries(unsigned char* q_s, const CUtensorMap* all, const CUtensorMap* box,
                                             const Cursor& cur, int tok0, int lane, Load load) {
  const int n = query_boxes(cur.g.n_tok, tok0), head = kGroup * cur.j, tok = cur.seq.q0 + cur.g.tok + tok0;
  if (n > kQueryBoxes / 2) {
    if (lane == 0) load(all, q_s, head, tok, 0);
  } else {
    const int line = lane % kQueryLines<QT>, b = lane / kQueryLines<QT>;
    if (b < n) load(box, q_s + line * kLineBytes + b * kQueryBox, head, tok + kQueryBoxTokens * b, line);
  }
}

// row r of fp32 queries into halves, in place: its 256 bytes in lines 2 i and
// 2 i + 1 become those of line i of the halves and of the remainders
__device__ __forceinline__ void split_query(unsigned char* q_s, int i, int r) {
  unsigned char* row = q_s + 2 * i * kLineBytes + r * 128;
  float4 x[16];
#pragma unroll
  for (int c = 0; c < 16; ++c)
    x[c] = *reinterpret_cast<const float4*>(row + (c >> 3) * kLineBytes + (((c & 7) ^ (r & 7)) << 4));
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float v[8] = {x[2 * c].x,     x[2 * c].y,     x[2 * c].z,     x[2 * c].w,
                        x[2 * c + 1].x, x[2 * c + 1].y, x[2 * c + 1].z, x[2 * c + 1].w};
    uint4 hi, lo;
    split8(v, hi, lo);
    *reinterpret_cast<uint4*>(row + ((c ^ (r & 7)) << 4)) = hi;
    *reinterpret_cast<uint4*>(row + kLineBytes + ((c ^ (r & 7)) << 4)) = lo;
  }
}

// rows [token][head][256] as [line][token][head][128 bytes]
template <typename QT>
bool make_query_map(CUtensorMap* map, const Args& p, int tokens, int lines) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  constexpr cuuint64_t es = sizeof(QT);
  const cuuint64_t dims[4] = {128 / es, (cuuint64_t)(kGroup * p.n_kv), (cuuint64_t)p.n_tokens, kQueryLines<QT>};
  const cuuint64_t strides[3] = {kHeadDim * es, (cuuint64_t)p.q_ld * es, 128};
  const cuuint32_t shape[4] = {128 / es, kGroup, (cuuint32_t)tokens, (cuuint32_t)lines};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, es == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void*>(p.q), dims, strides, shape, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
template <typename QT>
bool make_query_maps(CUtensorMap* all, CUtensorMap* box, const Args& p) {
  return make_query_map<QT>(all, p, paged::kChunkTokens, kQueryLines<QT>) &&
         make_query_map<QT>(box, p, kQueryBoxTokens, 1);
}

// The columns x0 .. x1 of a tile that a row sees, as one bit per column of
// the 32 from `first`.
__device__ __forceinline__ uint32_t seen32(int x0, int x1, int first) {
  const int a = x0 - first, b = x1 + 1 - first;  // bits [a, b)
  const uint32_t below_b = b >= 32 ? 0xffffffffu : b <= 0 ? 0u : (1u << b) - 1u;
  const uint32_t below_a = a >= 32 ? 0xffffffffu : a <= 0 ? 0u : (1u << a) - 1u;
  return below_b & ~below_a;
}

// 32 scores of a row become P = e^(scale s - ref) in bf16 (SPLIT: and the
// remainders) over their own columns at `ts`.
template <bool SPLIT>
__device__ __forceinline__ void exp32(uint32_t ts, const uint32_t (&s)[32], float scale, float ref, float2 (&sum)[2]) {
  uint32_t hi[16], lo[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 t = ffma2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])),
                           make_float2(scale, scale), make_float2(-ref, -ref));
    const float2 e = make_float2(ex2(t.x), ex2(t.y));
    sum[i & 1] = fadd2(sum[i & 1], e);
    hi[i] = pack2(e.x, e.y);
    if (SPLIT) {
      const float2 f = bf16x2_to_f32x2(hi[i]);
      lo[i] = pack2(e.x - f.x, e.y - f.y);
    }
  }
  tc::st16(ts, hi);
  if (SPLIT) tc::st16(ts + 16, lo);
}

// scores a row does not see become -inf (whatever they are: the rows of K
// behind a sequence's end may hold anything)
__device__ __forceinline__ void mask32(uint32_t (&s)[32], uint32_t seen) {
#pragma unroll
  for (int i = 0; i < 32; ++i) s[i] = ((seen >> i) & 1u) ? s[i] : 0xFF800000u;
}

__device__ __forceinline__ void max32(const uint32_t (&s)[32], float (&mx)[4]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      mx[k] = fmaxf(mx[k], fmaxf(__uint_as_float(s[i + k]), __uint_as_float(s[i + k + 4])));
}

// scores of a negative or zero scale
__device__ __forceinline__ void sign32(uint32_t (&s)[32], float sign) {
#pragma unroll
  for (int i = 0; i < 32; ++i) s[i] = __float_as_uint(__uint_as_float(s[i]) * sign);
}

// 32 output dims of a row
__device__ __forceinline__ void store32(__nv_bfloat16* dst, const uint32_t (&o)[32], float inv) {
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = pack2(__uint_as_float(o[i + 2 * k]) * inv, __uint_as_float(o[i + 2 * k + 1]) * inv);
    reinterpret_cast<uint4*>(dst)[i / 8] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

constexpr int kStageRow = 64 + 16;             // bytes of a row of an output stage: 32 bf16 dims, padding
constexpr int kStageBytes = 32 * kStageRow;    // of a warp

// The four softmax warps (st: their thread, 0 .. 127) of a CTA of RANKS that
// share a group, one row per thread: scores to probabilities, the running
// maximum and sum, the output at the group's end.  arrive_q, arrive_p: one
// lane per warp tells the MMA warp that fp32 queries are in halves, or the
// probabilities in a buffer.  STAGE: whole groups' outputs leave through
// `stage`.
template <typename QT, int RANKS, bool STAGE, typename ArriveQ, typename ArriveP>
__device__ __forceinline__ void softmax_warps(const Args& p, const Shape& sh, Cursor cur, int64_t u0, int64_t u1,
                                              int64_t total, int G, int c, int rank, unsigned char* q_s, uint32_t tmem,
                                              uint64_t* q_raw, uint64_t* s_full, uint64_t* pv_done,
                                              volatile int* flags, unsigned char* stage, int warp, int st,
                                              ArriveQ arrive_q, ArriveP arrive_p) {
  const int quad = warp & 3, lane = st & 31, tok0 = rank * paged::kChunkTokens;
  const int row = quad * 32 + lane;
  const int prow = rank * kRows + row;  // the row in a partial state
  const uint32_t lanes = (uint32_t)(quad * 32) << 16;
  // a scale of zero or below is taken to the scores before they are masked: a
  // masked one of -inf stays that
  const float sign = p.scale_log2 < 0.f ? -1.f : p.scale_log2 > 0.f ? 1.f : 0.f;
  const float scale = sign == 0.f ? 1.f : fabsf(p.scale_log2);
  QT* out = static_cast<QT*>(p.a);
  uint32_t tile = 0;
  bool ok = true;
  constexpr bool kSplit = std::is_same<QT, float>::value;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, flags, kWaitLimitNs));
    tc::fence_after();
    return ok;
  };
  // fp32 queries have landed: into halves
  uint32_t item = 0;
  auto split_queries = [&](const Cursor& at) {
    if (!wait(q_raw, item++ & 1)) return;
#pragma unroll 1
    for (int b = 0; b < query_boxes(at.g.n_tok, tok0); ++b) split_query(q_s, quad, 32 * b + lane);  // a line per warp
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMAs read it through the async proxy
    __syncwarp();
    if (lane == 0) arrive_q();
  };
  if (kSplit) split_queries(cur);
  for (;;) {
    const int64_t t0 = cur.begin > u0 ? cur.begin : u0, t1 = cur.end < u1 ? cur.end : u1;
    const paged::Group g = cur.g;
    const int tok = tok0 + (row >> 2);
    // positions the row sees; rows behind the last token take the last one's
    const int pos_hi = cur.seq.p0 + g.tok + (tok < g.n_tok ? tok : g.n_tok - 1);
    const int pos_lo = p.window > 0 && pos_hi + 1 > p.window ? pos_hi + 1 - p.window : 0;
    const bool live = tok0 + 8 * quad < g.n_tok;  // the warp has a row
    const int w_hi = __shfl_sync(0xffffffffu, pos_hi, 0), w_lo = __shfl_sync(0xffffffffu, pos_lo, 31);
    float m = -INFINITY, l = 0.f;
    for (int64_t u = t0; u < t1; ++u, ++tile) {
      const uint32_t buf = tile & 1;
      if (!wait(&s_full[buf], (tile >> 1) & 1)) break;
      if (tile >= 2 && !wait(&pv_done[buf], ((tile - 2) >> 1) & 1)) break;  // long done: S(i) came after it
      if (live) {
        const int pos = (g.tile0 + (int)(u - cur.begin)) * kPos;
        const uint32_t ts = tmem + lanes + kColS + buf * kPos;
        const bool whole = pos + kPos - 1 <= w_hi && pos >= w_lo;  // every row of the warp sees every position
        const int x0 = pos_lo - pos, x1 = pos_hi - pos;            // columns the row sees
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        uint32_t s0[32], s1[32], s2[32], s3[32];
        tc::ld32(ts, s0);
        tc::ld32(ts + 32, s1);
        tc::ld32(ts + 64, s2);
        tc::ld32(ts + 96, s3);
        tc::wait_ld(s0);
        tc::wait_ld(s1);
        tc::wait_ld(s2);
        tc::wait_ld(s3);
        if (sign != 1.f) {
          sign32(s0, sign);
          sign32(s1, sign);
          sign32(s2, sign);
          sign32(s3, sign);
        }
        if (!whole) {
          uint32_t seen[4] = {seen32(x0, x1, 0), seen32(x0, x1, 32), seen32(x0, x1, 64), seen32(x0, x1, 96)};
          mask32(s0, seen[0]);
          mask32(s1, seen[1]);
          mask32(s2, seen[2]);
          mask32(s3, seen[3]);
        }
        max32(s0, mx);
        max32(s1, mx);
        max32(s2, mx);
        max32(s3, mx);
        float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        mt = mt == -INFINITY || tok >= g.n_tok ? -INFINITY : mt * scale;
        if (u == t0) {
          m = mt;
        } else if (__any_sync(0xffffffffu, mt > m + kRaise)) {
          const float mn = fmaxf(m, mt);
          const float corr = m == -INFINITY ? 0.f : ex2(m - mn);
          m = mn;
          l *= corr;
          // every earlier product is in O before it is rescaled
          if (!wait(&pv_done[buf ^ 1], ((tile - 1) >> 1) & 1)) break;
#pragma unroll 1
          for (int d = 0; d < kHeadDim; d += 32) {
            uint32_t o[32];
            tc::ld32(tmem + lanes + d, o);
            tc::wait_ld(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
            tc::st32(tmem + lanes + d, o);
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        exp32<kSplit>(ts, s0, scale, ref, sum);
        exp32<kSplit>(ts + 32, s1, scale, ref, sum);
        exp32<kSplit>(ts + 64, s2, scale, ref, sum);
        exp32<kSplit>(ts + 96, s3, scale, ref, sum);
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tc::wait_st();
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) arrive_p(buf);
    }
    if (!ok) break;
    // (the next group's fp32 queries are split while this one's last product runs)
    Cursor nxt = cur;
    const bool more = nxt.advance(p, sh, u1);
    if (kSplit && more) split_queries(nxt);
    if (!wait(&pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1)) break;
    const bool split = cur.begin < u0 || cur.end > u1;
    if (live) {
      const int64_t r = cur.seq.q0 + g.tok + tok;
      float* part = p.part + (int64_t)paged::partial_slot(c, cur.begin, total, G) * (RANKS * paged::kChunkPart);
      QT* dst = out + ((r * p.n_kv + cur.j) * kGroup + (row & 3)) * kHeadDim;
      const float inv = 1.0f / l;
      constexpr int kAll = RANKS * kRows;
      // A partial state is [dims / 4][row][4], then the maxima and the sums: the
      // lanes' rows lie next to one another (row by row, 32 lines of 128 bytes
      // per store, the output took 10000 cycles a group).
      auto put = [&](int d, const uint32_t (&o)[32]) {
        if (split) {
          float4* to = reinterpret_cast<float4*>(part) + (d / 4) * kAll + prow;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            to[i * kAll] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                       __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
        } else if constexpr (STAGE) {
          // through the warp's stage, 32 rows of 64 bytes and 16 of padding: a
          // row's dims leave next to one another
          unsigned char* mine = stage + quad * kStageBytes;
          uint4* at = reinterpret_cast<uint4*>(mine + lane * kStageRow);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            at[i] = make_uint4(pack2(__uint_as_float(o[8 * i]) * inv, __uint_as_float(o[8 * i + 1]) * inv),
                               pack2(__uint_as_float(o[8 * i + 2]) * inv, __uint_as_float(o[8 * i + 3]) * inv),
                               pack2(__uint_as_float(o[8 * i + 4]) * inv, __uint_as_float(o[8 * i + 5]) * inv),
                               pack2(__uint_as_float(o[8 * i + 6]) * inv, __uint_as_float(o[8 * i + 7]) * inv));
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = 8 * i + (lane >> 2);  // the warp's row
            const uint4 w = *reinterpret_cast<const uint4*>(mine + rr * kStageRow + (lane & 3) * 16);
            const int t = tok0 + 8 * quad + (rr >> 2);
            if (t < g.n_tok)
              *reinterpret_cast<uint4*>(
                  out + (((cur.seq.q0 + g.tok + t) * (int64_t)p.n_kv + cur.j) * kGroup + (rr & 3)) * kHeadDim + d +
                  (lane & 3) * 8) = w;
          }
          __syncwarp();
        } else if constexpr (!kSplit) {
          if (tok < g.n_tok) store32(dst + d, o, inv);
        }
      };
      uint32_t oa[32], ob[32];
      if (kSplit && !split) {
        // whole rows of fp32: four lanes write 32 bytes of a row at a time
        auto at = [&](int x) { return tmem + lanes + ((uint32_t)(x >> 2) << 20) + (x & 3) * 64; };
        auto rows = [&](int x, const uint32_t (&o)[32]) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int rr = 16 * (x >> 2) + 8 * i + (lane >> 2);  // the warp's row
            const float iv = __shfl_sync(0xffffffffu, inv, rr);
            const int t = tok0 + 8 * quad + (rr >> 2);
            float* to = static_cast<float*>(p.a) +
                        (((cur.seq.q0 + g.tok + t) * (int64_t)p.n_kv + cur.j) * kGroup + (rr & 3)) * kHeadDim +
                        (x & 3) * 64 + 2 * (lane & 3);
            if (t < g.n_tok)
#pragma unroll
              for (int k = 0; k < 8; ++k)
                *reinterpret_cast<float2*>(to + 8 * k) =
                    make_float2(__uint_as_float(o[4 * k + 2 * i]) * iv, __uint_as_float(o[4 * k + 2 * i + 1]) * iv);
          }
        };
        tc::ld16x64(at(0), oa);
#pragma unroll 1
        for (int x = 0; x < 8; x += 2) {
          tc::wait_ld(oa);
          tc::ld16x64(at(x + 1), ob);
          rows(x, oa);
          tc::wait_ld(ob);
          if (x + 2 < 8) tc::ld16x64(at(x + 2), oa);
          rows(x + 1, ob);
        }
      } else {
        tc::ld32(tmem + lanes, oa);
#pragma unroll 1
        for (int d = 0; d < kHeadDim; d += 64) {
          tc::wait_ld(oa);
          tc::ld32(tmem + lanes + d + 32, ob);
          put(d, oa);
          tc::wait_ld(ob);
          if (d + 64 < kHeadDim) tc::ld32(tmem + lanes + d + 64, oa);
          put(d + 32, ob);
        }
      }
      if (split) {
        part[RANKS * kRows * kHeadDim + prow] = m;
        part[RANKS * kRows * (kHeadDim + 1) + prow] = l;
      }
    }
    tc::fence_before();  // O is read before the next group's first product (its P arrives after this)
    if (!more) break;
    cur = nxt;
  }
  if (!ok && lane == 0) {
    if (!flags[0]) atomicOr(p.err, kErrWaitTimeout);
    flags[0] = 1;
  }
  if (st == 0 && rank == 0) {
    // the group that begins in this share and goes on behind it, if any
    paged::Join j = {};
    if (ok && cur.end > u1 && cur.begin >= u0) {
      j.row0 = cur.seq.q0 + cur.g.tok;
      j.n_rows = 4 * cur.g.n_tok;
      j.head = cur.j;
      j.last = paged::cta_at(cur.end - 1, total, G);
      j.begin = cur.begin;
      j.total = total;
      j.G = G;
    }
    p.joins[c] = j;
  }
}

// Join the partial states of the groups that a share's border cut, the parts
// in CTA order: block (share c, 32 rows of the group that begins in it and
// goes on, 256 / kJoinSplit dims).  Lane r has row r, warp w the dims 4 w + 32
// i, so that the reads are the partial states' lines; the rows then go through
// shared memory to be written line by line.  Bound by what an SM takes in from
// L2 where a few groups have many parts (one sequence of 8 tokens at 12000: 26.7
// us with whole rows to a block, 25.0 with halves, 24.1 with quarters, but one
// of 48 at 300 13.8, 14.2 and 15.5), by the states' bytes where there are many
// groups (40 MB for a chunk of 4096 tokens on 76 pairs).  Four parts at a time
// read the last one more often than they hide: 228 against 224 us there.
constexpr int kJoinRows = 32;
constexpr int kJoinWarps = 8;
constexpr int kJoinParts = 2;                         // loaded at a time
constexpr int kJoinSplit = 2;                         // blocks that share a row
constexpr int kJoinWidth = kHeadDim / kJoinSplit;     // dims of a block
constexpr int kJoinDims = kJoinWidth / 4 / kJoinWarps;  // float4 of a thread
constexpr int kJoinStride = kJoinWidth + 4;           // floats of a row in shared memory
static_assert(kJoinDims >= 1, "a float4 a thread at least");

template <typename QT, int RANKS>
__global__ void __launch_bounds__(32 * kJoinWarps) k_paged_join(const __grid_constant__ Args p) {
  __shared__ float4 rows[kJoinRows * kJoinStride / 4];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.y * kJoinRows, row = row0 + lane, d0 = blockIdx.z * kJoinWidth;
  const paged::Join* jp = p.joins + c;
  const int4 a = __ldcg(reinterpret_cast<const int4*>(jp));  // row0, n_rows, head, last
  if (row0 >= a.y) return;
  const longlong2 bt = __ldcg(reinterpret_cast<const longlong2*>(jp) + 1);  // begin, total
  const int G = __ldcg(&jp->G), last = a.w;
  constexpr int kAll = RANKS * kRows;
  float M = -INFINITY, L = 0.f;
  float4 O[kJoinDims];
#pragma unroll
  for (int i = 0; i < kJoinDims; ++i) O[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  // (the first part's slot depends on where the group begins, the others are
  // their CTAs' first)
  const int first = paged::partial_slot(c, bt.x, bt.y, G);
#pragma unroll 1
  for (int q0 = c; q0 <= last; q0 += kJoinParts) {
    float m[kJoinParts], l[kJoinParts];
    float4 x[kJoinParts][kJoinDims];
#pragma unroll
    for (int t = 0; t < kJoinParts; ++t) {
      // (behind the last part the last once more, at weight 0: loads without
      // a condition stay in flight together)
      const int q = min(q0 + t, last), slot = q == c ? first : 2 * q;
      const float* part = p.part + (int64_t)slot * (RANKS * paged::kChunkPart);
      m[t] = __ldcg(part + kAll * kHeadDim + row);
      l[t] = __ldcg(part + kAll * (kHeadDim + 1) + row);
#pragma unroll
      for (int i = 0; i < kJoinDims; ++i)
        x[t][i] = __ldcg(reinterpret_cast<const float4*>(part) + (d0 / 4 + warp + kJoinWarps * i) * kAll + row);
      if (q0 + t > last) m[t] = -INFINITY;
    }
#pragma unroll
    for (int t = 0; t < kJoinParts; ++t) {
      const float mn = fmaxf(M, m[t]);
      // (a part in which the row saw nothing holds no state)
      const float s = M == -INFINITY ? 0.f : exp2f(M - mn), r = m[t] == -INFINITY ? 0.f : exp2f(m[t] - mn);
      M = mn;
      L = L * s + l[t] * r;
#pragma unroll
      for (int i = 0; i < kJoinDims; ++i)
        if (r != 0.f || s != 1.f) {
          O[i].x = O[i].x * s + x[t][i].x * r;
          O[i].y = O[i].y * s + x[t][i].y * r;
          O[i].z = O[i].z * s + x[t][i].z * r;
          O[i].w = O[i].w * s + x[t][i].w * r;
        }
    }
  }
  const float inv = 1.0f / L;
#pragma unroll
  for (int i = 0; i < kJoinDims; ++i)
    rows[lane * (kJoinStride / 4) + warp + kJoinWarps * i] =
        make_float4(O[i].x * inv, O[i].y * inv, O[i].z * inv, O[i].w * inv);
  __syncthreads();
  // 8 dims a thread
  constexpr int kThreadsRow = kJoinWidth / 8;
  for (int e = threadIdx.x; e < kJoinRows * kThreadsRow; e += 32 * kJoinWarps) {
    const int r = e / kThreadsRow, d = 8 * (e % kThreadsRow);
    if (row0 + r >= a.y) break;
    const float4 x = rows[r * (kJoinStride / 4) + d / 4], y = rows[r * (kJoinStride / 4) + d / 4 + 1];
    QT* dst = static_cast<QT*>(p.a) + (((int64_t)a.x + ((row0 + r) >> 2)) * p.n_kv + a.z) * (kGroup * kHeadDim) +
              ((row0 + r) & 3) * kHeadDim + d0 + d;
    if constexpr (std::is_same<QT, float>::value) {
      reinterpret_cast<float4*>(dst)[0] = x;
      reinterpret_cast<float4*>(dst)[1] = y;
    } else {
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack2(x.x, x.y), pack2(x.z, x.w), pack2(y.x, y.y), pack2(y.z, y.w));
    }
  }
}

// A pool [rows][n_kv][256] bf16 as the chunk kernels load it: boxes of `lines`
// lines of `box` rows of one KV head (kAtom's layout).  Its dimensions are a
// line's elements, the row of a group, the line, the group, the head.
inline bool make_chunk_map(CUtensorMap* map, const void* base, int n_kv, int64_t rows, int box, int lines) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t row = (cuuint64_t)n_kv * kHeadDim * 2;
  const cuuint64_t dims[5] = {64, 8, 4, (cuuint64_t)rows / 8, (cuuint64_t)n_kv};
  const cuuint64_t strides[4] = {row, 128, 8 * row, kHeadDim * 2};
  const cuuint32_t shape[5] = {64, 8, (cuuint32_t)lines, (cuuint32_t)box / 8, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, shape, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace chunk
}  // namespace spark
