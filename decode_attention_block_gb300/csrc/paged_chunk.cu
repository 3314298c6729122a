// paged_chunk.cu -- attention of chunks of new tokens over a paged bf16 cache
// on the tensor cores (tcgen05, accumulators in tensor memory).
//
// A group is up to 32 consecutive tokens of one sequence with one KV head:
// their 4 x 32 query heads are the 128 rows of one MMA tile, row 4 t + h.  Per
// tile of 128 positions
//   S = Q K^T          128 x 128, K = 256 dims, both operands in shared memory
//   P = e^(S - m)      in registers, one row per thread
//   O += P V           128 x 256, P from tensor memory, V as it lies in its
//                      pages (positions are the MMA's K dimension)
// with a running maximum m and sum per row.  m is only raised when a row's
// scores pass it by 2^8: the products and the sum share whatever m is, so the
// result does not change, and O is rescaled a few times per row, not per tile.
//
// Precision: bf16 queries meet P rounded to bf16 (as the output is); fp32
// queries are carried as two bf16 halves (both multiplied against the same
// K), and so is P: 16 significant bits each, fp32 sums.
//
// Tensor memory (512 columns): O 256, two buffers of 128 for S; P overwrites
// its own S, 32 positions at a time (hi in the first 16 of their columns, lo
// in the others).  Shared memory: Q
// (64 KB, 128 KB in two halves) and a ring of 32 KB slots, each 128 positions
// x 128 dims of K or V.  Warp 0 fills the ring (TMA boxes of the part of a
// page inside the tile), warp 1 issues the MMAs in the order S(i+1), P V(i),
// so the tensor cores run S(i+1) while warps 2-5 turn S(i) into P(i).
//
// Work is the flat list of paged.h (128-position tiles), every CTA an equal
// share: a group cut by a share's border leaves fp32 partial states, joined
// in CTA order by k_paged_join.
#include <math.h>

#include <type_traits>

#include "launch.h"
#include "paged_launch.h"
#include "paged_parts.cuh"
#include "tmem.cuh"

namespace spark {
namespace {

using paged::Args;
using paged::Cursor;
using paged::Shape;

constexpr int kRows = 128;                      // rows of a group: 32 tokens x 4 heads
constexpr int kPos = 128;                       // positions of a tile
constexpr int kThreads = 192;
constexpr int kSoft = 128;                      // softmax threads, one row each
constexpr uint32_t kLineBytes = kPos * 128;     // 64 dims of 128 rows or positions
constexpr uint32_t kSlot = 2 * kLineBytes;      // 128 dims
constexpr uint32_t kQBytes = 4 * kLineBytes;
constexpr uint32_t kCols = 512;
constexpr uint32_t kColS = 256;                 // first column of S buffer 0; O starts at 0
constexpr float kRaise = 8.0f;                  // m is raised once a score passes it by 2^8
constexpr int kMinTiles = 2;                    // tiles per CTA at least

static_assert(kRows == kGroup * paged::kChunkTokens, "a row per query head of a token");

// Q halves and ring slots: 224 KB either way
template <bool SPLIT>
struct ChunkSmem {
  static constexpr int kQ = SPLIT ? 2 : 1;
  static constexpr int kSlots = SPLIT ? 3 : 5;
  static constexpr uint32_t kRing = kQ * kQBytes;
  static constexpr uint32_t kBars = kRing + kSlots * kSlot;
  static constexpr uint32_t kBytes = kBars + 8 * (2 * kSlots + 8) + 32;
  static constexpr uint32_t kAlloc = kBytes + 1024;  // slack to align the base (128-byte swizzle)
};
static_assert(ChunkSmem<true>::kAlloc <= 232448 && ChunkSmem<false>::kAlloc <= 232448, "227 KB per CTA");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) { return ffma2(a, make_float2(1.f, 1.f), b); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// eight elements of a query row, the sign of a negative scale folded in, as
// bf16 (and the remainders, for fp32 queries)
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

// The group's queries into shared memory: 64-dim lines of 128 rows, 16-byte
// chunk c of row r at c ^ (r % 8) (the 128-byte swizzle).  Rows behind the
// last token are zero.
template <typename QT>
__device__ __forceinline__ void load_queries(unsigned char* q_s, const Args& p, const Cursor& cur, bool flip, int tid) {
  const QT* q = static_cast<const QT*>(p.q) + (int64_t)cur.j * kGroup * kHeadDim;
  const int64_t row0 = cur.seq.q0 + cur.g.tok;
  constexpr int kBatch = 8;  // rows in flight per warp
  const int ch = tid & 31;
  for (int r0 = tid >> 5; r0 < kRows; r0 += 4 * kBatch) {
    uint4 v[kBatch][sizeof(QT) / 2];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + 4 * i;
      const bool in = (r >> 2) < cur.g.n_tok;
      const uint4* src = reinterpret_cast<const uint4*>(q + (row0 + (r >> 2)) * p.q_ld + (r & 3) * kHeadDim + 8 * ch);
#pragma unroll
      for (int k = 0; k < (int)sizeof(QT) / 2; ++k) v[i][k] = in ? __ldcg(src + k) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + 4 * i;
      const uint32_t at = (uint32_t)(ch >> 3) * kLineBytes + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
      if constexpr (std::is_same<QT, float>::value) {
        float x[8];
        const float s = flip ? -1.f : 1.f;
        const uint32_t w[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = s * __uint_as_float(w[k]);
        uint4 hi, lo;
        split8(x, hi, lo);
        *reinterpret_cast<uint4*>(q_s + at) = hi;
        *reinterpret_cast<uint4*>(q_s + kQBytes + at) = lo;
      } else {
        uint4 w = v[i][0];
        const uint32_t f = flip ? 0x80008000u : 0u;
        w.x ^= f; w.y ^= f; w.z ^= f; w.w ^= f;
        *reinterpret_cast<uint4*>(q_s + at) = w;
      }
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMAs read it through the async proxy
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
template <bool EDGE, bool SPLIT>
__device__ __forceinline__ void exp32(uint32_t ts, const uint32_t (&s)[32], float scale, float ref, uint32_t seen,
                                      float2 (&sum)[2]) {
  uint32_t hi[16], lo[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 t = ffma2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])),
                           make_float2(scale, scale), make_float2(-ref, -ref));
    float2 e = make_float2(ex2(t.x), ex2(t.y));
    if (EDGE) {
      e.x = ((seen >> (2 * i)) & 1u) ? e.x : 0.f;
      e.y = ((seen >> (2 * i + 1)) & 1u) ? e.y : 0.f;
    }
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

template <bool EDGE>
__device__ __forceinline__ void max32(const uint32_t (&s)[32], uint32_t seen, float (&mx)[4]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x = !EDGE || ((seen >> (i + k)) & 1u) ? __uint_as_float(s[i + k]) : -INFINITY;
      const float y = !EDGE || ((seen >> (i + k + 4)) & 1u) ? __uint_as_float(s[i + k + 4]) : -INFINITY;
      mx[k] = fmaxf(mx[k], fmaxf(x, y));
    }
}

// 32 output dims of a row
// 32 output dims of a row
__device__ __forceinline__ void store32(float* dst, const uint32_t (&o)[32], float inv) {
#pragma unroll
  for (int i = 0; i < 32; i += 4)
    reinterpret_cast<float4*>(dst)[i / 4] = make_float4(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv,
                                                        __uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv);
}
__device__ __forceinline__ void store32(__nv_bfloat16* dst, const uint32_t (&o)[32], float inv) {
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = pack2(__uint_as_float(o[i + 2 * k]) * inv, __uint_as_float(o[i + 2 * k + 1]) * inv);
    reinterpret_cast<uint4*>(dst)[i / 8] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <typename QT>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_chunk(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ Args p, int box) {
  constexpr bool kSplit = std::is_same<QT, float>::value;
  using S = ChunkSmem<kSplit>;
  constexpr int NS = S::kSlots;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(base + S::kBars);
  uint64_t* empty = full + NS;
  uint64_t* s_full = empty + NS;   // [2] S(i) is in its buffer
  uint64_t* p_full = s_full + 2;   // [2] P(i) is
  uint64_t* pv_done = p_full + 2;  // [2] P(i) V(i) is in O (one per buffer: a thread waits for each phase, none is skipped)
  uint64_t* q_full = pv_done + 2;
  uint64_t* drained = q_full + 1;  // every MMA has completed
  volatile int* flags = reinterpret_cast<volatile int*>(drained + 1);  // [0] abort
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 2);

  // (the warp's number, and below the MMA warp's loop bounds, by way of a
  // shuffle: known to be the same in every lane, they and what follows from
  // them stay in uniform registers, where an MMA takes its operands from)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], kSoft);
      mbar_init(&pv_done[b], 1);
    }
    mbar_init(q_full, kSoft);
    mbar_init(drained, 1);
    flags[0] = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  // tables, lengths, rows and queries may come from the kernel before
  pdl_wait();
  pdl_trigger();
  const Shape sh{paged::kChunkTokens, kPos, p.window};
  // the ring is not in use yet: room for the prefix sums
  int64_t* prefix = reinterpret_cast<int64_t*>(base + S::kRing);
  paged::work_prefix<kThreads>(p, sh, prefix, prefix + SPARK_MAX_BATCH + 2);
  const int64_t total = prefix[p.n_seqs];
  const int c = blockIdx.x;
  const int G = total > 0 ? paged::ctas_for(total, kMinTiles, gridDim.x) : 0;
  if (c >= G) {
    if (tid == 0) p.joins[c].n_rows = 0;
    return;
  }
  const int64_t u0 = paged::share_begin(total, G, c), u1 = paged::share_begin(total, G, c + 1);
  Cursor cur;
  cur.seek(p, sh, prefix, u0);
  if (warp == 1) tc::alloc(tmem_slot, kCols);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the prefix sums make way for TMA's writes
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp == 0) {
    // ---- producer: K(0), then K(i), V(i - 1) for the tiles of each group
    uint32_t k = 0;
    bool ok = true;
    const int per = kPos / box;  // boxes of a tile
    auto slot = [&](const CUtensorMap* map, int half, int z, int b0, int b1) {
      const int s = (int)(k % NS);
      const uint32_t r = k / NS;
      if (ok && r > 0 && !mbar_wait_bounded(&empty[s], (r - 1) & 1, flags, kWaitLimitNs)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      const int n = b1 - b0;
      if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(2 * n * box) * 128u);
      __syncwarp();
      // lane: (line of the half, box); z is the row of the lane's box
      if (lane < 2 * per) {
        const int b = lane % per, line = lane / per;
        if (b >= b0 && b < b1)
          tma_load_4d(base + S::kRing + s * kSlot + line * kLineBytes + b * box * 128, map, &full[s], 0, z,
                      2 * half + line, cur.j);
      }
      ++k;
    };
    for (;;) {
      const int64_t t0 = cur.begin > u0 ? cur.begin : u0, t1 = cur.end < u1 ? cur.end : u1;
      // the boxes [b0, b1) of tile u that hold rows the group reads; the table's
      // entry for the lane's box, asked for one tile ahead
      auto boxes = [&](int64_t u, int& pos, int& b0, int& b1) {
        pos = (cur.g.tile0 + (int)(u - cur.begin)) * kPos;
        b0 = cur.g.lo > pos ? (cur.g.lo - pos) / box : 0;
        b1 = cur.g.hi - pos >= kPos ? per : (cur.g.hi - pos) / box + 1;
      };
      auto entry = [&](int64_t u) {
        int pos, b0, b1;
        boxes(u, pos, b0, b1);
        const int b = lane % per;
        return b >= b0 && b < b1 ? paged::page_entry(p, cur.s, paged::page_col(pos + b * box, p.page_size)) : 0;
      };
      int z_v = 0, v0 = 0, v1 = 0;  // the tile before
      int ahead = entry(t0);
      for (int64_t u = t0; u <= t1 && ok; ++u) {
        int z = 0, b0 = 0, b1 = 0;
        if (u < t1) {
          int pos;
          boxes(u, pos, b0, b1);
          z = paged::page_of(p, ahead) * p.page_size + paged::page_row(pos + (lane % per) * box, p.page_size);
          if (u + 1 < t1) ahead = entry(u + 1);
          slot(&tm_k, 0, z, b0, b1);
          slot(&tm_k, 1, z, b0, b1);
        }
        if (u > t0) {
          slot(&tm_v, 0, z_v, v0, v1);
          slot(&tm_v, 1, z_v, v0, v1);
        }
        z_v = z;
        v0 = b0;
        v1 = b1;
      }
      if (!ok || cur.end >= u1) break;
      cur.next(p, sh);
    }
    if (!ok && lane == 0) {
      if (!flags[0]) atomicOr(p.err, kErrWaitTimeout);
      flags[0] = 1;
    }
    if (flags[0]) {
      // let the copies in flight land before the CTA can exit
      int never = 0;
      for (uint32_t i = k > (uint32_t)NS ? k - NS : 0; i < k; ++i)
        mbar_wait_bounded(&full[i % NS], (i / NS) & 1, &never, kWaitLimitNs);
    }
  } else if (warp == 1) {
    // ---- MMA issuer (one elected lane); the whole warp clears the rows of V tiles that
    // no token of the group sees (their P is 0, but they may hold anything)
    constexpr uint32_t kIdS = tc::idesc(kRows, kPos, false), kIdO = tc::idesc(kRows, kPos, true);
    const uint32_t q_addr = smem_u32(base), ring = smem_u32(base + S::kRing);
    uint32_t k = 0, tile = 0, item = 0;
    bool ok = true;
    const bool one = tc::elect();
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, flags, kWaitLimitNs));
      tc::fence_after();
      return ok;
    };
    auto scores = [&](uint32_t i) {
      const uint32_t d = tmem + kColS + (i & 1) * kPos;
#pragma unroll
      for (int half = 0; half < 2; ++half, ++k) {
        const int s = (int)(k % NS);
        if (!wait(&full[s], (k / NS) & 1)) return;
        const uint64_t b0 = tc::desc_k_major(ring + s * kSlot), a0 = tc::desc_k_major(q_addr + 2 * half * kLineBytes);
        if (one) {
#pragma unroll
          for (int line = 0; line < 2; ++line)
#pragma unroll
            for (int part = 0; part < S::kQ; ++part)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                tc::mma_ss(d, a0 + ((part * kQBytes + line * kLineBytes) >> 4) + 2 * ks,
                           b0 + (line * kLineBytes >> 4) + 2 * ks, kIdS, half + line + part + ks > 0);
          tc::commit(&empty[s]);
          if (half == 1) tc::commit(&s_full[i & 1]);
        }
        __syncwarp();
      }
    };
    auto values = [&](uint32_t i, bool first, int r0, int r1) {
      const uint32_t a = tmem + kColS + (i & 1) * kPos;
      if (!wait(&p_full[i & 1], (i >> 1) & 1)) return;
#pragma unroll
      for (int half = 0; half < 2; ++half, ++k) {
        const int s = (int)(k % NS);
        if (!wait(&full[s], (k / NS) & 1)) return;
        if (r0 > 0 || r1 < kPos) {
          unsigned char* v = base + S::kRing + s * kSlot;
          // 16 lanes clear a row's two lines
          for (int r = lane >> 4; r < kPos; r += 2)
            if (r < r0 || r >= r1)
              *reinterpret_cast<uint4*>(v + ((lane >> 3) & 1) * kLineBytes + r * 128 + (lane & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        const uint64_t b0 = tc::desc_mn_major(ring + s * kSlot, kLineBytes);
        const uint32_t d = tmem + half * 128;
        if (one) {
#pragma unroll
          for (int part = 0; part < S::kQ; ++part)
#pragma unroll
            for (int ks = 0; ks < kPos / 16; ++ks)  // 16 positions: two 8-row groups, eight columns of P
              tc::mma_ts(d, a + (ks >> 1) * 32 + part * 16 + (ks & 1) * 8, b0 + ks * (2048 >> 4), kIdO,
                         !first || part + ks > 0);
          tc::commit(&empty[s]);
          if (half == 1) tc::commit(&pv_done[i & 1]);
        }
        __syncwarp();
      }
    };
    for (;;) {
      const int64_t t0 = cur.begin > u0 ? cur.begin : u0, t1 = cur.end < u1 ? cur.end : u1;
      const int n = __shfl_sync(0xffffffffu, (int)(t1 - t0), 0);  // tiles of the group in this share
      const int pos0 = __shfl_sync(0xffffffffu, (cur.g.tile0 + (int)(t0 - cur.begin)) * kPos, 0);
      const int lo = __shfl_sync(0xffffffffu, cur.g.lo, 0), hi = __shfl_sync(0xffffffffu, cur.g.hi, 0);
      if (!wait(q_full, item & 1)) break;
      ++item;
      for (int i = 0; i <= n && ok; ++i) {
        if (i < n) scores(tile + i);
        if (i > 0 && ok) {
          const int pos = pos0 + (i - 1) * kPos;
          values(tile + i - 1, i == 1, lo > pos ? lo - pos : 0, hi + 1 - pos < kPos ? hi + 1 - pos : kPos);
        }
      }
      tile += n;
      if (!ok || __shfl_sync(0xffffffffu, (int)(cur.end >= u1), 0)) break;
      cur.next(p, sh);
    }
    if (one) {
      if (!ok) {
        if (!flags[0]) atomicOr(p.err, kErrWaitTimeout);
        flags[0] = 1;
      }
      // every MMA has ended before tensor and shared memory are let go
      int never = 0;
      tc::commit(drained);
      mbar_wait_bounded(drained, 0, &never, kWaitLimitNs);
    }
    __syncwarp();
  } else {
    // ---- softmax: one row per thread
    const int quad = warp & 3, st = tid - 64;
    const int row = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const bool flip = p.scale_log2 < 0.f;
    const float scale = fabsf(p.scale_log2);
    QT* out = static_cast<QT*>(p.a);
    uint32_t tile = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, flags, kWaitLimitNs));
      tc::fence_after();
      return ok;
    };
    load_queries<QT>(base, p, cur, flip, st);
    mbar_arrive(q_full);
    for (;;) {
      const int64_t t0 = cur.begin > u0 ? cur.begin : u0, t1 = cur.end < u1 ? cur.end : u1;
      const paged::Group g = cur.g;
      const int tok = row >> 2;
      // positions the row sees; rows behind the last token take the last one's
      const int pos_hi = cur.seq.p0 + g.tok + (tok < g.n_tok ? tok : g.n_tok - 1);
      const int pos_lo = p.window > 0 && pos_hi + 1 > p.window ? pos_hi + 1 - p.window : 0;
      const bool live = 8 * quad < g.n_tok;  // the warp has a row
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
          // a whole tile's scores stay in registers; a masked one (a group's
          // last, or its first behind a window) is read twice by a short loop
          uint32_t s0[32], s1[32], s2[32], s3[32];
          if (whole) {
            tc::ld32(ts, s0);
            tc::ld32(ts + 32, s1);
            tc::ld32(ts + 64, s2);
            tc::ld32(ts + 96, s3);
            tc::wait_ld(s0);
            tc::wait_ld(s1);
            tc::wait_ld(s2);
            tc::wait_ld(s3);
            max32<false>(s0, 0, mx);
            max32<false>(s1, 0, mx);
            max32<false>(s2, 0, mx);
            max32<false>(s3, 0, mx);
          } else {
#pragma unroll 1
            for (int ch = 0; ch < kPos; ch += 32) {
              tc::ld32(ts + ch, s0);
              tc::wait_ld(s0);
              max32<true>(s0, seen32(x0, x1, ch), mx);
            }
          }
          float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          mt = mt == -INFINITY ? mt : mt * scale;
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
          if (whole) {
            exp32<false, kSplit>(ts, s0, scale, ref, 0, sum);
            exp32<false, kSplit>(ts + 32, s1, scale, ref, 0, sum);
            exp32<false, kSplit>(ts + 64, s2, scale, ref, 0, sum);
            exp32<false, kSplit>(ts + 96, s3, scale, ref, 0, sum);
          } else {
#pragma unroll 1
            for (int ch = 0; ch < kPos; ch += 32) {
              tc::ld32(ts + ch, s0);
              tc::wait_ld(s0);
              exp32<true, kSplit>(ts + ch, s0, scale, ref, seen32(x0, x1, ch), sum);
            }
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tc::wait_st();
        }
        tc::fence_before();
        mbar_arrive(&p_full[buf]);
      }
      if (!ok) break;
      // Q is free (the last S is done): the next group's queries load while
      // this one's last product runs
      Cursor nxt = cur;
      const bool more = cur.end < u1;
      if (more) {
        nxt.next(p, sh);
        load_queries<QT>(base, p, nxt, flip, st);
        mbar_arrive(q_full);
      }
      if (!wait(&pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1)) break;
      const bool split = cur.begin < u0 || cur.end > u1;
      if (live) {
        const int64_t r = cur.seq.q0 + g.tok + tok;
        float* part = p.part + (int64_t)paged::partial_slot(c, cur.begin, total, G) * paged::kChunkPart;
        QT* dst = out + ((r * p.n_kv + cur.j) * kGroup + (row & 3)) * kHeadDim;
        const float inv = 1.0f / l;
#pragma unroll 1
        for (int d = 0; d < kHeadDim; d += 32) {
          uint32_t o[32];
          tc::ld32(tmem + lanes + d, o);
          tc::wait_ld(o);
          if (tok < g.n_tok) {
            if (split)
              store32(part + row * kHeadDim + d, o, 1.0f);
            else
              store32(dst + d, o, inv);
          }
        }
        if (split) {
          part[kRows * kHeadDim + row] = m;
          part[kRows * kHeadDim + kRows + row] = l;
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
    if (st == 0) {
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
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tmem, kCols);
  }
}

// Join the partial states of the groups that a share's border cut: block
// (share c, 8 rows of the group that begins in it and goes on), one row per
// warp, eight dims per lane, the parts in CTA order.
constexpr int kJoinRows = 8;

template <typename QT>
__global__ void __launch_bounds__(32 * kJoinRows) k_paged_join(const __grid_constant__ Args p) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.y * kJoinRows + warp;
  if (row >= __ldcg(&p.joins[c].n_rows)) return;
  const int last = __ldcg(&p.joins[c].last), G = __ldcg(&p.joins[c].G);
  const int64_t begin = __ldcg(&p.joins[c].begin), total = __ldcg(&p.joins[c].total);
  float M = -INFINITY, L = 0.f, O[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) O[i] = 0.f;
  for (int q = c; q <= last; ++q) {
    const float* part = p.part + (int64_t)paged::partial_slot(q, begin, total, G) * paged::kChunkPart;
    const float m = __ldcg(part + kRows * kHeadDim + row), l = __ldcg(part + kRows * kHeadDim + kRows + row);
    const float4* src = reinterpret_cast<const float4*>(part + row * kHeadDim + 8 * lane);
    const float4 x = __ldcg(src), y = __ldcg(src + 1);
    const float mn = fmaxf(M, m);
    const float a = M == -INFINITY ? 0.f : exp2f(M - mn), b = m == -INFINITY ? 0.f : exp2f(m - mn);
    M = mn;
    L = L * a + l * b;
    O[0] = O[0] * a + x.x * b; O[1] = O[1] * a + x.y * b; O[2] = O[2] * a + x.z * b; O[3] = O[3] * a + x.w * b;
    O[4] = O[4] * a + y.x * b; O[5] = O[5] * a + y.y * b; O[6] = O[6] * a + y.z * b; O[7] = O[7] * a + y.w * b;
  }
  const float inv = 1.0f / L;
  const int64_t r = __ldcg(&p.joins[c].row0) + (row >> 2);
  QT* dst = static_cast<QT*>(p.a) + ((r * p.n_kv + __ldcg(&p.joins[c].head)) * kGroup + (row & 3)) * kHeadDim + 8 * lane;
  if constexpr (std::is_same<QT, float>::value) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(O[0] * inv, O[1] * inv, O[2] * inv, O[3] * inv);
    reinterpret_cast<float4*>(dst)[1] = make_float4(O[4] * inv, O[5] * inv, O[6] * inv, O[7] * inv);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack2(O[0] * inv, O[1] * inv), pack2(O[2] * inv, O[3] * inv),
                                                pack2(O[4] * inv, O[5] * inv), pack2(O[6] * inv, O[7] * inv));
  }
}

// A pool [rows][n_kv][256] bf16 as the chunk kernel loads it: boxes of one
// 128-byte line of `box` rows of one KV head.
bool make_chunk_map(CUtensorMap* map, const void* base, int n_kv, int64_t rows, int box) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[4] = {64, (cuuint64_t)rows, 4, (cuuint64_t)n_kv};
  const cuuint64_t strides[3] = {(cuuint64_t)n_kv * kHeadDim * 2, 128, kHeadDim * 2};
  const cuuint32_t shape[4] = {64, (cuuint32_t)box, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, shape, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename QT>
cudaError_t launch_chunk(const Args& p, const void* k, const void* v, cudaStream_t st) {
  using S = ChunkSmem<std::is_same<QT, float>::value>;
  int box = kPos;  // the largest box that divides both a tile and a page
  while (p.page_size % box != 0) box /= 2;
  CUtensorMap mk, mv;
  const int64_t rows = (int64_t)p.n_pages * p.page_size;
  if (!make_chunk_map(&mk, k, p.n_kv, rows, box) || !make_chunk_map(&mv, v, p.n_kv, rows, box))
    return cudaErrorInvalidValue;
  auto kern = k_paged_chunk<QT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kAlloc);
  if (e != cudaSuccess) return e;
  int grid = device_sm_count();
  if (grid > paged::kMaxChunkCtas) grid = paged::kMaxChunkCtas;
  e = launch_pdl(kern, dim3(grid), dim3(kThreads), S::kAlloc, st, mk, mv, p, box);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_paged_join<QT>, dim3(grid, kRows / kJoinRows), dim3(32 * kJoinRows), 0, st, p);
}

}  // namespace

cudaError_t launch_paged_chunk(const paged::Args& p, int qdtype, const void* k, const void* v, cudaStream_t st) {
  return qdtype == SPARK_BF16 ? launch_chunk<__nv_bfloat16>(p, k, v, st) : launch_chunk<float>(p, k, v, st);
}

}  // namespace spark
