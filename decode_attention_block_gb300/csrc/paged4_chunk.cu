// paged4_chunk.cu -- attention of chunks of new tokens over 4-bit pages on the
// tensor cores: paged_chunk.cu with fp16 operands, K and V converted from codes
// by eight warps on their way into shared memory.
//
// Groups, rows, tensor memory, softmax, joins and precision as there, with fp16
// in place of bf16: an element of K or V is an fp16 number as it is, queries are
// scaled row by row by a power of two (fp32 ones as two fp16 halves), and
// probabilities are fp16 (fp32 queries: two halves).  Warp 0 loads the queries,
// which warps 4-7 (softmax) convert, warp 1 issues the MMAs, warps 8-15 fill
// the ring, warp 8 + w with positions 16 w .. + 15 of a tile.
// Rows of V that no token of the group sees are stored as zeros.
//
// Bound by shared memory: a tile's operands are written (128 KB) and read by the
// MMAs (192 KB; 384 with fp32 queries), 2560 cycles at 128 bytes a cycle against
// 2048 of MMA, and the codes' loads go through the same pipe.  32 sequences at
// 4096-8192 (0.23 GB), bf16 queries: 4 tokens each 98 us, 32 tokens 113 (bf16 pages,
// 0.82 GB: 132 and 147); fp32 queries 166; a mixed batch of 32, 4 of them with
// chunks of ~400 tokens, 135 and 226 (bf16 pages 107 and 131 to 141).  What it cost
// on the way (4 tokens each): half lines of codes a load 15 more, scores kept in 240
// registers a thread, the MMA warp spilling, 4.  As it is ptxas spills 48 bytes of a
// thread with bf16 queries, 368 with fp32 ones (on pairs 496); by which warps is not
// known, nor what it costs.
#include "paged4_chunk_parts.cuh"

namespace spark {
namespace {

using namespace chunk4;

constexpr int kMinUnits4 = 1;

// Q halves and ring slots: 224 KB either way
template <bool SPLIT>
struct Chunk4Smem {
  static constexpr int kQ = SPLIT ? 2 : 1;
  static constexpr uint32_t kQLine = kQ * kLineBytes;  // a line of the queries, with that of the remainders
  static constexpr int kSlots = SPLIT ? 3 : 5;
  static constexpr int kLead = SPLIT ? 2 : 1;  // a group's cost beyond its tiles, in tiles
  static constexpr uint32_t kRing = kQ * kQBytes;
  static constexpr uint32_t kBars = kRing + kSlots * kSlot;
  static constexpr uint32_t kBytes = kBars + 8 * (2 * kSlots + 10) + 32;
  static constexpr uint32_t kAlloc = kBytes + 1024;  // slack to align the base (128-byte swizzle)
};
static_assert(Chunk4Smem<true>::kAlloc <= 232448 && Chunk4Smem<false>::kAlloc <= 232448, "227 KB per CTA");
static_assert(kSlot >= 8 * (SPARK_MAX_BATCH + 2 + kThreads4 / 16), "room for the prefix sums");

template <typename QT>
__global__ void __launch_bounds__(kThreads4, 1)
    k_paged4_chunk(const unsigned char* pk, const unsigned char* pv, const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_q8, const __grid_constant__ Args p) {
  constexpr bool kSplit = std::is_same<QT, float>::value;
  using S = Chunk4Smem<kSplit>;
  constexpr int NS = S::kSlots;
  using R = Regs<120, 152, 120>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(base + S::kBars);
  uint64_t* empty = full + NS;
  uint64_t* s_full = empty + NS;   // [2] S(i) is in its buffer
  uint64_t* p_full = s_full + 2;   // [2] P(i) is
  uint64_t* pv_done = p_full + 2;  // [2] P(i) V(i) is in O
  uint64_t* q_full = pv_done + 2;
  uint64_t* q_raw = q_full + 1;    // they have landed, not yet fp16
  uint64_t* q_empty = q_raw + 1;   // the group's last S is done
  uint64_t* drained = q_empty + 1;  // every MMA has completed
  volatile int* flags = reinterpret_cast<volatile int*>(drained + 1);  // [0] abort
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 2);

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], kDequant);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], kSoft / 32);
      mbar_init(&pv_done[b], 1);
    }
    mbar_init(q_full, kSoft / 32);
    mbar_init(q_raw, 1);
    mbar_init(q_empty, 1);
    mbar_init(drained, 1);
    flags[0] = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_q8);
  }
  // tables, lengths, rows and queries may come from the kernel before
  pdl_wait();
  pdl_trigger();
  const Shape sh{paged::kChunkTokens, kPos, p.window, S::kLead};
  // the ring is not in use yet: room for the prefix sums
  int64_t* prefix = reinterpret_cast<int64_t*>(base + S::kRing);
  const int c = blockIdx.x;
  paged::Share share;
  if (!paged::find_share<kThreads4>(p, sh, c, kMinUnits4, gridDim.x, prefix, share)) {
    if (tid == 0) p.joins[c].n_rows = 0;
    return;
  }
  const int64_t total = share.total, u0 = share.u0, u1 = share.u1;
  const int G = share.G;
  Cursor cur = share.cur;
  if (warp == 1) tc::alloc(tmem_slot, kCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp >= kFirstDequant) {
    // ---- K(0), then K(i), V(i - 1) for the tiles of each group, a half of the dims
    // a slot: warp 8 + w positions 16 w .. 16 w + 15, one block
    fewer_registers<R::kDequant>();
    const int w = warp - kFirstDequant;
    int s0 = 0;           // the next slot, and the one behind it
    uint32_t turn = 1;    // parity to wait for in s0: the first time round it is free
    bool ok = true;
    const RowLanes in_k(pk, lane), in_v(pv, lane);
    // the lane's line in a slot
    const uint32_t line = smem_u32(base + S::kRing) + 2 * w * kGroupBytes<2> + in_k.line * kAtom;
    auto store = [&](const RowPart (&x)[4]) {
      const int s1 = s0 + 1 < NS ? s0 + 1 : 0;
      const uint32_t turn1 = s0 + 1 < NS ? turn : turn ^ 1u;
      ok = __all_sync(0xffffffffu, ok && mbar_wait_bounded(&empty[s0], turn, flags, kWaitLimitNs) &&
                                       mbar_wait_bounded(&empty[s1], turn1, flags, kWaitLimitNs));
      if (!ok) return;
      const uint32_t to = line + (in_k.h ? s1 : s0) * kSlot;
#pragma unroll
      for (int u = 0; u < 4; ++u) store_rows(to + ((u & 1) ? in_k.at1 : in_k.at0) + (u >> 1) * kGroupBytes<2>, x[u]);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMAs read it through the async proxy
      __syncwarp();
      if (lane < 2) mbar_arrive(&full[lane ? s1 : s0]);
      s0 = s1 + 1 < NS ? s1 + 1 : 0;
      turn = s1 + 1 < NS ? turn1 : turn1 ^ 1u;
    };
    auto load = [&](RowPart (&x)[4], const RowLanes& l, uint32_t at) {
      load_rows<0>(x[0], l, at);
      load_rows<1>(x[1], l, at);
      load_rows<2>(x[2], l, at);
      load_rows<3>(x[3], l, at);
    };
    for (;;) {
      const int64_t t0 = cur.begin > u0 ? cur.begin : u0, t1 = cur.end < u1 ? cur.end : u1;
      const int n = (int)(t1 - t0);
      int x = (cur.g.tile0 + (int)(t0 - cur.begin)) * kPos + 16 * w;
      const int end = x + n * kPos;  // behind the share's tiles
      Blocks blocks;
      blocks.find(p, cur, x, end, lane);
      RowPart kp[4], vp[4];
      uint32_t at = blocks.of(0);
      load(kp, in_k, at);
      for (int i = 0; i <= n && ok; ++i, x += kPos) {
        const uint32_t at_v = at;
        if (i < n) {
          store(kp);
          if ((i + 1) % Blocks::kTiles == 0) blocks.find(p, cur, x + kPos, end, lane);
          at = blocks.of(i + 1);
          load(kp, in_k, at);
        }
        if (i > 0 && ok) {
          // rows that no token of the group sees: their P is 0, but they may hold anything
          if (x - kPos < cur.g.lo || x - kPos + 15 > cur.g.hi) {
            const int r0 = x - kPos + ((lane & 3) < 2 ? lane & 3 : (lane & 3) + 4), r1 = x - kPos + (lane & 3) + 2;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int row = ((u & 1) ? r1 : r0) + 8 * (u >> 1);
              if (row < cur.g.lo || row > cur.g.hi) vp[u].scale = 0u;
            }
          }
          store(vp);
        }
        if (i < n) load(vp, in_v, at_v);
      }
      if (!ok || !cur.advance(p, sh, u1)) break;
    }
    if (!ok && lane == 0) {
      if (!flags[0]) atomicOr(p.err, kErrWaitTimeout);
      flags[0] = 1;
    }
  } else if (warp >= kFirstSoft) {
    more_registers<R::kSoft>();
    softmax_warps<QT, 1, false, true, true>(p, sh, cur, u0, u1, total, G, c, 0, base, tmem, q_raw, s_full, pv_done, flags, nullptr,
                                      warp, tid - 32 * kFirstSoft, [&] { mbar_arrive(q_full); },
                                      [&](uint32_t buf) { mbar_arrive(&p_full[buf]); });
  } else {
    fewer_registers<R::kIssue>();
    if (warp == 0) {
      // ---- the groups' queries, each once the group before has its last S
      uint32_t item = 0;
      bool ok = true;
      for (;;) {
        if (item > 0 && !mbar_wait_bounded(q_empty, (item - 1) & 1, flags, kWaitLimitNs)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(q_raw, query_bytes<QT>(cur.g.n_tok, 0));
        __syncwarp();
        load_queries<QT>(base, &tm_q, &tm_q8, cur, 0, lane,
                         [&](const CUtensorMap* map, void* to, int head, int tok, int line) {
                           tma_load_4d(to, map, q_raw, 0, head, tok, line);
                         });
        ++item;
        if (!cur.advance(p, sh, u1)) break;
      }
      if (!ok && lane == 0) {
        if (!flags[0]) atomicOr(p.err, kErrWaitTimeout);
        flags[0] = 1;
      }
      if (item > 0) {
        // let the copies in flight land before the CTA can exit
        int never = 0;
        mbar_wait_bounded(q_raw, (item - 1) & 1, &never, kWaitLimitNs);
      }
    } else if (warp == 1) {
      // ---- MMA issuer (one elected lane)
      constexpr uint32_t kIdS = tc::idesc(kRows, kPos, false, true), kIdO = tc::idesc(kRows, kPos, true, true);
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
          const uint64_t b0 = tc::desc_k_major(ring + s * kSlot, kGroupBytes<2>);
          const uint64_t a0 = tc::desc_k_major(q_addr + 2 * half * S::kQLine);
          if (one) {
#pragma unroll
            for (int part = S::kQ - 1; part >= 0; --part)  // (the remainders first: kFoldTiles)
#pragma unroll
              for (int line = 0; line < 2; ++line)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                  tc::mma_ss(d, a0 + ((part * kLineBytes + line * S::kQLine) >> 4) + 2 * ks,
                             b0 + (line * kAtom >> 4) + 2 * ks, kIdS, half > 0 || part < S::kQ - 1 || line + ks > 0);
            tc::commit(&empty[s]);
            if (half == 1) tc::commit(&s_full[i & 1]);
          }
          __syncwarp();
        }
      };
      auto values = [&](uint32_t i, bool first) {
        const uint32_t a = tmem + kColS + (i & 1) * kPos;
        if (!wait(&p_full[i & 1], (i >> 1) & 1)) return;
#pragma unroll
        for (int half = 0; half < 2; ++half, ++k) {
          const int s = (int)(k % NS);
          if (!wait(&full[s], (k / NS) & 1)) return;
          const uint64_t b0 = tc::desc_mn_major(ring + s * kSlot, kAtom, kGroupBytes<2>);
          const uint32_t d = tmem + half * 128;
          if (one) {
#pragma unroll
            for (int part = 0; part < S::kQ; ++part)
#pragma unroll
              for (int ks = 0; ks < kPos / 16; ++ks)  // 16 positions: two 8-row groups, eight columns of P
                tc::mma_ts(d, a + (ks >> 1) * 32 + part * 16 + (ks & 1) * 8, b0 + ks * (2 * kGroupBytes<2> >> 4), kIdO,
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
        if (!wait(q_full, item & 1)) break;
        ++item;
        for (int i = 0; i <= n && ok; ++i) {
          if (i < n) scores(tile + i);
          if (i == n - 1 && ok && one) tc::commit(q_empty);
          if (i > 0 && ok) values(tile + i - 1, i == 1);
        }
        tile += n;
        if (!ok || !__shfl_sync(0xffffffffu, (int)cur.advance(p, sh, u1), 0)) break;
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
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tmem, kCols);
  }
}

template <typename QT>
cudaError_t launch_chunk4(const Args& p, const void* k, const void* v, cudaStream_t st) {
  using S = Chunk4Smem<std::is_same<QT, float>::value>;
  CUtensorMap mq, mq8;
  if (!make_query_maps<QT>(&mq, &mq8, p)) return cudaErrorInvalidValue;
  auto kern = k_paged4_chunk<QT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kAlloc);
  if (e != cudaSuccess) return e;
  int grid = device_sm_count();
  if (grid > paged::kMaxChunkCtas) grid = paged::kMaxChunkCtas;
  e = launch_pdl(kern, dim3(grid), dim3(kThreads4), S::kAlloc, st, static_cast<const unsigned char*>(k),
                 static_cast<const unsigned char*>(v), mq, mq8, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_paged_join<QT, 1>, dim3(grid, kRows / kJoinRows, kJoinSplit), dim3(32 * kJoinWarps), 0, st, p);
}

}  // namespace

cudaError_t launch_paged4_chunk(const paged::Args& p, int qdtype, const void* k, const void* v, cudaStream_t st) {
  return qdtype == SPARK_BF16 ? launch_chunk4<__nv_bfloat16>(p, k, v, st) : launch_chunk4<float>(p, k, v, st);
}

}  // namespace spark
