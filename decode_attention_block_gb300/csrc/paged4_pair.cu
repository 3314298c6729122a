// paged4_pair.cu -- the chunk attention of paged4_chunk.cu on pairs of CTAs, for
// batches of mostly long chunks: paged_pair.cu with fp16 operands and K and V
// converted from codes.
//
// A pair's CTAs hold half of a tile each (the keys of 64 of its 128 positions,
// 128 of the 256 dims of its values), and convert that half alone.  Alone a CTA
// writes 128 KB of operands a tile into its shared memory and its MMAs read 192:
// 2560 cycles at 128 bytes a cycle, against 2048 of MMA; of a pair each writes 64
// and reads 128.
//
// The softmax warps keep a row's 128 scores in registers here (240 a thread): their
// chain of a tile is what is longest (read twice with 152 registers: 278 us for a
// chunk of 4096 tokens at 4096, against 262).
//
// Measured, a chunk of 4096 tokens at 4096: bf16 queries 265 us in a graph, 1550
// TFLOP/s, 0.79 of the measured bf16 rate (bf16 pages 223: a tile takes 2600 cycles
// against 2048 of MMA, the softmax slowed by the converting warps beside it on its
// schedulers); fp32 queries 555 (bf16 pages 409), two MMAs for each and their sums
// into memory (kFoldTiles); a window of 512 73.  On single CTAs 328, 596 and 77.
//
// A tile's scores, softmax and product follow one another, and two tiles are in
// flight: 1024 + 1800 + 1024 cycles and the reports between them.  Neither two
// softmax warps a row (64 positions each: 406 us, their maxima exchanged and their
// registers short) nor a report of the first 64 probabilities ahead of the others
// (280, one more wait of the issuing warp) made that shorter.
//
// Each CTA's eight converting warps report a half to its own CTA, rank 1's warp 1
// passes it on to rank 0, whose warp 1 issues the MMAs over both: one wait for the
// nine (one for each CTA's, fp32 queries: 559 us against 547).
#include "paged4_chunk_parts.cuh"
#include "paged_pair_parts.cuh"

namespace spark {
namespace {

using namespace chunk4;

constexpr int kMinUnits4 = 2;

template <bool SPLIT>
struct Pair4Smem {
  static constexpr int kQ = SPLIT ? 2 : 1;
  static constexpr uint32_t kQLine = kQ * kLineBytes;  // a line of the queries, with that of the remainders
  static constexpr int kK = SPLIT ? 1 : 2;
  static constexpr int kV = 2;
  static constexpr int kLead = SPLIT ? 3 : 2;  // a group's cost beyond its tiles, in tiles
  static constexpr uint32_t kRingK = kQ * kQBytes;
  static constexpr uint32_t kRingV = kRingK + kK * kSlot;
  static constexpr uint32_t kStage = kRingV + kV * kSlot;  // the output's, where there is room
  static constexpr uint32_t kBars = kStage + (SPLIT ? 0 : 4 * kStageBytes);
  static constexpr uint32_t kBytes = kBars + 8 * (2 * kK + 2 * kV + 10) + 32;
  static constexpr uint32_t kAlloc = kBytes + 1024;  // slack to align the base (128-byte swizzle)
};
static_assert(Pair4Smem<true>::kAlloc <= 232448 && Pair4Smem<false>::kAlloc <= 232448, "227 KB per CTA");
static_assert(kSlot >= 8 * (SPARK_MAX_BATCH + 2 + kThreads4 / 16), "room for the prefix sums");

template <typename QT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads4, 1)
    k_paged4_pair(const unsigned char* pk, const unsigned char* pv, const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ CUtensorMap tm_q8, const __grid_constant__ Args p) {
  constexpr bool kSplit = std::is_same<QT, float>::value;
  using S = Pair4Smem<kSplit>;
  using R = Regs<96, 240, 88>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // this CTA's half of a tile is there; rank 0: rank 1's too
  uint64_t* k_here = reinterpret_cast<uint64_t*>(base + S::kBars);
  uint64_t* k_empty = k_here + S::kK;
  uint64_t* v_here = k_empty + S::kK;
  uint64_t* v_empty = v_here + S::kV;
  uint64_t* s_full = v_empty + S::kV;  // [2] S(i) is in its buffer
  uint64_t* p_full = s_full + 2;       // [2] rank 0: P(i) is, in both CTAs
  uint64_t* pv_done = p_full + 2;      // [2] P(i) V(i) is in O
  uint64_t* q_full = pv_done + 2;      // rank 0: the queries are there, in both CTAs
  uint64_t* q_raw = q_full + 1;        // this CTA's have landed, not yet fp16
  uint64_t* q_empty = q_raw + 1;       // the group's last S is done
  uint64_t* drained = q_empty + 1;     // rank 0: every MMA has completed
  volatile int* flags = reinterpret_cast<volatile int*>(drained + 1);  // [0] abort
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 2);

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = (int)cluster_rank();
  if (tid == 0) {
    for (int s = 0; s < S::kK; ++s) {
      mbar_init(&k_here[s], kDequant + (rank == 0 ? 1 : 0));
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < S::kV; ++s) {
      mbar_init(&v_here[s], kDequant + (rank == 0 ? 1 : 0));
      mbar_init(&v_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], 2 * kSoft / 32);
      mbar_init(&pv_done[b], 1);
    }
    mbar_init(q_full, 2 * kSoft / 32);
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
  const Shape sh{kPairTokens, kPos, p.window, S::kLead};
  // the rings are not in use yet: room for the prefix sums
  int64_t* prefix = reinterpret_cast<int64_t*>(base + S::kRingK);
  const int c = blockIdx.x >> 1;
  paged::Share share;
  if (!paged::find_share<kThreads4>(p, sh, c, kMinUnits4, gridDim.x >> 1, prefix, share)) {  // both CTAs of the pair
    if (tid == 0 && rank == 0) p.joins[c].n_rows = 0;
    return;
  }
  const int64_t total = share.total, u0 = share.u0, u1 = share.u1;
  const int G = share.G;
  Cursor cur = share.cur;
  if (warp == 1) tc::alloc2(tmem_slot, kCols);
  tc::fence_before();
  __syncthreads();
  pair_sync();  // the barriers of both CTAs are ready
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp >= kFirstDequant) {
    // ---- K(0), then K(i), V(i - 1) for the tiles of each group.  Of K warp 8 + w
    // takes half w % 2 of the rows of block w / 2 of this CTA's four, of V this
    // CTA's half of the dims of block w.
    fewer_registers<R::kDequant>();
    const int w = warp - kFirstDequant;
    uint32_t kk = 0, kv = 0;
    bool ok = true;
    RowLanes in_k(pk, lane);
    if (w & 1) {
      in_k.x0 += in_k.d0;
      in_k.x1 += in_k.d1;
      in_k.y0 += 8 * fp4::kScales;
      in_k.y1 += 8 * fp4::kScales;
    }
    const Lanes in_v(pv, lane);
    uint32_t places[4];
    part_places(places, lane);
    // the lane's line in a slot
    const uint32_t line_k = smem_u32(base + S::kRingK) + w * kGroupBytes<4> + (2 * in_k.h + in_k.line) * kAtom;
    const uint32_t line_v = smem_u32(base + S::kRingV) + 2 * w * kGroupBytes<2> + (lane >> 4) * kAtom;
    auto freed = [&](uint64_t* bar, uint32_t use) {
      if (ok && use > 0 && !mbar_wait_bounded(bar, (use - 1) & 1, flags, kWaitLimitNs)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    auto report = [&](uint64_t* bar) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMAs read it through the async proxy
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    for (;;) {
      const int64_t t0 = cur.begin > u0 ? cur.begin : u0, t1 = cur.end < u1 ? cur.end : u1;
      const int n = (int)(t1 - t0);
      const int x0 = (cur.g.tile0 + (int)(t0 - cur.begin)) * kPos;
      int xk = x0 + 64 * rank + 16 * (w >> 1), xv = x0 + 16 * w;
      const int end_k = xk + n * kPos, end_v = xv + n * kPos;  // behind the share's tiles
      Blocks blocks_k, blocks_v;
      blocks_k.find(p, cur, xk, end_k, lane);
      blocks_v.find(p, cur, xv, end_v, lane);
      RowPart kp[2];
      Part vp;
      auto load_k = [&](uint32_t block) {
        load_rows<0>(kp[0], in_k, block);
        load_rows<1>(kp[1], in_k, block);
      };
      load_k(blocks_k.of(0));
      for (int i = 0; i <= n && ok; ++i, xk += kPos, xv += kPos) {
        if (i < n) {
          const int s = (int)(kk % S::kK);
          if (!freed(&k_empty[s], kk / S::kK)) break;
          store_rows(line_k + s * kSlot + in_k.at0, kp[0]);
          store_rows(line_k + s * kSlot + in_k.at1, kp[1]);
          report(&k_here[s]);
          ++kk;
          if (((i + 1) & 31) == 0) blocks_k.find(p, cur, xk + kPos, end_k, lane);
          load_k(blocks_k.of(i + 1));
        }
        if (i > 0) {
          // rows that no token of the group sees: their P is 0, but they may hold anything
          const int row = xv - kPos + (lane & 7);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (row + 8 * e < cur.g.lo || row + 8 * e > cur.g.hi) vp.scale[e] = 0u;
          const int s = (int)(kv % S::kV);
          if (!freed(&v_empty[s], kv / S::kV)) break;
          store_part(line_v + s * kSlot, places, kGroupBytes<2>, vp);
          report(&v_here[s]);
          ++kv;
        }
        if (i < n) {
          if (i > 0 && (i & 31) == 0) blocks_v.find(p, cur, xv, end_v, lane);
          in_v.load(vp, blocks_v.of(i), rank);
        }
      }
      if (!ok || !cur.advance(p, sh, u1)) break;
    }
    if (!ok && lane == 0) {
      if (!flags[0]) atomicOr(p.err, kErrWaitTimeout);
      flags[0] = 1;
    }
  } else if (warp >= kFirstSoft) {
    more_registers<R::kSoft>();
    const uint32_t q_bar = in_rank0(q_full), p_bar = in_rank0(p_full);
    softmax_warps<QT, 2, !kSplit, true>(p, sh, cur, u0, u1, total, G, c, rank, base, tmem, q_raw, s_full, pv_done, flags,
                                        base + S::kStage, warp, tid - 32 * kFirstSoft, [&] { arrive_at(q_bar); },
                                        [&](uint32_t buf) { arrive_tmem_at(p_bar + 8 * buf); });
  } else {
    fewer_registers<R::kIssue>();
    if (warp == 0) {
      // ---- the groups' queries, each once the group before has its last S
      uint32_t item = 0;
      bool ok = true;
      const int tok0 = rank * paged::kChunkTokens;
      for (;;) {
        if (item > 0 && !mbar_wait_bounded(q_empty, (item - 1) & 1, flags, kWaitLimitNs)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(q_raw, query_bytes<QT>(cur.g.n_tok, tok0));
        __syncwarp();
        load_queries<QT>(base, &tm_q, &tm_q8, cur, tok0, lane,
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
        // let the copies in flight land before the CTAs can exit
        int never = 0;
        mbar_wait_bounded(q_raw, (item - 1) & 1, &never, kWaitLimitNs);
      }
    } else if (warp == 1) {
      // ---- rank 0: MMA issuer (one elected lane); rank 1: its halves' reports
      constexpr uint32_t kIdS = tc::idesc(2 * kRows, kPos, false, true), kIdO = tc::idesc(2 * kRows, kHeadDim, true, true);
      const uint32_t q_addr = smem_u32(base), ring_k = smem_u32(base + S::kRingK), ring_v = smem_u32(base + S::kRingV);
      uint32_t kk = 0, kv = 0, tile = 0, item = 0;
      bool ok = true;
      const bool one = tc::elect();
      auto both = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, wait_pair(bar, parity, flags));
        tc::fence_after();
        return ok;
      };
      auto here = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, flags, kWaitLimitNs));
        return ok;
      };
      auto scores = [&](uint32_t i) {
        const uint32_t d = tmem + kColS + (i & 1) * kPos;
        const int s = (int)(kk % S::kK);
        if (!both(&k_here[s], (kk / S::kK) & 1)) return;
        const uint64_t a0 = tc::desc_k_major(q_addr);
        const uint64_t b0 = tc::desc_k_major(ring_k + s * kSlot, kGroupBytes<4>);
        if (one) {
#pragma unroll
          for (int part = S::kQ - 1; part >= 0; --part)  // (the remainders first: kFoldTiles)
#pragma unroll
            for (int line = 0; line < 4; ++line)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                tc::mma_ss2(d, a0 + ((part * kLineBytes + line * S::kQLine) >> 4) + 2 * ks,
                            b0 + (line * kAtom >> 4) + 2 * ks, kIdS, part < S::kQ - 1 || line + ks > 0);
          tc::commit_both(&k_empty[s]);
          tc::commit_both(&s_full[i & 1]);
        }
        __syncwarp();
        ++kk;
      };
      auto values = [&](uint32_t i, bool first) {
        const uint32_t a = tmem + kColS + (i & 1) * kPos;
        const int s = (int)(kv % S::kV);
        if (!both(&v_here[s], (kv / S::kV) & 1)) return;
        if (!both(&p_full[i & 1], (i >> 1) & 1)) return;
        const uint64_t b0 = tc::desc_mn_major(ring_v + s * kSlot, kAtom, kGroupBytes<2>);
        if (one) {
#pragma unroll
          for (int part = 0; part < S::kQ; ++part)
#pragma unroll
            for (int ks = 0; ks < kPos / 16; ++ks)  // 16 positions: two 8-row groups, eight columns of P
              tc::mma_ts2(tmem, a + (ks >> 1) * 32 + part * 16 + (ks & 1) * 8, b0 + ks * (2 * kGroupBytes<2> >> 4), kIdO,
                          !first || part + ks > 0);
          tc::commit_both(&v_empty[s]);
          tc::commit_both(&pv_done[i & 1]);
        }
        __syncwarp();
        ++kv;
      };
      for (;;) {
        const int64_t t0 = cur.begin > u0 ? cur.begin : u0, t1 = cur.end < u1 ? cur.end : u1;
        const int n = __shfl_sync(0xffffffffu, (int)(t1 - t0), 0);  // tiles of the group in this share
        if (rank == 0 && !both(q_full, item & 1)) break;
        ++item;
        for (int i = 0; i <= n && ok; ++i) {
          if (rank == 0) {
            if (i < n) scores(tile + i);
            if (i == n - 1 && ok && one) tc::commit_both(q_empty);
            if (i > 0 && ok) values(tile + i - 1, i == 1);
          } else {
            if (i < n && here(&k_here[kk % S::kK], (kk / S::kK) & 1)) {
              if (lane == 0) arrive_at(in_rank0(&k_here[kk % S::kK]));
              ++kk;
            }
            if (i > 0 && here(&v_here[kv % S::kV], (kv / S::kV) & 1)) {
              if (lane == 0) arrive_at(in_rank0(&v_here[kv % S::kV]));
              ++kv;
            }
          }
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
        if (rank == 0) {
          int never = 0;
          tc::commit2(drained);
          mbar_wait_bounded(drained, 0, &never, kWaitLimitNs);
        }
      }
      __syncwarp();
    }
  }
  tc::fence_before();
  __syncthreads();
  pair_sync();  // neither CTA's memory is touched by the other after this
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc2(tmem, kCols);
  }
}

template <typename QT>
cudaError_t launch_pair4(const Args& p, const void* k, const void* v, cudaStream_t st) {
  using S = Pair4Smem<std::is_same<QT, float>::value>;
  CUtensorMap mq, mq8;
  if (!make_query_maps<QT>(&mq, &mq8, p)) return cudaErrorInvalidValue;
  auto kern = k_paged4_pair<QT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kAlloc);
  if (e != cudaSuccess) return e;
  int pairs = device_sm_count() / 2;
  if (pairs > paged::kMaxChunkCtas / 2) pairs = paged::kMaxChunkCtas / 2;
  if (pairs < 1) pairs = 1;
  e = launch_pdl(kern, dim3(2 * pairs), dim3(kThreads4), S::kAlloc, st, static_cast<const unsigned char*>(k),
                 static_cast<const unsigned char*>(v), mq, mq8, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_paged_join<QT, 2>, dim3(pairs, 2 * kRows / kJoinRows, kJoinSplit), dim3(32 * kJoinWarps), 0, st, p);
}

}  // namespace

cudaError_t launch_paged4_pair(const paged::Args& p, int qdtype, const void* k, const void* v, cudaStream_t st) {
  return qdtype == SPARK_BF16 ? launch_pair4<__nv_bfloat16>(p, k, v, st) : launch_pair4<float>(p, k, v, st);
}

}  // namespace spark
