// paged_pair.cu -- the chunk attention of paged_chunk.cu on pairs of CTAs, for
// batches of mostly long chunks.
//
// A pair (a cluster of 2) takes a group of 64 consecutive tokens of one
// sequence with one KV head: 256 rows, 128 in each CTA, one MMA of M = 256
// over both (tcgen05 cta_group::2, issued by rank 0).  Each CTA loads and
// holds half of a tile: the keys of 64 of its 128 positions (half of the N
// side of S = Q K^T) and 128 of the 256 dims of its values (half of the N
// side of O += P V).  So a CTA takes in 64 KB per tile instead of 128: alone
// it was bound by that (32 KB in 700 cycles against 512 of MMA), and a tile
// takes two ring slots instead of four, so loads run a tile further ahead.
//
// Rows, tensor memory, softmax and joins are as in paged_chunk.cu (rank r
// has the group's tokens 32 r .. 32 r + 31).  The MMA warp of rank 0 waits for
// both CTAs: K tiles complete on its barrier (either CTA's copies count their
// bytes there), V tiles on each CTA's own, where the rows that no token of the
// group sees are cleared before rank 1 reports to rank 0; queries and
// probabilities are reported by a lane of each softmax warp of both.  What the
// MMAs release (slots, scores, output) they release in both CTAs.
//
// Measured, a chunk of 4096 tokens at 4096 (2.1e11 multiply-adds): bf16 queries
// 223 us in a graph of ten calls, 1850 TFLOP/s, 0.96 of the measured bf16 rate
// (240 us on pages of 16 rows), and 245 us, 1680 TFLOP/s, where calls follow
// one another for a second and the power limit holds the SMs at 1.72 GHz (0.96
// of the rate measured so); fp32 queries (two MMAs for each) 409 and 448 us;
// with a window of 512 54 and 90 us.  A tile takes
// 2050 cycles against 2048 of MMA, the softmax 1850 beside it; the rest is the
// start, the first and last tile of a group (its queries come by TMA, its
// output leaves through a stage: with both done by the softmax threads row by
// row it was 250 us) and the join.
#include "paged_chunk_parts.cuh"
#include "paged_pair_parts.cuh"

namespace spark {
namespace {

using namespace chunk;

// Units per pair at least (one sequence of 48 tokens at 1000, bf16 queries: 15.7
// us at 2, 16.9 at 1, 18.2 at 3).
constexpr int kMinUnits = 2;

template <bool SPLIT>
struct PairSmem {
  static constexpr int kQ = SPLIT ? 2 : 1;
  static constexpr uint32_t kQLine = kQ * kLineBytes;  // a line of the queries, with that of the remainders
  // (fp32 queries leave room for three slots: V, with a hop more to the MMA,
  // gets two; a third for bf16 ones gave nothing, and the output's stage wants room)
  static constexpr int kK = SPLIT ? 1 : 2;
  static constexpr int kV = 2;
  // A group's cost beyond its tiles, in tiles.  Four chunks of 258 to 517
  // tokens, fp32 queries: 92 us at 0, 82, 73 and 70 at 1, 2 and 3, 73 at 4;
  // bf16 ones 55.7, 49.5, 45.3, 44.7 and 44.9 (a chunk of 4096 230 us at 0,
  // 229 at 2, 231 at 3).
  static constexpr int kLead = SPLIT ? 3 : 2;
  static constexpr uint32_t kRingK = kQ * kQBytes;
  static constexpr uint32_t kRingV = kRingK + kK * kSlot;
  static constexpr uint32_t kStage = kRingV + kV * kSlot;  // the output's, where there is room
  static constexpr uint32_t kBars = kStage + (SPLIT ? 0 : 4 * kStageBytes);
  static constexpr uint32_t kBytes = kBars + 8 * (2 * kK + 3 * kV + 10) + 32;
  static constexpr uint32_t kAlloc = kBytes + 1024;  // slack to align the base (128-byte swizzle)
};
static_assert(PairSmem<true>::kAlloc <= 232448 && PairSmem<false>::kAlloc <= 232448, "227 KB per CTA");

// TMA into this CTA's shared memory, its bytes counted on a barrier of rank 0
__device__ __forceinline__ void tma_load_4d_pair(void* dst, const CUtensorMap* map, uint32_t cluster_bar, int c0, int c1,
                                                 int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// ... a box of rows (tma_load_rows)
__device__ __forceinline__ void tma_load_rows_pair(void* dst, const CUtensorMap* map, uint32_t cluster_bar, int row,
                                                   int line, int head, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(0), "r"(line), "r"(row >> 3), "r"(head), "l"(policy)
      : "memory");
}

template <typename QT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_paged_pair(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q8,
                 const __grid_constant__ Args p, int box_k, int box_v) {
  constexpr bool kSplit = std::is_same<QT, float>::value;
  using S = PairSmem<kSplit>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(base + S::kBars);  // rank 0: both halves of a K tile are there
  uint64_t* k_empty = k_full + S::kK;
  uint64_t* v_here = k_empty + S::kK;  // this CTA's half of a V tile is there
  uint64_t* v_peer = v_here + S::kV;   // rank 0: rank 1's is, and cleared
  uint64_t* v_empty = v_peer + S::kV;
  uint64_t* s_full = v_empty + S::kV;  // [2] S(i) is in its buffer
  uint64_t* p_full = s_full + 2;       // [2] rank 0: P(i) is, in both CTAs
  uint64_t* pv_done = p_full + 2;      // [2] P(i) V(i) is in O
  uint64_t* q_full = pv_done + 2;      // rank 0: the queries are there, in both CTAs
  uint64_t* q_raw = q_full + 1;        // fp32: this CTA's are, not yet in halves
  uint64_t* q_empty = q_raw + 1;       // the group's last S is done
  uint64_t* drained = q_empty + 1;     // rank 0: every MMA has completed
  volatile int* flags = reinterpret_cast<volatile int*>(drained + 1);  // [0] abort
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 2);

  // (the warp's number, and below the MMA warp's loop bounds, by way of a
  // shuffle: known to be the same in every lane, they and what follows from
  // them stay in uniform registers, where an MMA takes its operands from)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = (int)cluster_rank();
  if (tid == 0) {
    for (int s = 0; s < S::kK; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < S::kV; ++s) {
      mbar_init(&v_here[s], 1);
      mbar_init(&v_peer[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], 2 * kSoft / 32);
      mbar_init(&pv_done[b], 1);
    }
    mbar_init(q_full, kSplit ? 2 * kSoft / 32 : 1);
    mbar_init(q_raw, 1);
    mbar_init(q_empty, 1);
    mbar_init(drained, 1);
    flags[0] = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
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
  if (!paged::find_share<kThreads>(p, sh, c, kMinUnits, gridDim.x >> 1, prefix, share)) {  // both CTAs of the pair
    if (tid == 0 && rank == 0) p.joins[c].n_rows = 0;
    return;
  }
  const int64_t total = share.total, u0 = share.u0, u1 = share.u1;
  const int G = share.G;
  Cursor cur = share.cur;
  if (warp == 1) tc::alloc2(tmem_slot, kCols);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the prefix sums make way for TMA's writes
  tc::fence_before();
  __syncthreads();
  pair_sync();  // the barriers of both CTAs are ready
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp == 0) {
    // ---- producer: K(0), then K(i), V(i - 1) for the tiles of each group
    uint32_t kk = 0, kv = 0, item = 0;
    bool ok = true;
    const int per_k = 64 / box_k, per_v = kPos / box_v;  // boxes of a half's keys, of a tile's values
    const int bk = lane % per_k, bv = lane % per_v;      // the lane's boxes
    const uint64_t once = policy_once(), again = policy_again();
    auto freed = [&](uint64_t* bar, uint32_t use) {
      if (ok && use > 0 && !mbar_wait_bounded(bar, (use - 1) & 1, flags, kWaitLimitNs)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    for (;;) {
      const int64_t t0 = cur.begin > u0 ? cur.begin : u0, t1 = cur.end < u1 ? cur.end : u1;
      // the group's queries, once the group before has its last S: fp32 ones on
      // each CTA's barrier, the bytes of bf16 ones in both on that of rank 0
      if (!freed(q_empty, item)) break;
      const int tok0 = rank * paged::kChunkTokens;
      if (lane == 0) {
        if (kSplit)
          mbar_arrive_expect_tx(q_raw, query_bytes<QT>(cur.g.n_tok, tok0));
        else if (rank == 0)
          mbar_arrive_expect_tx(q_full, query_bytes<QT>(cur.g.n_tok, 0) + query_bytes<QT>(cur.g.n_tok, paged::kChunkTokens));
      }
      __syncwarp();
      load_queries<QT>(base, &tm_q, &tm_q8, cur, tok0, lane,
                       [&](const CUtensorMap* map, void* to, int head, int tok, int line) {
                         if (kSplit)
                           tma_load_4d(to, map, q_raw, 0, head, tok, line);
                         else
                           tma_load_4d_pair(to, map, in_rank0(q_full), 0, head, tok, line);
                       });
      ++item;
      const int lo = cur.g.lo, hi = cur.g.hi;
      auto pos_of = [&](int64_t u) { return (cur.g.tile0 + (int)(u - cur.begin)) * kPos; };
      // whether a box of `n` positions from `x` holds a row the group reads
      auto wanted = [&](int x, int n) { return x <= hi && x + n > lo; };
      auto row_of = [&](int x, int entry) {
        return paged::page_of(p, entry) * p.page_size + paged::page_row(p, x);
      };
      auto entry = [&](int x, int n) { return wanted(x, n) ? paged::page_entry(p, cur.s, paged::page_col(p, x)) : 0; };
      // the tables' entries of the lane's boxes, asked for one tile ahead
      int next_k = entry(pos_of(t0) + 64 * rank + bk * box_k, box_k), next_v = entry(pos_of(t0) + bv * box_v, box_v);
      int z_v = 0, pos_v = 0;  // the tile before
      for (int64_t u = t0; u <= t1 && ok; ++u) {
        int z = 0, pos = 0;
        if (u < t1) {
          pos = pos_of(u);
          const int xk = pos + 64 * rank + bk * box_k, xv = pos + bv * box_v;
          const int zk = row_of(xk, next_k);
          z = row_of(xv, next_v);
          if (u + 1 < t1) {
            next_k = entry(xk + kPos, box_k);
            next_v = entry(xv + kPos, box_v);
          }
          const int s = (int)(kk % S::kK);
          if (!freed(&k_empty[s], kk / S::kK)) break;
          // rank 0 expects the bytes of both halves
          if (rank == 0) {
            int n = 0;
            for (int b = 0; b < 2 * per_k; ++b) n += wanted(pos + b * box_k, box_k);
            if (lane == 0) mbar_arrive_expect_tx(&k_full[s], (uint32_t)(n * box_k) * 512u);
            __syncwarp();
          }
          if (lane < per_k && wanted(xk, box_k))
            tma_load_rows_pair(base + S::kRingK + s * kSlot + lane * (box_k / 8) * kGroupBytes<4>, &tm_k,
                               in_rank0(&k_full[s]), zk, 0, cur.j, cur.groups == 1 ? once : again);
          ++kk;
        }
        if (u > t0) {
          const int s = (int)(kv % S::kV);
          if (!freed(&v_empty[s], kv / S::kV)) break;
          int n = 0;
          for (int b = 0; b < per_v; ++b) n += wanted(pos_v + b * box_v, box_v);
          if (lane == 0) mbar_arrive_expect_tx(&v_here[s], (uint32_t)(n * box_v) * 256u);
          __syncwarp();
          if (lane < per_v && wanted(pos_v + lane * box_v, box_v))
            tma_load_rows(base + S::kRingV + s * kSlot + lane * (box_v / 8) * kGroupBytes<2>, &tm_v, &v_here[s], z_v,
                          2 * rank, cur.j, cur.groups == 1 ? once : again);
          ++kv;
        }
        z_v = z;
        pos_v = pos;
      }
      if (!ok || !cur.advance(p, sh, u1)) break;
    }
    if (!ok && lane == 0) {
      if (!flags[0]) atomicOr(p.err, kErrWaitTimeout);
      flags[0] = 1;
    }
    if (flags[0]) {
      // let the copies in flight land before the CTAs can exit
      int never = 0;
      if (rank == 0)
        for (uint32_t i = kk > (uint32_t)S::kK ? kk - S::kK : 0; i < kk; ++i)
          mbar_wait_bounded(&k_full[i % S::kK], (i / S::kK) & 1, &never, kWaitLimitNs);
      if ((kSplit || rank == 0) && item > 0)
        mbar_wait_bounded(kSplit ? q_raw : q_full, (item - 1) & 1, &never, kWaitLimitNs);
      for (uint32_t i = kv > (uint32_t)S::kV ? kv - S::kV : 0; i < kv; ++i)
        mbar_wait_bounded(&v_here[i % S::kV], (i / S::kV) & 1, &never, kWaitLimitNs);
    }
  } else if (warp == 1) {
    // ---- rank 0: MMA issuer (one elected lane); both: the whole warp clears
    // the rows of V tiles that no token of the group sees (their P is 0, but
    // they may hold anything)
    constexpr uint32_t kIdS = tc::idesc(2 * kRows, kPos, false), kIdO = tc::idesc(2 * kRows, kHeadDim, true);
    const uint32_t q_addr = smem_u32(base), ring_k = smem_u32(base + S::kRingK), ring_v = smem_u32(base + S::kRingV);
    uint32_t kk = 0, kv = 0, tile = 0, item = 0;
    bool ok = true;
    const bool one = tc::elect();
    auto both = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, wait_pair(bar, parity, flags));
      tc::fence_after();
      return ok;
    };
    // this CTA's half of the next V tile: rows outside [r0, r1) cleared
    auto values_here = [&](int r0, int r1) {
      const int s = (int)(kv % S::kV);
      ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(&v_here[s], (kv / S::kV) & 1, flags, kWaitLimitNs));
      if (!ok) return false;
      if (r0 > 0 || r1 < kPos) clear_rows(base + S::kRingV + s * kSlot, r0, r1, lane);
      __syncwarp();
      return true;
    };
    auto scores = [&](uint32_t i) {
      const uint32_t d = tmem + kColS + (i & 1) * kPos;
      const int s = (int)(kk % S::kK);
      if (!both(&k_full[s], (kk / S::kK) & 1)) return;
      const uint64_t a0 = tc::desc_k_major(q_addr);
      const uint64_t b0 = tc::desc_k_major(ring_k + s * kSlot, kGroupBytes<4>);
      if (one) {
#pragma unroll
        for (int line = 0; line < 4; ++line)
#pragma unroll
          for (int part = 0; part < S::kQ; ++part)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc::mma_ss2(d, a0 + ((part * kLineBytes + line * S::kQLine) >> 4) + 2 * ks,
                          b0 + (line * kAtom >> 4) + 2 * ks, kIdS, line + part + ks > 0);
        tc::commit_both(&k_empty[s]);
        tc::commit_both(&s_full[i & 1]);
      }
      __syncwarp();
      ++kk;
    };
    auto values = [&](uint32_t i, bool first, int r0, int r1) {
      const uint32_t a = tmem + kColS + (i & 1) * kPos;
      const int s = (int)(kv % S::kV);
      if (!values_here(r0, r1)) return;
      if (!both(&v_peer[s], (kv / S::kV) & 1)) return;
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
      const int pos0 = __shfl_sync(0xffffffffu, (cur.g.tile0 + (int)(t0 - cur.begin)) * kPos, 0);
      const int lo = __shfl_sync(0xffffffffu, cur.g.lo, 0), hi = __shfl_sync(0xffffffffu, cur.g.hi, 0);
      if (rank == 0 && !both(q_full, item & 1)) break;
      ++item;
      for (int i = 0; i <= n && ok; ++i) {
        if (rank == 0 && i < n) {
          scores(tile + i);
          if (i == n - 1 && ok && one) tc::commit_both(q_empty);
        }
        if (i > 0 && ok) {
          const int pos = pos0 + (i - 1) * kPos;
          const int r0 = lo > pos ? lo - pos : 0, r1 = hi + 1 - pos < kPos ? hi + 1 - pos : kPos;
          if (rank == 0) {
            values(tile + i - 1, i == 1, r0, r1);
          } else if (values_here(r0, r1)) {
            if (lane == 0) arrive_at(in_rank0(&v_peer[kv % S::kV]));
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
  } else {
    const uint32_t q_bar = in_rank0(q_full), p_bar = in_rank0(p_full);
    softmax_warps<QT, 2, !kSplit>(p, sh, cur, u0, u1, total, G, c, rank, base, tmem, q_raw, s_full, pv_done, flags,
                                        base + S::kStage, warp, tid - 64, [&] { arrive_at(q_bar); },
                                        [&](uint32_t buf) { arrive_tmem_at(p_bar + 8 * buf); });
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
cudaError_t launch_pair(const Args& p, const void* k, const void* v, int box_k, int box_v, cudaStream_t st) {
  using S = PairSmem<std::is_same<QT, float>::value>;
  CUtensorMap mk, mv;
  const int64_t rows = (int64_t)p.n_pages * p.page_size;
  if (!make_chunk_map(&mk, k, p.n_kv, rows, box_k, 4) ||
      !make_chunk_map(&mv, v, p.n_kv, rows, box_v, 2))
    return cudaErrorInvalidValue;
  CUtensorMap mq, mq8;
  if (!make_query_maps<QT>(&mq, &mq8, p)) return cudaErrorInvalidValue;
  auto kern = k_paged_pair<QT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kAlloc);
  if (e != cudaSuccess) return e;
  int pairs = device_sm_count() / 2;
  if (pairs > paged::kMaxChunkCtas / 2) pairs = paged::kMaxChunkCtas / 2;
  if (pairs < 1) pairs = 1;
  e = launch_pdl(kern, dim3(2 * pairs), dim3(kThreads), S::kAlloc, st, mk, mv, mq, mq8, p, box_k, box_v);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_paged_join<QT, 2>, dim3(pairs, 2 * kRows / kJoinRows, kJoinSplit), dim3(32 * kJoinWarps), 0, st, p);
}

}  // namespace

cudaError_t launch_paged_pair(const paged::Args& p, int qdtype, const void* k, const void* v, cudaStream_t st) {
  int box_v = kPos;  // the largest boxes that divide a tile's values, a half's keys, and a page
  while (p.page_size % box_v != 0) box_v /= 2;
  const int box_k = box_v < 64 ? box_v : 64;
  return qdtype == SPARK_BF16 ? launch_pair<__nv_bfloat16>(p, k, v, box_k, box_v, st)
                              : launch_pair<float>(p, k, v, box_k, box_v, st);
}

}  // namespace spark
