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
// in the others).  Shared memory: Q (64 KB, 128 KB in two halves) and a ring
// of 32 KB slots, each 128 positions x 128 dims of K or V.  Warp 0 fills the
// ring (TMA boxes of the part of a page inside the tile) and loads the
// queries (fp32 ones are put in halves by warps 2-5), warp 1 issues the MMAs in the
// order S(i+1), P V(i), so the tensor cores run S(i+1) while warps 2-5 turn
// S(i) into P(i).
//
// Work is the flat list of paged.h (128-position tiles), every CTA an equal
// share: a group cut by a share's border leaves fp32 partial states, joined
// in CTA order by k_paged_join.
//
// This kernel takes chunks of up to 32 tokens, which are bound by the rows
// read from HBM (32 sequences at 4096-8192, 0.82 GB, bf16 queries: 4 tokens
// each 132 us, 6.2 TB/s; 32 tokens 147 us, 5.6 TB/s, 707 TFLOP/s), and batches
// with few longer ones (32 sequences, 4 of them with chunks of ~400 tokens:
// 107 us; 131 to 141 us for fp32 queries, whose MMAs alone take 80); many longer ones
// are bound by what a CTA alone takes in from L2, and go to paged_pair.cu.
// What it cost on the way (a chunk of 4096 tokens at 4096): 128 columns
// unrolled in the softmax missed the instruction cache, 566 us; operands of an
// MMA moved to uniform registers one by one, 361 -> 335; scores read twice,
// 335 -> 330; the table's entry looked up when needed, 330 -> 309.
#include "paged_chunk_parts.cuh"

namespace spark {
namespace {

using namespace chunk;

// Units per CTA at least (one sequence of 8 tokens at 1000, bf16 queries: 13.6
// us at 1, 14.6 at 2; one of 4 at 500 13.1 and 14.4).
constexpr int kMinUnits = 1;

static_assert(kRows == kGroup * paged::kChunkTokens, "a row per query head of a token");

// Q halves and ring slots: 224 KB either way
template <bool SPLIT>
struct ChunkSmem {
  static constexpr int kQ = SPLIT ? 2 : 1;
  static constexpr uint32_t kQLine = kQ * kLineBytes;  // a line of the queries, with that of the remainders
  static constexpr int kSlots = SPLIT ? 3 : 5;
  // A group's cost beyond its tiles, in tiles.  A mixed batch of 32 (pages of
  // 16 rows line by line), fp32 queries: 195 us at 0, 160, 154 and 157 at 1, 2
  // and 3; bf16 ones 137 at 0 and 136, 141 and 144.
  static constexpr int kLead = SPLIT ? 2 : 1;
  static constexpr uint32_t kRing = kQ * kQBytes;
  static constexpr uint32_t kBars = kRing + kSlots * kSlot;
  static constexpr uint32_t kBytes = kBars + 8 * (2 * kSlots + 10) + 32;
  static constexpr uint32_t kAlloc = kBytes + 1024;  // slack to align the base (128-byte swizzle)
};
static_assert(ChunkSmem<true>::kAlloc <= 232448 && ChunkSmem<false>::kAlloc <= 232448, "227 KB per CTA");

template <typename QT>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_chunk(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q8,
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
  uint64_t* q_raw = q_full + 1;    // fp32: they are, not yet in halves
  uint64_t* q_empty = q_raw + 1;   // the group's last S is done
  uint64_t* drained = q_empty + 1;  // every MMA has completed
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
      mbar_init(&p_full[b], kSoft / 32);
      mbar_init(&pv_done[b], 1);
    }
    mbar_init(q_full, kSplit ? kSoft / 32 : 1);
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
  const Shape sh{paged::kChunkTokens, kPos, p.window, S::kLead};
  // the ring is not in use yet: room for the prefix sums
  int64_t* prefix = reinterpret_cast<int64_t*>(base + S::kRing);
  const int c = blockIdx.x;
  paged::Share share;
  if (!paged::find_share<kThreads>(p, sh, c, kMinUnits, gridDim.x, prefix, share)) {
    if (tid == 0) p.joins[c].n_rows = 0;
    return;
  }
  const int64_t total = share.total, u0 = share.u0, u1 = share.u1;
  const int G = share.G;
  Cursor cur = share.cur;
  if (warp == 1) tc::alloc(tmem_slot, kCols);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the prefix sums make way for TMA's writes
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp == 0) {
    // ---- producer: K(0), then K(i), V(i - 1) for the tiles of each group
    uint32_t k = 0, item = 0;
    bool ok = true;
    uint64_t* q_here = kSplit ? q_raw : q_full;
    const int per = kPos / box;  // boxes of a tile
    const uint64_t once = policy_once(), again = policy_again();
    auto slot = [&](const CUtensorMap* map, int half, int z, int b0, int b1) {
      const int s = (int)(k % NS);
      const uint32_t r = k / NS;
      if (ok && r > 0 && !mbar_wait_bounded(&empty[s], (r - 1) & 1, flags, kWaitLimitNs)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      const int n = b1 - b0;
      if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(n * box) * 256u);
      __syncwarp();
      // a lane per box, its two lines at once; z is the box's row
      if (lane >= b0 && lane < b1)
        tma_load_rows(base + S::kRing + s * kSlot + lane * (box / 8) * kGroupBytes<2>, map, &full[s], z, 2 * half, cur.j,
                      cur.groups == 1 ? once : again);
      ++k;
    };
    for (;;) {
      const int64_t t0 = cur.begin > u0 ? cur.begin : u0, t1 = cur.end < u1 ? cur.end : u1;
      // the group's queries, once the group before has its last S
      if (item > 0 && !mbar_wait_bounded(q_empty, (item - 1) & 1, flags, kWaitLimitNs)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(q_here, query_bytes<QT>(cur.g.n_tok, 0));
      __syncwarp();
      load_queries<QT>(base, &tm_q, &tm_q8, cur, 0, lane,
                       [&](const CUtensorMap* map, void* to, int head, int tok, int line) {
                         tma_load_4d(to, map, q_here, 0, head, tok, line);
                       });
      ++item;
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
        return lane >= b0 && lane < b1 ? paged::page_entry(p, cur.s, paged::page_col(p, pos + lane * box)) : 0;
      };
      int z_v = 0, v0 = 0, v1 = 0;  // the tile before
      int ahead = entry(t0);
      for (int64_t u = t0; u <= t1 && ok; ++u) {
        int z = 0, b0 = 0, b1 = 0;
        if (u < t1) {
          int pos;
          boxes(u, pos, b0, b1);
          z = paged::page_of(p, ahead) * p.page_size + paged::page_row(p, pos + lane * box);
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
      if (!ok || !cur.advance(p, sh, u1)) break;
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
      if (item > 0) mbar_wait_bounded(q_here, (item - 1) & 1, &never, kWaitLimitNs);
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
        const uint64_t b0 = tc::desc_k_major(ring + s * kSlot, kGroupBytes<2>);
        const uint64_t a0 = tc::desc_k_major(q_addr + 2 * half * S::kQLine);
        if (one) {
#pragma unroll
          for (int line = 0; line < 2; ++line)
#pragma unroll
            for (int part = 0; part < S::kQ; ++part)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                tc::mma_ss(d, a0 + ((part * kLineBytes + line * S::kQLine) >> 4) + 2 * ks,
                           b0 + (line * kAtom >> 4) + 2 * ks, kIdS, half + line + part + ks > 0);
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
          clear_rows(base + S::kRing + s * kSlot, r0, r1, lane);
          __syncwarp();
        }
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
      const int pos0 = __shfl_sync(0xffffffffu, (cur.g.tile0 + (int)(t0 - cur.begin)) * kPos, 0);
      const int lo = __shfl_sync(0xffffffffu, cur.g.lo, 0), hi = __shfl_sync(0xffffffffu, cur.g.hi, 0);
      if (!wait(q_full, item & 1)) break;
      ++item;
      for (int i = 0; i <= n && ok; ++i) {
        if (i < n) scores(tile + i);
        if (i == n - 1 && ok && one) tc::commit(q_empty);
        if (i > 0 && ok) {
          const int pos = pos0 + (i - 1) * kPos;
          values(tile + i - 1, i == 1, lo > pos ? lo - pos : 0, hi + 1 - pos < kPos ? hi + 1 - pos : kPos);
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
      int never = 0;
      tc::commit(drained);
      mbar_wait_bounded(drained, 0, &never, kWaitLimitNs);
    }
    __syncwarp();
  } else {
    softmax_warps<QT, 1, false>(p, sh, cur, u0, u1, total, G, c, 0, base, tmem, q_raw, s_full, pv_done, flags, nullptr,
                                warp, tid - 64, [&] { mbar_arrive(q_full); },
                                [&](uint32_t buf) { mbar_arrive(&p_full[buf]); });
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tmem, kCols);
  }
}

template <typename QT>
cudaError_t launch_chunk(const Args& p, const void* k, const void* v, cudaStream_t st) {
  using S = ChunkSmem<std::is_same<QT, float>::value>;
  int box = kPos;  // the largest box that divides both a tile and a page
  while (p.page_size % box != 0) box /= 2;
  CUtensorMap mk, mv;
  const int64_t rows = (int64_t)p.n_pages * p.page_size;
  if (!make_chunk_map(&mk, k, p.n_kv, rows, box, 2) || !make_chunk_map(&mv, v, p.n_kv, rows, box, 2))
    return cudaErrorInvalidValue;
  CUtensorMap mq, mq8;
  if (!make_query_maps<QT>(&mq, &mq8, p)) return cudaErrorInvalidValue;
  auto kern = k_paged_chunk<QT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kAlloc);
  if (e != cudaSuccess) return e;
  int grid = device_sm_count();
  if (grid > paged::kMaxChunkCtas) grid = paged::kMaxChunkCtas;
  e = launch_pdl(kern, dim3(grid), dim3(kThreads), S::kAlloc, st, mk, mv, mq, mq8, p, box);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_paged_join<QT, 1>, dim3(grid, kRows / kJoinRows, kJoinSplit), dim3(32 * kJoinWarps), 0, st, p);
}

}  // namespace

cudaError_t launch_paged_chunk(const paged::Args& p, int qdtype, const void* k, const void* v, cudaStream_t st) {
  return qdtype == SPARK_BF16 ? launch_chunk<__nv_bfloat16>(p, k, v, st) : launch_chunk<float>(p, k, v, st);
}

}  // namespace spark
