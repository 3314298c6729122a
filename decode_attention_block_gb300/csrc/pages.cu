// pages.cu -- the page tables of a step (spark_pages_remap) and compaction
// (spark_pages_compact): a plan over the tables, then the copies it asks for.
//
// Who holds a page is computed from the tables of the call, not kept: a page
// is free when no slot keeps it.  One array `state` of a word per page says
//   remap    INT_MAX free, -1 kept whole by some slot, s >= 0 kept in part,
//            slot s the lowest of those that keep it so (atomicMin of either,
//            so the outcome does not depend on the order of arrivals);
//   compact  0 unused, 1 used, then the page's rank among those that move.
// The plan is a few dependent passes over the tables and the pages' words.
// Small pools and tables (kSmallPages, kSmallEntries) take one CTA with the
// words in shared memory, larger ones a cluster of 8 CTAs with the words in
// the workspace and hardware cluster barriers between the passes; so a step
// costs one launch for the plan and one for the copies, which read the list
// of moves the plan left.
//
// Measured: the tables of a step of 64 sequences 9.5 us (the cluster form took
// 12 for the plan alone); 112 forks in 36 layers (0.52 GB moved) 92 us, the
// copies at 6.4 TB/s; half of a pool of 900 pages in 36 layers (1.06 GB) 180
// us, 6.3 TB/s in the copies.
#include <limits.h>

#include "attn_parts.cuh"
#include "launch.h"
#include "pages.h"

namespace spark {
namespace {

using pages::Move;

constexpr int kPlanCtas = 8;
constexpr int kPlanThreads = 1024;
constexpr int64_t kSmallPages = 24576;    // state and list: 192 KB of shared memory
constexpr int64_t kSmallEntries = 65536;  // table entries: 256 KB, 64 a thread
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;                                   // 16-byte words per thread and piece
constexpr int kPiece = kCopyThreads * kCopyVecs * 16;          // bytes a CTA copies at a time

struct PlanSmem {
  long long sums[kPlanThreads / 32];
  long long total;
  int off[SPARK_MAX_BATCH];   // first new page of each slot
  int copy[SPARK_MAX_BATCH];  // its index among the copies, or -1
};

// bytes of pages' words (4096 pages) that fit beside it without asking for more
constexpr size_t kPlanDefault = 32 * 1024;
static_assert(kPlanDefault + sizeof(PlanSmem) + 1024 <= 48 * 1024, "shared memory of a block by default");

// exclusive sum over the block's threads; `total` gets the block's sum
__device__ __forceinline__ long long block_scan(long long v, PlanSmem& sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long run = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += up;
  }
  if (lane == 31) sm.sums[warp] = run;
  __syncthreads();
  if (warp == 0) {
    const long long w = sm.sums[lane];
    long long s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += up;
    }
    sm.sums[lane] = s - w;
    if (lane == 31) sm.total = s;
  }
  __syncthreads();
  const long long r = sm.sums[warp] + run - v;
  __syncthreads();  // sums may be written again
  return r;
}

struct PlanArgs {
  const int32_t* table;
  int32_t* new_table;
  int32_t n_slots, max_pages, n_pages, page_size;
  const int32_t *parent, *keep, *grow;  // remap
  int32_t* n_live;                      // compact
  uint32_t* err;
  pages::Head* head;
  Move* moves;
  int32_t* state;  // [n_pages]
  int32_t* list;   // [n_pages]
};

// The plan's CTAs, with the pages' words in shared memory (one CTA) or in the
// workspace (a cluster).
template <int CTAS>
struct Plan {
  static constexpr int kAll = CTAS * kPlanThreads;
  int32_t *state, *list;
  __device__ __forceinline__ explicit Plan(const PlanArgs& p) {
    extern __shared__ int32_t small[];
    state = CTAS == 1 ? small : p.state;
    list = CTAS == 1 ? small + p.n_pages : p.list;
  }
  __device__ __forceinline__ static void sync() {
    if (CTAS == 1)
      __syncthreads();
    else
      cluster_sync_all();
  }
  // a word that other threads wrote
  __device__ __forceinline__ static int get(const int32_t* w) { return CTAS == 1 ? *w : __ldcg(w); }
  // the range of pages a thread counts
  __device__ __forceinline__ static void my_pages(const PlanArgs& p, int cta, int& lo, int& hi) {
    const long long n = p.n_pages, i = (long long)cta * kPlanThreads + threadIdx.x;
    lo = (int)(n * i / kAll);
    hi = (int)(n * (i + 1) / kAll);
  }
  // pages counted by the CTAs before this one, and by all
  __device__ __forceinline__ static void totals(const PlanArgs& p, const PlanSmem& sm, int cta, long long& before,
                                                long long& all) {
    before = all = 0;
    if (CTAS == 1) {
      all = sm.total;
      return;
    }
    if (threadIdx.x == 0) p.head->totals[cta] = (int)sm.total;
    sync();
    for (int c = 0; c < CTAS; ++c) {
      const int t = __ldcg(&p.head->totals[c]);
      if (c < cta) before += t;
      all += t;
    }
  }
};

template <int CTAS>
__global__ void __launch_bounds__(kPlanThreads) k_pages_remap(const __grid_constant__ PlanArgs p) {
  __shared__ PlanSmem sm;
  using P = Plan<CTAS>;
  const P pl(p);
  const int tid = threadIdx.x, lane = tid & 31, cta = blockIdx.x;
  const int all = cta * kPlanThreads + tid, warps = P::kAll / 32, wid = all >> 5;
  pdl_wait();
  for (int i = all; i < p.n_pages; i += P::kAll) pl.state[i] = INT_MAX;
  if (all == 0) {
    p.head->bad = 0;
    p.head->n_moves = 0;
  }
  P::sync();
  // who keeps what
  for (int s = wid; s < p.n_slots; s += warps) {
    const int par = __ldcg(p.parent + s), keep = __ldcg(p.keep + s), grow = __ldcg(p.grow + s);
    const bool ok = par >= -1 && par < p.n_slots && keep >= 0 && keep <= grow && (par >= 0 || keep == 0) &&
                    (long long)grow <= (long long)p.max_pages * p.page_size;
    bool bad = !ok;
    if (ok && keep > 0) {
      const int32_t* old = p.table + (long long)par * p.max_pages;
      const int whole = keep / p.page_size, kept = whole + (keep % p.page_size != 0);
      for (int i = lane; i < kept; i += 32) {
        const int pg = __ldcg(old + i);
        if (pg < 0 || pg >= p.n_pages)
          bad = true;
        else
          atomicMin(&pl.state[pg], i < whole ? -1 : s);
      }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) p.head->bad = 1;
  }
  P::sync();
  const bool bad = __ldcg(&p.head->bad) != 0;  // the same in every CTA
  // pages each slot needs, and where they start among all new pages (every
  // CTA for itself: n_slots <= the block)
  int need = 0, copied = 0;
  if (!bad && tid < p.n_slots) {
    const int keep = __ldcg(p.keep + tid), grow = __ldcg(p.grow + tid);
    const int rest = keep % p.page_size;
    if (rest != 0) {
      const int pg = __ldcg(p.table + (long long)__ldcg(p.parent + tid) * p.max_pages + keep / p.page_size);
      copied = P::get(&pl.state[pg]) != tid;
    }
    need = copied + (int)(((long long)grow + p.page_size - 1) / p.page_size) -
           (int)(((long long)keep + p.page_size - 1) / p.page_size);
  }
  // (need summed in the low 40 bits, copies above them)
  const long long scan = block_scan((long long)need | ((long long)copied << 40), sm);
  const long long want = sm.total & ((1ll << 40) - 1);
  const int n_copies = (int)(sm.total >> 40);
  if (tid < p.n_slots) {
    sm.off[tid] = (int)(scan & ((1ll << 40) - 1));  // at most n_slots * (max_pages + 1)
    sm.copy[tid] = copied ? (int)(scan >> 40) : -1;
  }
  // the free pages, lowest first
  int lo, hi, mine = 0;
  P::my_pages(p, cta, lo, hi);
  for (int i = lo; i < hi; ++i) mine += P::get(&pl.state[i]) == INT_MAX;
  const long long rank = block_scan(mine, sm);
  long long before, free_all;
  P::totals(p, sm, cta, before, free_all);
  if (bad || want > free_all) {
    if (all == 0) atomicOr(p.err, bad ? kErrIndex : kErrPages);
    return;  // every CTA of the cluster alike
  }
  long long r = before + rank;
  for (int i = lo; i < hi && r < want; ++i)
    if (P::get(&pl.state[i]) == INT_MAX) pl.list[r++] = i;
  P::sync();
  // the new tables and the copies
  for (int s = wid; s < p.n_slots; s += warps) {
    const int par = __ldcg(p.parent + s), keep = __ldcg(p.keep + s), grow = __ldcg(p.grow + s);
    const int32_t* old = p.table + (long long)(par < 0 ? 0 : par) * p.max_pages;
    int32_t* out = p.new_table + (long long)s * p.max_pages;
    const int whole = keep / p.page_size, rest = keep % p.page_size, kept = whole + (rest != 0);
    const int end = (int)(((long long)grow + p.page_size - 1) / p.page_size);
    const int off = sm.off[s], cp = sm.copy[s];
    for (int i = lane; i < p.max_pages; i += 32) {
      int pg = -1;
      if (i < whole || (i < kept && cp < 0)) {
        pg = __ldcg(old + i);
      } else if (i < end) {
        pg = P::get(&pl.list[off + i - whole - (cp < 0 && rest != 0 ? 1 : 0)]);
        if (i < kept) p.moves[cp] = Move{__ldcg(old + i), pg, rest, 0};
      }
      out[i] = pg;
    }
  }
  if (all == 0) p.head->n_moves = n_copies;
}

template <int CTAS>
__global__ void __launch_bounds__(kPlanThreads) k_pages_compact(const __grid_constant__ PlanArgs p) {
  __shared__ PlanSmem sm;
  using P = Plan<CTAS>;
  const P pl(p);
  const int tid = threadIdx.x, cta = blockIdx.x, all = cta * kPlanThreads + tid;
  const long long entries = (long long)p.n_slots * p.max_pages;
  pdl_wait();
  for (int i = all; i < p.n_pages; i += P::kAll) pl.state[i] = 0;
  if (all == 0) {
    p.head->bad = 0;
    p.head->n_moves = 0;
    p.head->below = 0;
  }
  P::sync();
  bool bad = false;
  for (long long i = all; i < entries; i += P::kAll) {
    const int pg = __ldcg(p.table + i);
    if (pg < -1 || pg >= p.n_pages)
      bad = true;
    else if (pg >= 0)
      pl.state[pg] = 1;
  }
  if (bad) p.head->bad = 1;
  P::sync();
  bad = __ldcg(&p.head->bad) != 0;
  int lo, hi, mine = 0;
  P::my_pages(p, cta, lo, hi);
  for (int i = lo; i < hi; ++i) mine += P::get(&pl.state[i]);
  const long long rank = block_scan(mine, sm);
  long long before, n_live;
  P::totals(p, sm, cta, before, n_live);
  if (bad) {
    if (all == 0) {
      atomicOr(p.err, kErrIndex);
      *p.n_live = -1;
    }
    return;  // every CTA of the cluster alike
  }
  // used pages before page n_live
  if (lo <= n_live && n_live < hi) {
    int b = (int)(before + rank);
    for (int i = lo; i < (int)n_live; ++i) b += P::get(&pl.state[i]);
    p.head->below = b;
  } else if (n_live == p.n_pages && all == 0) {
    p.head->below = p.n_pages;
  }
  P::sync();
  const int below = __ldcg(&p.head->below);
  // move i: the i-th used page at or behind n_live to the i-th unused one before it
  int used = (int)(before + rank);
  for (int i = lo; i < hi; ++i) {
    const int u = P::get(&pl.state[i]);
    if (i < n_live) {
      if (u == 0) {
        p.moves[i - used].dst = i;
        p.moves[i - used].rows = p.page_size;
      }
    } else if (u != 0) {
      p.moves[used - below].src = i;
      pl.state[i] = used - below;
    }
    used += u;
  }
  P::sync();
  for (long long i = all; i < entries; i += P::kAll) {
    const int pg = __ldcg(p.table + i);
    p.new_table[i] = pg < n_live ? pg : __ldcg(&p.moves[P::get(&pl.state[pg])].dst);
  }
  if (all == 0) {
    *p.n_live = (int)n_live;
    p.head->n_moves = (int)n_live - below;
  }
}

// The moves of a plan in every pool's K and V: a CTA copies pieces of 16 KB,
// all of a piece's loads in flight together, the next piece's move asked for
// before them.  Sources are kept pages and targets free ones, so no page is
// read and written.  Pieces are numbered move by move, then by pool and side,
// and dealt to the CTAs in turn.
__global__ void __launch_bounds__(kCopyThreads)
    k_pages_copy(const pages::Head* head, const Move* moves, int row_bytes, int pieces, int n_pools,
                 const __grid_constant__ pages::Pools pools, int64_t page_bytes) {
  pdl_wait();
  const int n_moves = __ldcg(&head->n_moves);
  const int per_move = 2 * n_pools * pieces;
  int m = (int)(blockIdx.x / per_move), at = (int)(blockIdx.x % per_move);
  const int dm = (int)(gridDim.x / per_move), dat = (int)(gridDim.x % per_move);
  auto load = [&](int i) { return __ldcg(reinterpret_cast<const int4*>(moves) + i); };  // src, dst, rows
  int4 next = m < n_moves ? load(m) : make_int4(0, 0, 0, 0);
  while (m < n_moves) {
    const int4 mv = next;
    const int side = at / pieces;
    const int64_t off = (int64_t)(at - side * pieces) * kPiece;
    m += dm;
    at += dat;
    if (at >= per_move) {
      at -= per_move;
      ++m;
    }
    if (m < n_moves) next = load(m);
    const int64_t bytes = (int64_t)mv.z * row_bytes;
    if (off >= bytes) continue;
    unsigned char* base = static_cast<unsigned char*>(pools.p[side]);
    const unsigned char* from = base + mv.x * page_bytes + off;
    unsigned char* to = base + mv.y * page_bytes + off;
    const int n = bytes - off < kPiece ? (int)(bytes - off) : kPiece;
    uint4 v[kCopyVecs];
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i) {
      const int o = 16 * ((int)threadIdx.x + i * kCopyThreads);
      if (o < n) v[i] = __ldcs(reinterpret_cast<const uint4*>(from + o));
    }
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i) {
      const int o = 16 * ((int)threadIdx.x + i * kCopyThreads);
      if (o < n) __stcs(reinterpret_cast<uint4*>(to + o), v[i]);
    }
  }
}

template <int CTAS>
cudaError_t launch_plan(bool remap, const PlanArgs& p, cudaStream_t st) {
  auto kern = remap ? k_pages_remap<CTAS> : k_pages_compact<CTAS>;
  const size_t smem = CTAS == 1 ? 2 * sizeof(int32_t) * (size_t)p.n_pages : 0;
  // without the attribute the pages' words and the plan's own shared memory
  // have 48 KB together
  if (smem > kPlanDefault) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(2 * sizeof(int32_t) * kSmallPages));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CTAS);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CTAS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_pages(const pages::Call& c, cudaStream_t st) {
  const pages::WsLayout L = pages::ws_layout(c.n_pages, c.n_slots);
  unsigned char* ws = static_cast<unsigned char*>(c.workspace);
  PlanArgs p = {};
  p.table = c.table;
  p.new_table = c.new_table;
  p.n_slots = c.n_slots;
  p.max_pages = c.max_pages;
  p.n_pages = (int32_t)c.n_pages;
  p.page_size = c.page_size;
  p.parent = c.parent;
  p.keep = c.keep;
  p.grow = c.grow;
  p.n_live = c.n_live;
  p.err = reinterpret_cast<uint32_t*>(ws);
  p.head = reinterpret_cast<pages::Head*>(ws + L.head);
  p.moves = reinterpret_cast<Move*>(ws + L.moves);
  p.state = reinterpret_cast<int32_t*>(ws + L.state);
  p.list = reinterpret_cast<int32_t*>(ws + L.list);
  const bool small = c.n_pages <= kSmallPages && (int64_t)c.n_slots * c.max_pages <= kSmallEntries;
  const bool remap = c.parent != nullptr;
  cudaError_t e = small ? launch_plan<1>(remap, p, st) : launch_plan<kPlanCtas>(remap, p, st);
  if (e != cudaSuccess) return e;
  const int64_t page_bytes = (int64_t)c.page_size * c.row_bytes;
  const int pieces = (int)((page_bytes + kPiece - 1) / kPiece);
  return launch_pdl(k_pages_copy, dim3(8 * device_sm_count()), dim3(kCopyThreads), 0, st,
                    static_cast<const pages::Head*>(p.head), static_cast<const Move*>(p.moves), (int)c.row_bytes, pieces,
                    c.n_pools, c.pools, page_bytes);
}

}  // namespace spark
