// pages.cu -- the page tables of a step (spark_pages_remap) and compaction
// (spark_pages_compact): a plan over the tables, then the copies it asks for.
//
// Who holds a page is computed from the tables of the call, not kept: a page
// is free when no slot keeps it.  One array `state` of a word per page says
//   remap    INT_MAX free, -1 kept whole by some slot, s >= 0 kept in part,
//            slot s the lowest of those that keep it so (an atomicMin, so the
//            outcome does not depend on the order of arrivals);
//   compact  0 unused, 1 used, then the page's rank among those that move.
// The plan is a few dependent passes over tables and pages of a few hundred
// KB at most in use: one cluster of 8 CTAs runs them, hardware cluster
// barriers between the passes, so a step costs one launch for the plan and
// one for the copies, which read the list of moves the plan left.
#include <limits.h>

#include "attn_parts.cuh"
#include "launch.h"
#include "pages.h"

namespace spark {
namespace {

using pages::Move;

constexpr int kPlanCtas = 8;
constexpr int kPlanThreads = 1024;
constexpr int kPlanAll = kPlanCtas * kPlanThreads;
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;                                   // 16-byte words per thread and piece
constexpr int kPiece = kCopyThreads * kCopyVecs * 16;          // bytes a CTA copies at a time

struct PlanSmem {
  long long sums[kPlanThreads / 32];
  long long total;
  int off[SPARK_MAX_BATCH];   // first new page of each slot
  int copy[SPARK_MAX_BATCH];  // its index among the copies, or -1
};

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

// the range of pages a thread of the cluster counts
__device__ __forceinline__ void my_pages(const PlanArgs& p, int cta, int& lo, int& hi) {
  const long long n = p.n_pages, i = (long long)cta * kPlanThreads + threadIdx.x;
  lo = (int)(n * i / kPlanAll);
  hi = (int)(n * (i + 1) / kPlanAll);
}

// pages counted by the CTAs before this one, and by all (after a cluster barrier)
__device__ __forceinline__ void cta_totals(const PlanArgs& p, int cta, long long& before, long long& all) {
  before = all = 0;
  for (int c = 0; c < kPlanCtas; ++c) {
    const int t = __ldcg(&p.head->totals[c]);
    if (c < cta) before += t;
    all += t;
  }
}

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    k_pages_remap(const __grid_constant__ PlanArgs p) {
  __shared__ PlanSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, cta = blockIdx.x;
  const int all = cta * kPlanThreads + tid, warps = kPlanAll / 32, wid = all >> 5;
  pdl_wait();
  for (int i = all; i < p.n_pages; i += kPlanAll) p.state[i] = INT_MAX;
  if (all == 0) {
    p.head->bad = 0;
    p.head->n_moves = 0;
  }
  cluster_sync_all();
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
        else if (i < whole)
          p.state[pg] = -1;  // the lowest value there is: no order of arrival matters
        else
          atomicMin(&p.state[pg], s);
      }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) p.head->bad = 1;
  }
  cluster_sync_all();
  const bool bad = __ldcg(&p.head->bad) != 0;  // the same in every CTA
  // pages each slot needs, and where they start among all new pages (every
  // CTA for itself: n_slots <= the block)
  int need = 0, copied = 0;
  if (!bad && tid < p.n_slots) {
    const int keep = __ldcg(p.keep + tid), grow = __ldcg(p.grow + tid);
    const int rest = keep % p.page_size;
    if (rest != 0) {
      const int pg = __ldcg(p.table + (long long)__ldcg(p.parent + tid) * p.max_pages + keep / p.page_size);
      copied = __ldcg(&p.state[pg]) != tid;
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
  my_pages(p, cta, lo, hi);
  for (int i = lo; i < hi; ++i) mine += __ldcg(&p.state[i]) == INT_MAX;
  const long long rank = block_scan(mine, sm);
  if (tid == 0) p.head->totals[cta] = (int)sm.total;
  cluster_sync_all();
  long long before, free_all;
  cta_totals(p, cta, before, free_all);
  if (bad || want > free_all) {
    if (all == 0) atomicOr(p.err, bad ? kErrIndex : kErrPages);
    return;  // every CTA of the cluster alike
  }
  long long r = before + rank;
  for (int i = lo; i < hi && r < want; ++i)
    if (__ldcg(&p.state[i]) == INT_MAX) p.list[r++] = i;
  cluster_sync_all();
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
        pg = __ldcg(&p.list[off + i - whole - (cp < 0 && rest != 0 ? 1 : 0)]);
        if (i < kept) p.moves[cp] = Move{__ldcg(old + i), pg, rest, 0};
      }
      out[i] = pg;
    }
  }
  if (all == 0) p.head->n_moves = n_copies;
}

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    k_pages_compact(const __grid_constant__ PlanArgs p) {
  __shared__ PlanSmem sm;
  const int tid = threadIdx.x, cta = blockIdx.x, all = cta * kPlanThreads + tid;
  const long long entries = (long long)p.n_slots * p.max_pages;
  pdl_wait();
  for (int i = all; i < p.n_pages; i += kPlanAll) p.state[i] = 0;
  if (all == 0) {
    p.head->bad = 0;
    p.head->n_moves = 0;
    p.head->below = 0;
  }
  cluster_sync_all();
  bool bad = false;
  for (long long i = all; i < entries; i += kPlanAll) {
    const int pg = __ldcg(p.table + i);
    if (pg < -1 || pg >= p.n_pages)
      bad = true;
    else if (pg >= 0)
      p.state[pg] = 1;
  }
  if (bad) p.head->bad = 1;
  cluster_sync_all();
  bad = __ldcg(&p.head->bad) != 0;
  int lo, hi, mine = 0;
  my_pages(p, cta, lo, hi);
  for (int i = lo; i < hi; ++i) mine += __ldcg(&p.state[i]);
  const long long rank = block_scan(mine, sm);
  if (tid == 0) p.head->totals[cta] = (int)sm.total;
  cluster_sync_all();
  long long before, n_live;
  cta_totals(p, cta, before, n_live);
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
    for (int i = lo; i < (int)n_live; ++i) b += __ldcg(&p.state[i]);
    p.head->below = b;
  } else if (n_live == p.n_pages && all == 0) {
    p.head->below = p.n_pages;
  }
  cluster_sync_all();
  const int below = __ldcg(&p.head->below);
  // move i: the i-th used page at or behind n_live to the i-th unused one before it
  int used = (int)(before + rank);
  for (int i = lo; i < hi; ++i) {
    const int u = __ldcg(&p.state[i]);
    if (i < n_live) {
      if (u == 0) {
        p.moves[i - used].dst = i;
        p.moves[i - used].rows = p.page_size;
      }
    } else if (u != 0) {
      p.moves[used - below].src = i;
      p.state[i] = used - below;
    }
    used += u;
  }
  cluster_sync_all();
  for (long long i = all; i < entries; i += kPlanAll) {
    const int pg = __ldcg(p.table + i);
    p.new_table[i] = pg < n_live ? pg : __ldcg(&p.moves[__ldcg(&p.state[pg])].dst);
  }
  if (all == 0) {
    *p.n_live = (int)n_live;
    p.head->n_moves = (int)n_live - below;
  }
}

// The moves of a plan in every pool's K and V: a CTA copies pieces of 16 KB,
// all of a piece's loads in flight together.  Sources are kept pages and
// targets free ones, so no page is read and written.
__global__ void __launch_bounds__(kCopyThreads)
    k_pages_copy(const pages::Head* head, const Move* moves, int row_bytes, int pieces, int n_pools,
                 const __grid_constant__ pages::Pools pools, int64_t page_bytes) {
  pdl_wait();
  const int n_moves = __ldcg(&head->n_moves);
  const int sides = 2 * n_pools;
  const int64_t units = (int64_t)n_moves * sides * pieces;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int piece = (int)(u % pieces);
    const int64_t w = u / pieces;
    const int side = (int)(w % sides), m = (int)(w / sides);
    const int src = __ldcg(&moves[m].src), dst = __ldcg(&moves[m].dst), rows = __ldcg(&moves[m].rows);
    const int64_t bytes = (int64_t)rows * row_bytes, at = (int64_t)piece * kPiece;
    if (at >= bytes) continue;
    unsigned char* base = static_cast<unsigned char*>(pools.p[side]);
    const unsigned char* from = base + src * page_bytes + at;
    unsigned char* to = base + dst * page_bytes + at;
    uint4 v[kCopyVecs];
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i) {
      const int64_t o = 16 * (threadIdx.x + (int64_t)i * kCopyThreads);
      if (at + o < bytes) v[i] = __ldcs(reinterpret_cast<const uint4*>(from + o));
    }
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i) {
      const int64_t o = 16 * (threadIdx.x + (int64_t)i * kCopyThreads);
      if (at + o < bytes) __stcs(reinterpret_cast<uint4*>(to + o), v[i]);
    }
  }
}

cudaError_t launch_plan(void (*kern)(PlanArgs), const PlanArgs& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
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
  cudaError_t e = launch_plan(c.parent ? k_pages_remap : k_pages_compact, p, st);
  if (e != cudaSuccess) return e;
  const int64_t page_bytes = (int64_t)c.page_size * c.row_bytes;
  const int pieces = (int)((page_bytes + kPiece - 1) / kPiece);
  return launch_pdl(k_pages_copy, dim3(8 * device_sm_count()), dim3(kCopyThreads), 0, st,
                    static_cast<const pages::Head*>(p.head), static_cast<const Move*>(p.moves), (int)c.row_bytes, pieces,
                    c.n_pools, c.pools, page_bytes);
}

}  // namespace spark
