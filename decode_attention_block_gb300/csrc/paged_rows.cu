// paged_rows.cu -- rows of tokens into and out of pages beside the plain copy
// of paged_attn.cu: the append with the rotation of queries and keys on the
// way, the write and the read of 4-bit pages, and the table of rope angles.
//
// A warp takes one token, or a share of its rows where the tokens are few: finds
// where it lies, then takes its rows (query heads, key heads, value heads), a lane 8
// dims of each: a row is one load and one store of the warp, and the two halves of
// a rotated pair that lie in other lanes come by a shuffle.  The first rows are
// asked for before the token's place is looked up, a few more at a time after.
//
// Measured (in a graph): one token, 24 rows, 3.3 to 3.9 us; 64 into 4-bit pages 4.7;
// 9400 tokens of prompts, bf16, all dims rotated, into 4-bit pages 50 (4.0 TB/s; bf16
// pages 46, fp32 50, 5.0 and 5.4 TB/s), with 65% of issue slots and 43% of DRAM busy
// at a third of the warps; their k and v alone 21 (16, 25), out again 10 (13, 19);
// 47000 rows of prefixes out of 4-bit pages 41 (0.23 GB: 5.7 TB/s).
#include <math.h>

#include <type_traits>

#include "fp4.cuh"
#include "launch.h"
#include "paged_launch.h"
#include "paged_parts.cuh"

namespace spark {
namespace {

using paged::Args;

constexpr int kRowWarps = 4;      // of a CTA (9000 tokens of prompts in and out again 61.2 us, with 8 62.3, with 2 60.8)
constexpr int kRowThreads = 32 * kRowWarps;
constexpr int kWantedWarps = 32;  // an SM, before a token has a warp alone
constexpr int kRowCtas = 6;       // CTAs an SM of the append (32 warps: 64 registers, spilled: 8 prompts no faster)
constexpr int kBatch = 2;         // rows of a warp in flight, behind the two being rotated (8 prompts: with 1 10 us more, with 3 as many)
constexpr int kReadBatch = 8;
// Tokens of a warp of a long read: 47000 rows 47.7 us with one, 41.5 with two, 43
// with three, 47.5 with four (the writes spread), 10 CTAs an SM.
constexpr int kReadTokens = 2;
constexpr int kReadCtas = 10;
constexpr int kReadWarps = 24;    // an SM at least, for that (9000 tokens: two 2 us less)

// The warp's token and its rows: first, first + step, ..
struct Task {
  int token, first, step;
  __device__ __forceinline__ explicit Task(int split) {
    const int w = blockIdx.x * kRowWarps + (int)(threadIdx.x >> 5);
    token = w / split;
    first = w - token * split;
    step = split;
  }
};

// Where a token's row lies: position -1 where it belongs to no sequence, or
// to one whose entries make no sense.
struct Place {
  int pos, page, row;
};

// The sequence that token t belongs to, if any does, by a warp: 32 starts a step.
__device__ __forceinline__ int find_seq(const Args& p, int t, int lane) {
  int lo = 0, n = p.n_seqs;  // the last start at or before t is one of lo .. lo + n - 1, or none is
  while (n > 1) {
    const int step = (n + 31) / 32, s = lo + lane * step;
    const bool before = lane * step < n && __ldcg(p.q_start + s) <= t;
    const unsigned m = __ballot_sync(0xffffffffu, before);
    const int last = m == 0 ? 0 : 31 - __clz(m);
    lo += last * step;
    n = min(step, n - last * step);
    if (step == 1) break;
  }
  return lo;
}
// token t's place, of sequence i; `report` a bad entry
__device__ __forceinline__ Place place_in(const Args& p, int i, const paged::Seq& s, int t, bool report) {
  Place at = {-1, -1, 0};
  if (t < s.q0 || t >= s.q0 + s.n) return at;
  at.pos = s.p0 + (t - s.q0);
  const int pg = paged::page_entry(p, i, paged::page_col(p, at.pos));
  if (pg < 0 || pg >= p.n_pages) {
    if (report) atomicOr(p.err, kErrIndex);
    at.pos = -1;
    return at;
  }
  at.page = pg;
  at.row = paged::page_row(p, at.pos);
  return at;
}
__device__ __forceinline__ Place find_place(const Args& p, int t, int lane) {
  const int i = find_seq(p, t, lane);
  return place_in(p, i, paged::load_seq(p, i), t, lane == 0);
}

// every sequence is looked at, also one that no token's search ends in
__device__ __forceinline__ void report_bad(const Args& p) {
  for (int s = blockIdx.x * kRowThreads + (int)threadIdx.x; s < p.n_seqs; s += gridDim.x * kRowThreads)
    if (paged::load_seq(p, s).bad) atomicOr(p.err, kErrIndex);
}

// eight elements, as they are loaded
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcg(reinterpret_cast<const float4*>(p));
    b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
  }
};
template <>
struct Raw<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldcg(reinterpret_cast<const uint4*>(p)); }
};
__device__ __forceinline__ void widen(float (&x)[8], const Raw<float>& r) {
  x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w; x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
__device__ __forceinline__ void widen(float (&x)[8], const Raw<__nv_bfloat16>& r) {
  const uint4 v = r.v;
  const float2 a = bf16x2_to_f32x2(v.x), b = bf16x2_to_f32x2(v.y), c = bf16x2_to_f32x2(v.z), d = bf16x2_to_f32x2(v.w);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y; x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
}
__device__ __forceinline__ void put8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void put8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

struct Fp4 {};  // the type of 4-bit pages

// a c - b s rounded once: both products with their errors (fma), their
// difference with its error (Knuth's two-sum), the errors added at the end.
// A 4-bit code then is that of the exact rotation, but for a value within
// 2^-45 or so of a border.
__device__ __forceinline__ float turned(float a, float c, float b, float s) {
  const float p = __fmul_rn(a, c), pe = __fmaf_rn(a, c, -p);
  const float q = -__fmul_rn(b, s), qe = -__fmaf_rn(b, s, q);
  const float sum = __fadd_rn(p, q), z = __fsub_rn(sum, p);
  const float err = __fadd_rn(__fsub_rn(p, __fsub_rn(sum, z)), __fsub_rn(q, z));
  const float r = __fadd_rn(sum, __fadd_rn(err, __fadd_rn(pe, qe)));
  return fabsf(sum) < INFINITY ? r : sum;
}

// a c - b s within 1.5 ulp whatever cancels (Kahan's way with fma; the bound:
// Jeannerod, Louvet and Muller 2013): four operations where turned takes fifteen,
// of which a prompt's time was (9000 tokens, 24 rows each: 61 us, now 52).
__device__ __forceinline__ float turned_near(float a, float c, float b, float s) {
  const float w = __fmul_rn(b, s);
  return __fadd_rn(__fmaf_rn(a, c, -w), __fmaf_rn(-b, s, w));
}
template <bool EXACT>
__device__ __forceinline__ float turned_as(float a, float c, float b, float s) {
  return EXACT ? turned(a, c, b, s) : turned_near(a, c, b, s);
}

__device__ __forceinline__ Raw<float> shuffle(const Raw<float>& r, int from) {
  Raw<float> o;
  o.a = make_float4(__shfl_sync(0xffffffffu, r.a.x, from), __shfl_sync(0xffffffffu, r.a.y, from),
                    __shfl_sync(0xffffffffu, r.a.z, from), __shfl_sync(0xffffffffu, r.a.w, from));
  o.b = make_float4(__shfl_sync(0xffffffffu, r.b.x, from), __shfl_sync(0xffffffffu, r.b.y, from),
                    __shfl_sync(0xffffffffu, r.b.z, from), __shfl_sync(0xffffffffu, r.b.w, from));
  return o;
}
__device__ __forceinline__ Raw<__nv_bfloat16> shuffle(const Raw<__nv_bfloat16>& r, int from) {
  Raw<__nv_bfloat16> o;
  o.v = make_uint4(__shfl_sync(0xffffffffu, r.v.x, from), __shfl_sync(0xffffffffu, r.v.y, from),
                   __shfl_sync(0xffffffffu, r.v.z, from), __shfl_sync(0xffffffffu, r.v.w, from));
  return o;
}

// A row's rotation: lane l has dims 8 l .. 8 l + 7.  VEC: r is a multiple of 16,
// so that eight dims' partners lie in one lane, and their (cos, sin) stay for
// all rows of the token.
template <bool VEC>
struct Turn {
  float c[8], s[8];  // s negative for the second half of a pair
  int half, from;    // the partner's lane
  const float* cs;
  bool on;
  __device__ __forceinline__ void init(const float* rope, int pos, int half_, int lane) {
    half = half_;
    cs = rope + (int64_t)pos * 2 * half;
    if constexpr (VEC) {
      const int d = 8 * lane, lanes = half / 8;
      on = d < 2 * half;
      const bool second = d >= half;
      from = on ? (second ? lane - lanes : lane + lanes) : lane;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = 1.f;
        s[i] = 0.f;
      }
      if (on) {
        const float4* src = reinterpret_cast<const float4*>(cs + 2 * (second ? d - half : d));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = __ldg(src + i);
          c[2 * i] = v.x; s[2 * i] = second ? -v.y : v.y;
          c[2 * i + 1] = v.z; s[2 * i + 1] = second ? -v.w : v.w;
        }
      }
    }
  }
  // The row's eight dims, rotated.  src: the row in memory, where the partners
  // are read from without VEC.
  template <bool EXACT, typename XT>
  __device__ __forceinline__ void apply(float (&x)[8], const Raw<XT>& raw, const XT* src, int lane) const {
    widen(x, raw);
    if constexpr (VEC) {
      float y[8];
      widen(y, shuffle(raw, from));
      if (on)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = turned_as<EXACT>(x[i], c[i], y[i], s[i]);
    } else {
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const int d = 8 * lane + i;
        if (d >= 2 * half) break;
        const bool second = d >= half;
        const int e = second ? d - half : d;
        const float y = (float)src[second ? e : e + half];
        const float co = __ldg(cs + 2 * e), si = __ldg(cs + 2 * e + 1);
        float mine = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) mine = k == i ? x[k] : mine;
        mine = turned_as<EXACT>(mine, co, y, second ? -si : si);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = k == i ? mine : x[k];
      }
    }
  }
};

// Eight dims of a row into its page, by the whole warp.
template <typename CT>
__device__ __forceinline__ void put_row(unsigned char* pool, const Args& p, const Place& at, int head, const float (&x)[8],
                                        int lane) {
  put8(reinterpret_cast<CT*>(pool) + (((int64_t)at.page * p.page_size + at.row) * p.n_kv + head) * kHeadDim + 8 * lane, x);
}
template <>
__device__ __forceinline__ void put_row<Fp4>(unsigned char* pool, const Args& p, const Place& at, int head,
                                             const float (&x)[8], int lane) {
  float m = 0.f;
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    fine = fine && fabsf(x[i]) < INFINITY;
    m = fmaxf(m, fabsf(x[i]));
  }
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  fine = __shfl_xor_sync(0xffffffffu, (int)fine, 1) && fine;
  const uint32_t b = fine ? fp4::scale_of(m) : fp4::kScaleNan;
  const float s = fine ? fp4::scale_value(b) : 1.0f;
  // x / s rounded to fp32, by a step of Newton's for the quotient (Markstein):
  // with r = 1 / s rounded, q = x r is off by 2^-22 of the quotient at most, the
  // remainder x - q s is exact, and q + r (x - q s) off by 2^-44 before its
  // rounding.  s has 4 significant bits, so an x / s that is no tie of fp32's lies
  // 2^-29 of itself or more from one: the rounding is that of x / s.
  const float r = b == 0 ? 0.f : __frcp_rn(s);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = __fmul_rn(x[i], r);
    y[i] = __fmaf_rn(-__fmaf_rn(q, s, -x[i]), r, q);
  }
  unsigned char* block = pool + fp4::block_at(at.page, at.row, head, p.page_size, p.n_kv);
  const int row = at.row % fp4::kRows;
  *reinterpret_cast<uint32_t*>(block + fp4::code_at(row, 8 * lane)) = fp4::codes8(y);
  if ((lane & 1) == 0) block[fp4::scale_at(row, 8 * lane)] = (unsigned char)b;
}

// Eight dims of a row of a page, as they are loaded.
template <typename CT>
struct PageRow {
  Raw<CT> raw;
  __device__ __forceinline__ void load(const unsigned char* pool, const Args& p, const Place& at, int head, int lane) {
    raw.load(reinterpret_cast<const CT*>(pool) + (((int64_t)at.page * p.page_size + at.row) * p.n_kv + head) * kHeadDim + 8 * lane);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const { widen(x, raw); }
};
template <>
struct PageRow<Fp4> {
  uint32_t codes, scale;
  __device__ __forceinline__ void load(const unsigned char* pool, const Args& p, const Place& at, int head, int lane) {
    const unsigned char* block = pool + fp4::block_at(at.page, at.row, head, p.page_size, p.n_kv);
    const int row = at.row % fp4::kRows;
    codes = __ldcg(reinterpret_cast<const uint32_t*>(block + fp4::code_at(row, 8 * lane)));
    scale = __ldcg(block + fp4::scale_at(row, 8 * lane));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const float s = fp4::scale_value(scale);
    uint32_t h[4];
    fp4::halves8(codes, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = fp4::unpack(h[i]);
      x[2 * i] = f.x * s;
      x[2 * i + 1] = f.y * s;
    }
  }
};

// half 0: no rotation; q null: keys and values alone.
template <typename XT, typename CT, bool VEC>
__global__ void __launch_bounds__(kRowThreads, kRowCtas)
    k_paged_rope(const XT* q, const XT* k, const XT* v, int64_t ld, const float* rope, int half, int n_positions, XT* q_out,
                 int64_t q_out_ld, unsigned char* pk, unsigned char* pv, int split, const __grid_constant__ Args p) {
  const int lane = threadIdx.x & 31;
  const Task task(split);
  pdl_wait();
  // no early trigger: a kernel that reads pages before its own wait must not
  // start before these rows are written
  report_bad(p);
  if (task.token >= p.n_tokens) return;
  const int64_t t = task.token;
  const int n_q = q == nullptr ? 0 : kGroup * p.n_kv, rows = n_q + 2 * p.n_kv;
  auto source = [&](int r) {
    const bool is_q = r < n_q, is_k = !is_q && r < n_q + p.n_kv;
    return (is_q ? q + r * kHeadDim : is_k ? k + (r - n_q) * kHeadDim : v + (r - n_q - p.n_kv) * kHeadDim) + t * ld;
  };
  Raw<XT> raw[kBatch];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (r0 + i * task.step < rows) raw[i].load(source(r0 + i * task.step) + 8 * lane);
  };
  load(task.first);
  const Place at = find_place(p, task.token, lane);
  if (at.pos < 0) return;
  Turn<VEC> turn;
  if (half > 0) {
    if (at.pos >= n_positions) {
      if (lane == 0) atomicOr(p.err, kErrIndex);
      return;
    }
    turn.init(rope, at.pos, half, lane);
  }
  for (int r0 = task.first; r0 < rows; r0 += kBatch * task.step) {
    Raw<XT> now[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) now[i] = raw[i];
    load(r0 + kBatch * task.step);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * task.step;
      if (r >= rows) break;
      float x[8];
      if (r < n_q) {
        if (half > 0)
          turn.template apply<false>(x, now[i], source(r), lane);
        else
          widen(x, now[i]);
        __syncwarp();  // (in place, a row's partners are read before any is written)
        put8(q_out + t * q_out_ld + r * kHeadDim + 8 * lane, x);
        continue;
      }
      const bool is_k = r < n_q + p.n_kv;
      // (4-bit codes are those of the exact rotation)
      if (half > 0 && is_k)
        turn.template apply<std::is_same<CT, Fp4>::value>(x, now[i], source(r), lane);
      else
        widen(x, now[i]);
      put_row<CT>(is_k ? pk : pv, p, at, is_k ? r - n_q : r - n_q - p.n_kv, x, lane);
    }
  }
}

template <typename XT, typename CT>
__global__ void __launch_bounds__(kRowThreads)
    k_paged_read(const unsigned char* pk, const unsigned char* pv, XT* k, XT* v, int64_t ld, int split,
                 const __grid_constant__ Args p) {
  const int lane = threadIdx.x & 31;
  const Task task(split);
  pdl_wait();
  report_bad(p);
  if (task.token >= p.n_tokens) return;
  const Place at = find_place(p, task.token, lane);
  if (at.pos < 0) return;
  // row r: K of head r / 2, then V
  for (int r0 = task.first; r0 < 2 * p.n_kv; r0 += kReadBatch * task.step) {
    PageRow<CT> row[kReadBatch];
#pragma unroll
    for (int i = 0; i < kReadBatch; ++i) {
      const int r = r0 + i * task.step;
      if (r < 2 * p.n_kv) row[i].load((r & 1) ? pv : pk, p, at, r >> 1, lane);
    }
#pragma unroll
    for (int i = 0; i < kReadBatch; ++i) {
      const int r = r0 + i * task.step;
      if (r >= 2 * p.n_kv) break;
      float x[8];
      row[i].get(x);
      put8(((r & 1) ? v : k) + task.token * ld + (r >> 1) * kHeadDim + 8 * lane, x);
    }
  }
}

__global__ void __launch_bounds__(256) k_rope_table(float2* rope, int64_t n, int half, double theta, int r) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= n) return;
  const int i = (int)(e % half);
  double s, c;
  sincos((double)(e / half) * pow(theta, -2.0 * i / (double)r), &s, &c);
  rope[e] = make_float2((float)c, (float)s);
}

// warps that share a token's rows
int split_for(int n_tokens, int rows) {
  int split = kWantedWarps * device_sm_count() / n_tokens;
  if (split > 8) split = 8;
  if (split > rows) split = rows;
  return split < 1 ? 1 : split;
}
dim3 row_grid(int n_tokens, int split) { return dim3((unsigned)(((int64_t)n_tokens * split + kRowWarps - 1) / kRowWarps)); }

template <typename XT, typename CT>
cudaError_t rope_t(const Args& p, const paged::RopeRows& a, cudaStream_t st) {
  auto kern = a.half % 8 == 0 ? k_paged_rope<XT, CT, true> : k_paged_rope<XT, CT, false>;
  const int split = split_for(p.n_tokens, (a.q ? kGroup + 2 : 2) * p.n_kv);
  return launch_pdl(kern, row_grid(p.n_tokens, split), dim3(kRowThreads), 0, st, static_cast<const XT*>(a.q),
                    static_cast<const XT*>(a.k), static_cast<const XT*>(a.v), a.ld, a.rope, a.half, a.n_positions,
                    static_cast<XT*>(a.q_out), a.q_out_ld, static_cast<unsigned char*>(a.pk),
                    static_cast<unsigned char*>(a.pv), split, p);
}

// The same of kReadTokens tokens a warp: their places are looked up at once, a lane
// each, and a token's rows are on their way while the one before is written.
template <typename XT>
__global__ void __launch_bounds__(kRowThreads, kReadCtas)
    k_paged_read_run(const unsigned char* pk, const unsigned char* pv, XT* k, XT* v, int64_t ld, const __grid_constant__ Args p) {
  const int lane = threadIdx.x & 31;
  const int t0 = (int)(blockIdx.x * kRowWarps * kReadTokens + (threadIdx.x >> 5));  // and every kRowWarps-th behind it
  pdl_wait();
  report_bad(p);
  if (t0 >= p.n_tokens) return;
  const int i0 = find_seq(p, t0, lane);
  const paged::Seq s = paged::load_seq(p, i0);
  Place mine = {-1, -1, 0};
  if (lane < kReadTokens) mine = place_in(p, i0, s, t0 + lane * kRowWarps, true);
  PageRow<Fp4> row[2][kReadBatch];
  Place at[2];
  auto load = [&](int i, Place& to, PageRow<Fp4> (&x)[kReadBatch]) {
    to.pos = __shfl_sync(0xffffffffu, mine.pos, i);
    to.page = __shfl_sync(0xffffffffu, mine.page, i);
    to.row = __shfl_sync(0xffffffffu, mine.row, i);
    const int t = t0 + i * kRowWarps;
    if (t >= p.n_tokens)
      to.pos = -1;
    else if (t >= s.q0 + s.n)
      to = find_place(p, t, lane);  // another sequence's
    if (to.pos < 0) return;
#pragma unroll
    for (int r = 0; r < kReadBatch; ++r)
      if (r < 2 * p.n_kv) x[r].load((r & 1) ? pv : pk, p, to, r >> 1, lane);
  };
  load(0, at[0], row[0]);
#pragma unroll
  for (int i = 0; i < kReadTokens; ++i) {
    if (i + 1 < kReadTokens) load(i + 1, at[(i + 1) & 1], row[(i + 1) & 1]);
    if (at[i & 1].pos < 0) continue;
#pragma unroll
    for (int r = 0; r < kReadBatch; ++r) {
      if (r >= 2 * p.n_kv) break;
      float x[8];
      row[i & 1][r].get(x);
      put8(((r & 1) ? v : k) + (t0 + i * kRowWarps) * ld + (r >> 1) * kHeadDim + 8 * lane, x);
    }
  }
}

template <typename XT, typename CT>
cudaError_t read_t(const Args& p, const void* pk, const void* pv, void* k, void* v, int64_t ld, cudaStream_t st) {
  const int split = split_for(p.n_tokens, 2 * p.n_kv);
  // (4-bit rows: two registers each)
  if constexpr (std::is_same<CT, Fp4>::value)
    if (2 * p.n_kv <= kReadBatch && p.n_tokens / kReadTokens >= kReadWarps * device_sm_count())
      return launch_pdl(k_paged_read_run<XT>, row_grid((p.n_tokens + kReadTokens - 1) / kReadTokens, 1), dim3(kRowThreads), 0, st,
                        static_cast<const unsigned char*>(pk), static_cast<const unsigned char*>(pv), static_cast<XT*>(k),
                        static_cast<XT*>(v), ld, p);
  return launch_pdl(k_paged_read<XT, CT>, row_grid(p.n_tokens, split), dim3(kRowThreads), 0, st,
                    static_cast<const unsigned char*>(pk), static_cast<const unsigned char*>(pv), static_cast<XT*>(k),
                    static_cast<XT*>(v), ld, split, p);
}

}  // namespace

cudaError_t launch_paged_rope(const paged::Args& p, int xdtype, int cdtype, const paged::RopeRows& a, cudaStream_t st) {
  const bool bf = xdtype == SPARK_BF16;
  if (cdtype == SPARK_FP4) return bf ? rope_t<__nv_bfloat16, Fp4>(p, a, st) : rope_t<float, Fp4>(p, a, st);
  if (cdtype == SPARK_BF16)
    return bf ? rope_t<__nv_bfloat16, __nv_bfloat16>(p, a, st) : rope_t<float, __nv_bfloat16>(p, a, st);
  return bf ? rope_t<__nv_bfloat16, float>(p, a, st) : rope_t<float, float>(p, a, st);
}

cudaError_t launch_paged_read(const paged::Args& p, int xdtype, int cdtype, const void* pk, const void* pv, void* k,
                              void* v, int64_t ld, cudaStream_t st) {
  const bool bf = xdtype == SPARK_BF16;
  if (cdtype == SPARK_FP4)
    return bf ? read_t<__nv_bfloat16, Fp4>(p, pk, pv, k, v, ld, st) : read_t<float, Fp4>(p, pk, pv, k, v, ld, st);
  if (cdtype == SPARK_BF16)
    return bf ? read_t<__nv_bfloat16, __nv_bfloat16>(p, pk, pv, k, v, ld, st)
              : read_t<float, __nv_bfloat16>(p, pk, pv, k, v, ld, st);
  return bf ? read_t<__nv_bfloat16, float>(p, pk, pv, k, v, ld, st) : read_t<float, float>(p, pk, pv, k, v, ld, st);
}

cudaError_t launch_rope_table(float* rope, int n_positions, int rotary_dim, double theta, cudaStream_t st) {
  const int64_t n = (int64_t)n_positions * (rotary_dim / 2);
  k_rope_table<<<dim3((unsigned)((n + 255) / 256)), 256, 0, st>>>(reinterpret_cast<float2*>(rope), n, rotary_dim / 2, theta,
                                                                  rotary_dim);
  return cudaGetLastError();
}

}  // namespace spark
