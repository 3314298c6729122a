// score.cu -- log probabilities of given tokens, entropy and the highest
// alternatives of rows of logits (spark_token_logprobs).
//
// One pass over the logits: each thread keeps a running maximum m, the sum
// z = sum e^(x - m) and u = sum (x - m) e^(x - m), which a higher maximum
// m + d turns into z e^-d and (u - d z) e^-d; then logprob = x_t - m - ln z
// and entropy = ln z - u / z.  Bound by the logits' bytes: 4 (or 2) per
// element against about eight operations.  Few rows are split over the
// vocabulary; the last CTA of a row to arrive joins the parts in order.
//
// The alternatives ride along.  A logit and its index form one 64-bit key
// (value order first, then the lower index), so all keys differ and the
// outcome does not depend on any order of arrival.  The CTA holds its best k
// keys so far; after a row's first tile hardly a thread finds a larger one.  A
// tile that does brings its candidates to shared memory, at most kBufThreads
// threads' worth: where more threads hold one, a bound is found first, by
// bisection over the threads' largest keys, that k to kBufThreads of them reach.
#include <math.h>

#include "launch.h"
#include "score.h"

namespace spark {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;            // 16-byte words per thread and tile
constexpr int kBufThreads = 64;     // threads whose candidates fit the buffer
constexpr int kMaxK = SPARK_MAX_TOP;

using Key = unsigned long long;

__device__ __forceinline__ Key make_key(float x, uint32_t idx) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 and 0 are equal logits
  const uint32_t o = x != x ? 0u : (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((Key)o << 32) | (0xFFFFFFFFu - idx);
}
__device__ __forceinline__ float key_value(Key k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return o == 0u ? __uint_as_float(0x7FC00000u) : __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int32_t key_index(Key k) { return (int32_t)(0xFFFFFFFFu - (uint32_t)k); }

struct Stat {
  float m, z, u;
  int bad;  // a NaN or +inf among the logits
};

__device__ __forceinline__ Stat join(const Stat& a, const Stat& b) {
  Stat r;
  r.m = fmaxf(a.m, b.m);
  r.bad = a.bad | b.bad;
  const float ref = r.m == -INFINITY ? 0.f : r.m;
  const float da = a.m == -INFINITY ? 0.f : a.m - ref, db = b.m == -INFINITY ? 0.f : b.m - ref;
  const float ea = expf(da), eb = expf(db);
  r.z = fmaf(a.z, ea, b.z * eb);
  // (a mask of the type's lowest value: e = 0, and d z may overflow)
  r.u = (ea > 0.f ? (a.u + da * a.z) * ea : 0.f) + (eb > 0.f ? (b.u + db * b.z) * eb : 0.f);
  return r;
}

__device__ __forceinline__ Stat warp_join(Stat s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat t;
    t.m = __shfl_xor_sync(0xffffffffu, s.m, o);
    t.z = __shfl_xor_sync(0xffffffffu, s.z, o);
    t.u = __shfl_xor_sync(0xffffffffu, s.u, o);
    t.bad = __shfl_xor_sync(0xffffffffu, s.bad, o);
    s = join(s, t);
  }
  return s;
}

struct Smem {
  Stat stat[kThreads / 32];
  Key best[2][kMaxK];
  Key buf[kBufThreads * 16 + kMaxK];
  int count, which, last;
};

// Fold the block's keys (N per thread, 0 for none) into the best k: into
// sm.best[sm.which], in descending order.
template <int N>
__device__ __forceinline__ void fold_top(Smem& sm, const Key (&key)[N], int k) {
  static_assert(N <= 16, "the buffer holds 16 keys a thread");
  const int tid = threadIdx.x;
  Key least = sm.best[sm.which][k - 1];  // 0 while there are fewer than k
  Key mine = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) mine = key[i] > mine ? key[i] : mine;
  const int have = __syncthreads_count(mine > least);
  if (have == 0) return;
  if (have > kBufThreads) {
    // the highest bound found that at least k threads' largest keys reach
    Key lo = least, hi = ~0ull;  // count(>= lo + 1) = have > kBufThreads; count(>= hi) < k
    for (int it = 0; it < 64; ++it) {
      const Key mid = lo + (hi - lo) / 2;
      const int n = __syncthreads_count(mine > mid);
      if (n >= k) {
        lo = mid;
        if (n <= kBufThreads) break;
      } else {
        hi = mid;
      }
    }
    least = lo;
  }
  if (tid == 0) sm.count = 0;
  __syncthreads();
  if (mine > least) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (key[i] > least) sm.buf[atomicAdd(&sm.count, 1)] = key[i];
  }
  const Key* old = sm.best[sm.which];
  Key* out = sm.best[sm.which ^ 1];
  __syncthreads();
  const int n0 = sm.count;
  if (tid < k) sm.buf[n0 + tid] = old[tid];  // the best so far compete with them
  __syncthreads();
  const int n = n0 + k;
  for (int i = tid; i < n; i += kThreads) {
    const Key x = sm.buf[i];
    int rank = 0;
    // empty places (0) are equal: ordered by their place
    for (int j = 0; j < n; ++j) rank += sm.buf[j] > x || (sm.buf[j] == x && j < i);
    if (rank < k) out[rank] = x;
  }
  __syncthreads();
  if (tid == 0) sm.which ^= 1;
  __syncthreads();
}

// (loads that stay behind the wait on the kernel before, whose output the
// logits may be)
__device__ __forceinline__ uint4 load_word(const void* p) { return __ldcs(static_cast<const uint4*>(p)); }
__device__ __forceinline__ void unpack(uint4 w, float (&x)[4]) {
  x[0] = __uint_as_float(w.x);
  x[1] = __uint_as_float(w.y);
  x[2] = __uint_as_float(w.z);
  x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void unpack(uint4 w, float (&x)[8]) {
  const float2 a = bf16x2_to_f32x2(w.x), b = bf16x2_to_f32x2(w.y), c = bf16x2_to_f32x2(w.z), d = bf16x2_to_f32x2(w.w);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y; x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
}
__device__ __forceinline__ uint32_t bits_of(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }
// the larger of two, a NaN if one is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float load1(const float* p) { return __ldcg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(__ldcg(p)); }

// CTA (row, part): part c of C covers the 16-byte words [W c / C, W (c+1) / C)
// of the row's W aligned words (the first and last may belong to it in part).
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_score(const T* logits, int64_t ld, int vocab, const int32_t* targets, int k, int parts,
            float* logprob, float* entropy, int32_t* top_ids, float* top_logprobs, uint32_t* err, uint32_t* tickets,
            score::Part* part) {
  constexpr int kE = 16 / sizeof(T);  // elements of a 16-byte word
  constexpr int kPer = kVecs * 4;     // elements of a thread's tile: 16 either way
  constexpr int kWords = kPer / kE;   // 16-byte words of it
  __shared__ Smem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / parts, c = blockIdx.x % parts;
  if (tid < kMaxK) sm.best[0][tid] = 0;
  if (tid == 0) {
    sm.which = 0;
    sm.last = 0;
  }
  pdl_wait();
  pdl_trigger();
  const T* x = logits + row * ld;
  const int shift = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));  // elements before the row in its first word
  const T* base = x - shift;
  const int64_t words = ((int64_t)shift + vocab + kE - 1) / kE;
  const int64_t w0 = words * c / parts, w1 = words * (c + 1) / parts;
  Stat st = {-INFINITY, 0.f, 0.f, 0};
  __syncthreads();
  float least = -INFINITY;  // value of the k-th best so far: nothing below it is an alternative
  // the words of a tile; an edge of the row, or what lies behind the part, as
  // the bits of -inf
  auto fetch = [&](int64_t t, uint4 (&w)[kWords]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int64_t at = t + tid + (int64_t)i * kThreads;
      const int64_t e0 = at * kE - shift;  // index of the word's first element
      if (at < w1 && e0 >= 0 && e0 + kE <= vocab) {
        w[i] = load_word(base + at * kE);
      } else {
        constexpr uint32_t kNone = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
        uint32_t b[4] = {kNone, kNone, kNone, kNone};
        if (at < w1) {
#pragma unroll
          for (int j = 0; j < kE; ++j)
            if (e0 + j >= 0 && e0 + j < vocab) {
              const uint32_t v = bits_of(__ldcg(x + e0 + j));
              if (sizeof(T) == 4)
                b[j % 4] = v;
              else
                b[j / 2 % 4] = (j & 1) ? (b[j / 2 % 4] & 0xFFFFu) | (v << 16) : (b[j / 2 % 4] & 0xFFFF0000u) | v;
            }
        }
        w[i] = make_uint4(b[0], b[1], b[2], b[3]);
      }
    }
  };
  uint4 word[kWords];
  if (w0 < w1) fetch(w0, word);
  for (int64_t t = w0; t < w1; t += kThreads * kWords) {
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      float y[kE];
      unpack(word[i], y);
#pragma unroll
      for (int j = 0; j < kE; ++j) v[i * kE + j] = y[j];
    }
    // the next tile's loads run while this one is folded in
    if (t + kThreads * kWords < w1) fetch(t + kThreads * kWords, word);
    float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int i = 4; i < kPer; ++i) mx[i & 3] = max_nan(mx[i & 3], v[i]);
    const float tm = max_nan(max_nan(mx[0], mx[1]), max_nan(mx[2], mx[3]));
    st.bad |= !(tm < INFINITY);
    if (tm > st.m) {
      const float d = st.m == -INFINITY ? 0.f : st.m - tm, e = expf(d);
      st.u = e > 0.f ? (st.u + d * st.z) * e : 0.f;
      st.z *= e;
      st.m = tm;
    }
    const float ref = st.m == -INFINITY ? 0.f : st.m;
    float2 z = make_float2(0.f, 0.f), u = z;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      // e^-200 is 0 in fp32: what lies lower (-inf, a mask's value) adds the same nothing
      const float2 d = make_float2(fmaxf(v[i] - ref, -200.f), fmaxf(v[i + 1] - ref, -200.f));
      const float2 e = make_float2(ex2(d.x * 1.4426950408889634f), ex2(d.y * 1.4426950408889634f));
      z.x += e.x;
      z.y += e.y;
      u = ffma2(d, e, u);
    }
    st.z += z.x + z.y;
    st.u += u.x + u.y;
    // (a NaN among them hides the others: then all of the tile is looked at)
    if (k > 0 && __syncthreads_or(!(tm < least))) {
      Key key[kPer];
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int64_t at = t + tid + (int64_t)i * kThreads;
        const int64_t e0 = at * kE - shift;
#pragma unroll
        for (int j = 0; j < kE; ++j) {
          const int64_t e = e0 + j;
          key[i * kE + j] = at < w1 && e >= 0 && e < vocab ? make_key(v[i * kE + j], (uint32_t)e) : 0;
        }
      }
      fold_top(sm, key, k);
      const Key last = sm.best[sm.which][k - 1];
      least = last == 0 ? -INFINITY : key_value(last);
      if (!(least == least)) least = -INFINITY;  // a NaN is below everything
    }
  }
  st = warp_join(st);
  if (lane == 0) sm.stat[warp] = st;
  __syncthreads();
  st = sm.stat[0];
  for (int w = 1; w < kThreads / 32; ++w) st = join(st, sm.stat[w]);
  if (parts > 1) {
    score::Part* mine = part + (int64_t)row * parts + c;
    if (tid == 0) {
      mine->m = st.m;
      mine->z = st.z;
      mine->u = st.u;
      mine->bad = st.bad;
    }
    if (tid < k) mine->key[tid] = sm.best[sm.which][tid];
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      sm.last = atomicAdd(&tickets[row], 1u) == (uint32_t)(parts - 1);
      if (sm.last) tickets[row] = 0;
    }
    __syncthreads();
    if (!sm.last) return;
    __threadfence();
    const score::Part* all = part + (int64_t)row * parts;
    st = Stat{-INFINITY, 0.f, 0.f, 0};
    for (int q = 0; q < parts; ++q) {
      Stat s;
      s.m = __ldcg(&all[q].m);
      s.z = __ldcg(&all[q].z);
      s.u = __ldcg(&all[q].u);
      s.bad = __ldcg(&all[q].bad);
      st = join(st, s);
    }
    if (k > 0) {
      if (tid < kMaxK) sm.best[sm.which][tid] = 0;
      __syncthreads();
      constexpr int kN = score::kMaxParts * kMaxK / kThreads;
      Key key[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int e = tid + i * kThreads;
        key[i] = e < parts * k ? __ldcg(&all[e / k].key[e % k]) : 0;
      }
      fold_top(sm, key, k);
    }
  }
  const float lz = logf(st.z);
  const bool none = st.bad != 0 || st.m == -INFINITY;
  const float nan = __uint_as_float(0x7FC00000u);
  if (tid == 0) {
    const int32_t tg = __ldcg(targets + row);
    float lp = 0.f;
    if (tg != -1) {
      const bool in = tg >= 0 && tg < vocab;
      if (!in) atomicOr(err, kErrIndex);
      lp = in && !none ? load1(x + tg) - st.m - lz : nan;
    }
    logprob[row] = lp;
    entropy[row] = none ? nan : lz - st.u / st.z;
  }
  if (tid < k) {
    const Key key = sm.best[sm.which][tid];
    top_ids[(int64_t)row * k + tid] = key_index(key);
    top_logprobs[(int64_t)row * k + tid] = none ? nan : key_value(key) - st.m - lz;
  }
}

}  // namespace

cudaError_t launch_score(const void* logits, int64_t ld, int dtype, int n_rows, int vocab, const int32_t* targets, int k,
                         float* logprob, float* entropy, int32_t* top_ids, float* top_logprobs, void* workspace,
                         cudaStream_t st) {
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  uint32_t* err = reinterpret_cast<uint32_t*>(ws);
  uint32_t* tickets = reinterpret_cast<uint32_t*>(ws + score::kTickets);
  score::Part* part = reinterpret_cast<score::Part*>(ws + score::kParts);
  const int parts = score::parts_for(n_rows, vocab, device_sm_count());
  const dim3 grid((unsigned)n_rows * (unsigned)parts);
  if (dtype == SPARK_BF16)
    return launch_pdl(k_score<__nv_bfloat16>, grid, dim3(kThreads), 0, st, static_cast<const __nv_bfloat16*>(logits), ld,
                      vocab, targets, k, parts, logprob, entropy, top_ids, top_logprobs, err, tickets, part);
  return launch_pdl(k_score<float>, grid, dim3(kThreads), 0, st, static_cast<const float*>(logits), ld, vocab, targets,
                    k, parts, logprob, entropy, top_ids, top_logprobs, err, tickets, part);
}

}  // namespace spark
