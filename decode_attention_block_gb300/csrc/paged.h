// paged.h -- index arithmetic of the paged cache, shared by host and device
// (no CUDA types, so the host tests compile it alone): the sequences of a
// call as the kernels read them, and the list of attention work they make.
//
// Attention work is a flat list of units.  A group is up to `gt` consecutive
// new tokens of one sequence with one KV head; it reads the cache rows of the
// union of its tokens' windows in tiles of `tile` positions aligned to
// multiples of `tile`, and each (group, tile) is one unit.  A group costs more
// than its tiles (its queries, its output): `lead` units before its first tile
// stand for that.  The list is ordered by sequence, KV head, group, tile.  The
// CTAs of a launch take equal contiguous shares of it: CTA c of G the units
// [total c / G, total (c+1) / G); one whose share ends in a group's lead
// leaves the group to the next.
#pragma once

#include <math.h>
#include <stdint.h>

#if defined(__CUDACC__)
#define SPARK_HD __host__ __device__ inline
#else
#define SPARK_HD inline
#endif

namespace spark {
namespace paged {

// One sequence of a call: its first row of q, its new tokens, the position of
// the first of them.  n == 0 where it brings none, or where its entries make
// no sense (bad).
struct Seq {
  int32_t q0;
  int32_t n;
  int32_t p0;
  bool bad;
};

// q0, q1: q_start[s], q_start[s + 1]; len: seq_len[s].  rows: positions the
// table has room for (max_pages * page_size).
SPARK_HD Seq seq_of(int32_t q0, int32_t q1, int32_t len, int32_t n_tokens, int32_t max_q, int64_t rows) {
  Seq s;
  s.q0 = q0;
  s.n = 0;
  s.p0 = 0;
  s.bad = q0 < 0 || q1 < q0 || q1 > n_tokens;
  if (s.bad || q1 == q0) return s;
  const int32_t n = q1 - q0;
  if (n > max_q || len < n || (int64_t)len > rows) {
    s.bad = true;
    return s;
  }
  s.n = n;
  s.p0 = len - n;
  return s;
}

// sum over i < n of floor((a + step i) / tile), a >= 0, tile a multiple of
// step: floor((a + step i) / tile) = floor((floor(a / step) + i) / (tile / step)).
SPARK_HD int64_t floor_sum(int64_t a, int64_t n, int32_t step, int32_t tile) {
  const int64_t m = tile / step, b = a / step;
  const int64_t q1 = (b + n) / m, r1 = (b + n) % m, q0 = b / m, r0 = b % m;
  return m * (q1 * (q1 - 1) / 2) + r1 * q1 - (m * (q0 * (q0 - 1) / 2) + r0 * q0);
}

struct Shape {
  int32_t gt;      // tokens of a group
  int32_t tile;    // positions of a tile (a multiple of gt)
  int32_t window;  // 0: the whole history
  int32_t lead = 0;  // units before a group's tiles
};

SPARK_HD int32_t groups_of(const Seq& s, const Shape& sh) { return (s.n + sh.gt - 1) / sh.gt; }

// Group i of a sequence: its tokens, the positions it reads [lo, hi] and its
// tiles [tile0, tile1).
struct Group {
  int32_t tok, n_tok;
  int32_t lo, hi;
  int32_t tile0, tile1;
};

SPARK_HD Group group_of(const Seq& s, const Shape& sh, int32_t i) {
  Group g;
  g.tok = i * sh.gt;
  g.n_tok = s.n - g.tok < sh.gt ? s.n - g.tok : sh.gt;
  const int32_t first = s.p0 + g.tok;
  g.hi = first + g.n_tok - 1;
  g.lo = sh.window > 0 && first + 1 > sh.window ? first + 1 - sh.window : 0;
  g.tile0 = g.lo / sh.tile;
  g.tile1 = g.hi / sh.tile + 1;
  return g;
}

// units of the first x groups of a sequence, one KV head, their leads included
SPARK_HD int64_t units_before(const Seq& s, const Shape& sh, int32_t x) {
  if (x <= 0) return 0;
  const int32_t groups = groups_of(s, sh);
  const int32_t whole = x < groups ? x : groups - 1;  // groups of exactly gt tokens among them
  int64_t u = floor_sum((int64_t)s.p0 + sh.gt - 1, whole, sh.gt, sh.tile) + whole + (int64_t)sh.lead * x;
  if (x == groups) u += (int64_t)(s.p0 + s.n - 1) / sh.tile + 1;
  if (sh.window > 0) {
    const int64_t c = (int64_t)s.p0 + 1 - sh.window;
    const int64_t i0 = c >= 0 ? 0 : (-c + sh.gt - 1) / sh.gt;  // groups before it start at position 0
    if (i0 < x) u -= floor_sum(c + sh.gt * i0, x - i0, sh.gt, sh.tile);
  }
  return u;
}

SPARK_HD int64_t units_of(const Seq& s, const Shape& sh) { return units_before(s, sh, groups_of(s, sh)); }

// the group that holds unit u of a sequence's units (one KV head)
SPARK_HD int32_t group_at(const Seq& s, const Shape& sh, int64_t u) {
  int32_t lo = 0, hi = groups_of(s, sh) - 1;
  while (lo < hi) {
    const int32_t mid = lo + (hi - lo + 1) / 2;
    if (units_before(s, sh, mid) <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// a / b for 0 <= a, 0 < b, by 32-bit division where both fit (a 64-bit one is
// some hundred instructions on the GPU)
SPARK_HD int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 31) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// CTAs that share `total` units of `groups` groups (0 < groups <= total) out of
// at most `most`.  A part has at least `least` units, and a group of U units at
// most sqrt(spread U) parts: more would cost more to merge than they save.
// Where these parts of all groups fit `most`, the CTAs are a whole number a
// group, so that where groups are alike no CTA meets two of them.  Where they
// do not, all of `most` share the units and borders fall inside groups: 256
// groups of 33 units (64 sequences, 4 KV heads, a window of 512) on 304 CTAs
// are all cut and merged.
SPARK_HD int32_t ctas_for(int64_t total, int64_t groups, int32_t least, float spread, int32_t most) {
  if (groups >= most) return most;
  const int64_t units = quotient(total, groups);
  int64_t parts = quotient(units, least);
  const int64_t cap = (int64_t)sqrtf(spread * (float)units);
  if (parts > cap) parts = cap;
  if (parts < 1) parts = 1;
  return groups * parts > most ? most : (int32_t)(groups * parts);
}

SPARK_HD int64_t share_begin(int64_t total, int32_t G, int32_t c) { return quotient(total * c, G); }

// the CTA that holds unit u of `total`, for G CTAs
SPARK_HD int32_t cta_at(int64_t u, int64_t total, int32_t G) {
  const int64_t c = quotient((u + 1) * G - 1, total);
  return (int32_t)(c < G - 1 ? c : G - 1);
}

// Slot of CTA c's partial state of a group that begins at unit `begin`: a
// share meets at most two groups in part, its first (slot 2c) and its last
// (2c + 1); a group that begins inside the share, behind its start, is the last.
SPARK_HD int32_t partial_slot(int32_t c, int64_t begin, int64_t total, int32_t G) {
  return 2 * c + (begin > share_begin(total, G, c) ? 1 : 0);
}

// Where position `pos` lives: the table's column and the row of the page.
// The column by a product: with n = pos / 16 < 2^26, d = page_size / 16 <= 64
// and m = floor(2^32 / d) + 1 the error n (m d - 2^32) / (2^32 d) of n m / 2^32
// is below n / 2^32 < 1 / d, so floor(n m / 2^32) = floor(n / d).
SPARK_HD uint64_t page_mul(int32_t page_size) { return ((uint64_t)1 << 32) / (uint64_t)(page_size / 16) + 1; }
SPARK_HD int32_t page_col(int32_t pos, uint64_t mul) { return (int32_t)(((uint64_t)(pos >> 4) * mul) >> 32); }
SPARK_HD int32_t page_row(int32_t pos, int32_t col, int32_t page_size) { return pos - col * page_size; }

}  // namespace paged
}  // namespace spark
