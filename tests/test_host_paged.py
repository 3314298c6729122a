"""Host checks of the paged cache and the token scores (no GPU).

* The index arithmetic of ``csrc/paged.h``, compiled with the host C++
  compiler: the closed sums of the work list against loops, the groups and
  tiles of every unit, shares that tile the list, partial slots that no two
  groups share, sequences whose entries make no sense.
* The refusals of the entry points of ``include/spark_paged.h`` and
  ``include/spark_score.h``: every status is decided before anything touches
  a device.
"""

import ctypes
import os
import shutil
import subprocess

import pytest

from decode_attention_block_gb300 import build_lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "decode_attention_block_gb300", "csrc")

PROGRAM = r"""
#include <cstdint>
#include <cstdio>
#include <map>
#include <random>
#include <set>
#include <utility>
#include <vector>
#include "paged.h"
using namespace spark::paged;

static int fails = 0;
#define CHECK(c, ...) do { if (!(c)) { std::printf(__VA_ARGS__); std::printf("\n"); if (++fails > 20) return 1; } } while (0)

int main() {
  // the closed sum
  for (int step : {1, 4, 32})
    for (int tile : {step, 4 * step, 16 * step})
      for (int64_t a = 0; a < 3 * tile; a += step > 1 ? 3 : 1) {
        int64_t sum = 0;
        for (int n = 0; n < 40; ++n) {
          CHECK(floor_sum(a, n, step, tile) == sum, "floor_sum(%ld, %d, %d, %d)", (long)a, n, step, tile);
          sum += (a + (int64_t)step * n) / tile;
        }
      }
  // sequences
  struct { int q0, q1, len, n, p0; bool bad; } seqs[] = {
    {0, 3, 10, 3, 7, false}, {5, 5, 9, 0, 0, false}, {5, 5, -9, 0, 0, false}, {2, 1, 9, 0, 0, true},
    {-1, 1, 9, 0, 0, true}, {0, 101, 200, 0, 0, true}, {0, 9, 200, 0, 0, true}, {0, 3, 2, 0, 0, true},
    {0, 3, -2, 0, 0, true}, {0, 3, 257, 0, 0, true}, {0, 3, 256, 3, 253, false}, {97, 100, 3, 3, 0, false},
    {INT32_MIN, INT32_MAX, 1, 0, 0, true}, {INT32_MAX, INT32_MIN, 1, 0, 0, true}, {0, 1, INT32_MAX, 0, 0, true}};
  for (auto& t : seqs) {
    const Seq s = seq_of(t.q0, t.q1, t.len, 100, 8, 256);
    CHECK(s.n == t.n && s.p0 == t.p0 && s.bad == t.bad, "seq_of(%d, %d, %d)", t.q0, t.q1, t.len);
  }
  // groups and their tiles, at the edges of tiles and windows
  std::mt19937 rng(1);
  const Shape shapes[] = {{1, 16, 0}, {1, 16, 1}, {1, 16, 5}, {1, 16, 512}, {32, 128, 0}, {32, 128, 7}, {32, 128, 512},
                          {32, 128, INT32_MAX}, {64, 128, 0}, {64, 128, 100}, {32, 128, 0, 3}, {64, 128, 100, 1}};
  for (const Shape& sh : shapes)
    for (int it = 0; it < 400; ++it) {
      Seq s{0, 1 + (int)(rng() % 200), (int)(rng() % 1500), false};
      int64_t u = 0;
      for (int i = 0; i < groups_of(s, sh); ++i) {
        const Group g = group_of(s, sh, i);
        CHECK(units_before(s, sh, i) == u, "units_before gt %d n %d p0 %d group %d", sh.gt, s.n, s.p0, i);
        int lo = INT32_MAX, hi = -1;
        for (int t = g.tok; t < g.tok + g.n_tok; ++t) {
          const int p = s.p0 + t, first = sh.window > 0 && p + 1 > sh.window ? p + 1 - sh.window : 0;
          if (first < lo) lo = first;
          if (p > hi) hi = p;
        }
        CHECK(g.lo == lo && g.hi == hi && g.tok == i * sh.gt && g.tok + g.n_tok <= s.n, "group %d", i);
        CHECK(g.tile0 == lo / sh.tile && g.tile1 == hi / sh.tile + 1, "tiles of group %d", i);
        for (int k = g.tile0 - sh.lead; k < g.tile1; ++k, ++u) CHECK(group_at(s, sh, u) == i, "group_at");
      }
      CHECK(units_of(s, sh) == u, "units_of");
    }
  // the longest: 2^17 tokens at the end of 2^30 positions
  const Seq big{0, 1 << 17, (1 << 30) - (1 << 17), false};
  CHECK(units_of(big, Shape{1, 16, 0}) > 0 && units_of(big, Shape{1, 16, 0}) < ((int64_t)1 << 44), "units of the longest");
  // shares, tickets and partial slots
  for (int it = 0; it < 300; ++it) {
    std::vector<int64_t> begin{0};
    const int groups = 1 + rng() % 30, lead = it % 4;
    for (int i = 0; i < groups; ++i) begin.push_back(begin.back() + lead + 1 + rng() % (it % 3 ? 9 : 300));
    const int64_t total = begin.back();
    const int least = 1 + rng() % 6, most = 1 + rng() % 40;
    const float spread = 0.5f + rng() % 8;
    const int G = ctas_for(total, groups, least, spread, most);
    CHECK(G >= 1 && G <= total && G <= most, "ctas_for");
    // groups alike, as many CTAs as they want: a whole number each
    const int units = 1 + rng() % 900, H = ctas_for((int64_t)units * groups, groups, least, spread, 1 << 20);
    CHECK(H % groups == 0 && (H == groups || (H / groups * least <= units && (float)(H / groups) * (H / groups) <= spread * units)),
          "parts of groups alike");
    for (int i = 0; i <= groups; ++i)
      CHECK(share_begin((int64_t)units * groups, H, i * (H / groups)) == (int64_t)i * units, "shares of groups alike");
    std::set<int> slots, tickets;
    for (int i = 0; i < groups; ++i) {
      const int64_t b = begin[i] + lead, e = begin[i + 1];
      const int c0 = cta_at(b, total, G), c1 = cta_at(e - 1, total, G);
      for (int c = 0; c < G; ++c) {
        const int64_t u0 = share_begin(total, G, c), u1 = share_begin(total, G, c + 1);
        const bool meets = u0 < e && b < u1;
        CHECK(meets == (c >= c0 && c <= c1), "CTA %d of %d and group [%ld, %ld) of %ld", c, G, (long)b, (long)e, (long)total);
        if (meets && c0 != c1) {
          const int slot = partial_slot(c, b, total, G);
          CHECK(slot / 2 == c && slots.insert(slot).second, "slot %d of CTA %d twice", slot, c);
        }
      }
      if (c0 != c1) CHECK(tickets.insert(c0).second, "ticket %d twice", c0);
    }
    CHECK(share_begin(total, G, 0) == 0 && share_begin(total, G, G) == total, "shares");
  }
  for (int ps = 16; ps <= 1024; ps += 16) {
    const uint64_t m = page_mul(ps);
    for (int i = 0; i < 30000; ++i) {
      const int x = i < 5000 ? i : i < 10000 ? (1 << 30) - 1 - (i - 5000) : (int)(rng() >> 2);
      const int c = page_col(x, m), r = page_row(x, c, ps);
      CHECK(c == x / ps && r == x % ps, "page of %d at %d", x, ps);
    }
  }
  std::printf("%d failures\n", fails);
  return fails != 0;
}
"""


def test_index_arithmetic(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    src = tmp_path / "paged.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "paged"
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I", CSRC,
                    str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout[-3000:] + res.stderr[-2000:]


# -- refusals ------------------------------------------------------------------

FAKE = 1 << 40          # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def B():
    build_lib.build()
    from decode_attention_block_gb300 import binding
    binding.load()
    return binding


def _pool(B, **kw):
    f = dict(k=FAKE, v=FAKE, n_pages=100, page_size=64, dtype=B.SPARK_BF16)
    f.update(kw)
    return B.SparkPagePool(f["k"], f["v"], f["n_pages"], f["page_size"], f["dtype"])


def _batch(B, **kw):
    f = dict(table=FAKE, q_start=FAKE, seq_len=FAKE, n_seqs=4, max_pages=20, n_tokens=9, max_q_len=5)
    f.update(kw)
    return B.SparkPagedBatch(*f.values())


def _attention(B, geom=None, q=FAKE, ld=4096, dtype=1, pool=None, cls=1, batch=None, a=FAKE + (1 << 30), ws=FAKE, nbytes=None):
    lib = B.load()
    g = geom or B.spark_geom_default()
    nbytes = B.spark_paged_workspace_bytes(B.spark_geom_default()) if nbytes is None else nbytes
    return lib.spark_paged_attention(ctypes.byref(g), q, ld, dtype, ctypes.byref(pool or _pool(B)), cls,
                                     ctypes.byref(batch or _batch(B)), a, ws, nbytes, None)


def _append(B, k=FAKE, v=FAKE, ld=1024, dtype=0, pool=None, batch=None, ws=FAKE, nbytes=None):
    lib = B.load()
    g = B.spark_geom_default()
    nbytes = B.spark_paged_workspace_bytes(g) if nbytes is None else nbytes
    return lib.spark_paged_append(ctypes.byref(g), k, v, ld, dtype, ctypes.byref(pool or _pool(B)),
                                  ctypes.byref(batch or _batch(B)), ws, nbytes, None)


BAD_POOLS = [(dict(k=0), -1), (dict(v=FAKE + 8), -1), (dict(dtype=3), -1), (dict(n_pages=0), -1), (dict(page_size=0), -1),
             (dict(page_size=8), -5), (dict(page_size=24), -5), (dict(page_size=1040), -5),
             (dict(n_pages=(1 << 24) + 1, page_size=16), -5), (dict(n_pages=1 << 21, page_size=1024), -5)]
BAD_BATCHES = [(dict(table=0), -1), (dict(q_start=FAKE + 2), -1), (dict(seq_len=0), -1), (dict(n_seqs=0), -1),
               (dict(n_seqs=1025), -1), (dict(max_pages=0), -1), (dict(max_pages=(1 << 20) + 1), -5),
               (dict(n_tokens=0), -1), (dict(n_tokens=(1 << 17) + 1), -5), (dict(max_q_len=0), -1),
               (dict(max_q_len=10), -1)]


def test_pools_and_batches_are_validated(B):
    for kw, want in BAD_POOLS:
        assert _attention(B, pool=_pool(B, **kw)) == want, kw
        assert _append(B, pool=_pool(B, **kw)) == want, kw
    for kw, want in BAD_BATCHES:
        assert _attention(B, batch=_batch(B, **kw)) == want, kw
        assert _append(B, batch=_batch(B, **kw)) == want, kw


def test_attention_arguments_are_validated(B):
    assert _attention(B, q=0) == -1 and _attention(B, q=FAKE + 8) == -1
    assert _attention(B, a=0) == -1 and _attention(B, a=FAKE + 4) == -1
    rows = 9 * 4096 * 2                                                     # q and a do not overlap
    assert _attention(B, a=FAKE) == -1 and _attention(B, a=FAKE + rows - 16) == -1 and _attention(B, a=FAKE - rows + 16) == -1
    assert _attention(B, a=FAKE + rows, ws=0) == -4 and _attention(B, a=FAKE - rows, ws=0) == -4
    assert _attention(B, ld=4095) == -1 and _attention(B, ld=4100) == -1    # rows not 16-byte aligned
    assert _attention(B, ld=4098, dtype=0) == -1 and _attention(B, ld=4088) == -1
    assert _attention(B, dtype=2) == -1 and _attention(B, cls=2) == -1
    need = B.spark_paged_workspace_bytes(B.spark_geom_default())
    assert _attention(B, nbytes=need - 1) == -4 and _attention(B, ws=0) == -4 and _attention(B, ws=FAKE + 16) == -4
    g = B.spark_geom_default()
    g.head_dim = 128
    assert _attention(B, geom=g) == -5 and B.spark_paged_workspace_bytes(g) == 0


def test_append_arguments_are_validated(B):
    assert _append(B, k=0) == -1 and _append(B, v=FAKE + 4) == -1 and _append(B, dtype=-1) == -1
    assert _append(B, ld=1020) == -1 and _append(B, ld=1026) == -1
    assert _append(B, ld=1028, dtype=1) == -1
    assert _append(B, ws=0) == -4 and _append(B, nbytes=100) == -4


def test_block_arguments_are_validated(B):
    lib = B.load()
    g = B.spark_geom_default()
    w = B.SparkLayerWeights(FAKE, FAKE, FAKE, FAKE, B.SPARK_BF16)

    def call(pos=(1, 2, 3), batch=None, pool=None, cls=0, h=FAKE, ws=FAKE, nbytes=None, pws=FAKE, pbytes=None):
        b = batch or _batch(B, n_tokens=len(pos), max_q_len=1)
        nbytes = B.spark_attn_workspace_bytes(g, 3) if nbytes is None else nbytes
        pbytes = B.spark_paged_workspace_bytes(g) if pbytes is None else pbytes
        return lib.spark_attn_paged(ctypes.byref(g), h, ctypes.byref(w), ctypes.byref(pool or _pool(B)), cls,
                                    ctypes.byref(b), (ctypes.c_int32 * len(pos))(*pos), FAKE, ws, nbytes, pws, pbytes,
                                    None)
    assert call(pos=(1, -1, 3)) == -2 and call(pos=(1, 2**31 - 1, 3)) == -2
    assert call(batch=_batch(B, n_tokens=1025)) == -1
    assert call(h=0) == -1 and call(cls=7) == -1
    assert call(pool=_pool(B, page_size=20)) == -5
    assert call(nbytes=1000) == -4 and call(ws=0) == -4 and call(pws=0) == -4 and call(pbytes=1000) == -4


def _pages(B, compact, pools=None, table=FAKE, new=FAKE + (1 << 20), slots=8, width=16, ws=FAKE, nbytes=None, lists=FAKE):
    lib = B.load()
    g = B.spark_geom_default()
    pools = pools or [_pool(B), _pool(B)]
    arr = (B.SparkPagePool * max(1, len(pools)))(*pools)
    nbytes = B.spark_pages_workspace_bytes(100, 8) if nbytes is None else nbytes
    if compact:
        return lib.spark_pages_compact(ctypes.byref(g), arr, len(pools), table, slots, width, new, lists, ws, nbytes, None)
    return lib.spark_pages_remap(ctypes.byref(g), arr, len(pools), table, slots, width, lists, lists, lists, new, ws,
                                 nbytes, None)


@pytest.mark.parametrize("compact", [False, True])
def test_page_table_arguments_are_validated(B, compact):
    for kw, want in BAD_POOLS:
        assert _pages(B, compact, pools=[_pool(B), _pool(B, **kw)]) == want, kw
    assert _pages(B, compact, pools=[_pool(B), _pool(B, n_pages=99)]) == -1        # pools that differ
    assert _pages(B, compact, pools=[_pool(B), _pool(B, dtype=0)]) == -1
    assert _pages(B, compact, pools=[_pool(B)] * 129) == -5
    assert _pages(B, compact, slots=0) == -1 and _pages(B, compact, slots=1025) == -1
    assert _pages(B, compact, width=0) == -1 and _pages(B, compact, width=(1 << 20) + 1) == -5
    assert _pages(B, compact, slots=1024, width=(1 << 16) + 1) == -5
    assert _pages(B, compact, table=0) == -1 and _pages(B, compact, new=0) == -1 and _pages(B, compact, lists=0) == -1
    assert _pages(B, compact, new=FAKE + 16) == -1                                  # overlapping tables
    assert _pages(B, compact, ws=0) == -4 and _pages(B, compact, nbytes=511) == -4
    if not compact:
        assert _pages(B, compact, new=FAKE) == -1                                   # remap is not in place
    assert B.spark_pages_workspace_bytes(0, 8) == 0 and B.spark_pages_workspace_bytes(8, 0) == 0
    assert B.spark_pages_workspace_bytes((1 << 24) + 1, 8) == 0 and B.spark_pages_workspace_bytes(8, 1025) == 0
    assert B.spark_pages_workspace_bytes(1 << 24, 1024) > B.spark_pages_workspace_bytes(1, 1) > 0


def test_logprobs_arguments_are_validated(B):
    lib = B.load()
    need = B.spark_logprobs_workspace_bytes(4, 5)

    def call(x=FAKE, ld=1000, dtype=0, n=4, vocab=1000, t=FAKE, k=5, lp=FAKE, h=FAKE, ids=FAKE, tl=FAKE, ws=FAKE,
             nbytes=need):
        return lib.spark_token_logprobs(x, ld, dtype, n, vocab, t, k, lp, h, ids, tl, ws, nbytes, None)
    for kw in (dict(x=0), dict(x=FAKE + 2), dict(ld=999), dict(dtype=2), dict(n=0), dict(n=(1 << 20) + 1), dict(vocab=0),
               dict(vocab=(1 << 24) + 1, ld=1 << 25), dict(t=0), dict(t=FAKE + 2), dict(k=-1), dict(k=33),
               dict(vocab=4, k=5), dict(lp=0), dict(h=0), dict(ids=0), dict(tl=0)):
        assert call(**kw) == -1, kw
    assert call(ws=0) == -4 and call(ws=FAKE + 64) == -4 and call(nbytes=need - 1) == -4
    for n, k in ((0, 1), (1, -1), (1, 33), ((1 << 20) + 1, 1)):
        assert B.spark_logprobs_workspace_bytes(n, k) == 0
