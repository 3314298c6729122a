"""Attention over 4-bit pages where many probabilities are far below the row's
largest: a dominant key at the first position, all others 10 to 18 nats below.

The kernels hold probabilities as fp16 numbers of which the row's largest lies
between 2^11 and 2^15: half of fp16's smallest step is 2^-36 of it, and none of
the bounds here grows otherwise with the length.  Per element, with p relative to
the dominant key's (its score is exact here: one product of few bits):
* a position's score is off by ds <= scale (sum |q k| (2^-22 + 2^-15) + 2^-25 M
  sum |k|), M the largest query (the dominant dim's product is 0 there); its p,
  to base 2 in fp32 (scores up to 2^5: 2 * 2^5 * 2^-24 ln 2 < 2^-18) with the
  exponential (2^-21), by 1.01 ds + 2^-17 of itself, in numerator and sum.
* in the numerator p is rounded: 2^-22 of itself as two halves, 2^-11 as one (bf16
  queries of chunks), and 2^-36.
* the sum of the probabilities, rounded to nearest: of a token's fp32 queries at most
  64 additions between two folds into a sum in memory and 32 folds, of a chunk's 64
  within a tile, 4 of tiles, and folds with what they leave: 2^-16.  Of bf16 queries
  up to 2048 additions in a row: 2^-13.
* the output's sums: a matrix instruction cuts off, of each product, what lies 2^-25
  below its sum, and of the sum 2^-23 once in 16 positions: 1.25 * 2^-25 a position,
  twice where a product is of two halves (fp32 queries of chunks).  Sums begin anew
  after 1024 positions of a warp (bf16 queries 2048), 384 or 512 of a chunk (8192), and
  are added up in fp32, rounded to nearest (at most 342 times, of values that
  differ: 2^-19).  And the
  output's own rounding.
"""

import pytest
import torch

import fp4_ref
from test_gpu_paged import B, BF16, D, F32, _geom, _i32  # noqa: F401

pytestmark = pytest.mark.gpu
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
SCALE = 0.0625


def _pool(rows, entries, page):
    code, sc = fp4_ref.quantize(rows)
    pool = torch.full((len(entries), page // 16, 1, fp4_ref.BLOCK), 0xFF, dtype=torch.uint8, device="cuda")
    fp4_ref.write(pool, entries, page, torch.arange(len(rows), device="cuda"), code, sc)
    return pool, fp4_ref.values(code, sc)[:, 0]


# single tokens, chunks on single CTAs, on pairs: enough sequences for a share to hold a whole one
@pytest.mark.parametrize("n_seqs, n", [(480, 1), (160, 8), (80, 40)])
@pytest.mark.parametrize("q_type", [F32, BF16])
@pytest.mark.parametrize("c, top, spread, sink", [
    (131072, 46.5, 0.0, 0.0),    # all 17.4 below, the dominant value 0: the output is the tail's alone
    (131072, 45.25, 0.0, 1.0),   # 17 below
    (40000, 40.0, 0.0, 1.0),     # 15
    (40000, 26.5, 0.4, 0.0),     # 10, of keys that differ
    (131072, 48.0, 0.4, 0.0),    # 18
])
def test_a_dominant_key_leaves_the_others_their_weight(B, n_seqs, n, q_type, c, top, spread, sink):
    g, gen, page = _geom(B, 1, 512, SCALE), torch.Generator("cuda").manual_seed(9), 128
    entries = torch.randperm(-(-c // page), generator=gen, device="cuda").int()
    keys = torch.zeros(c, 1, D, device="cuda")
    keys[1:, :, 16:] = 0.25 * torch.randn(c - 1, 1, D - 16, generator=gen, device="cuda") if spread else 0.0
    keys[0, 0, 0] = 6.0
    rows = torch.rand(c, 1, D, generator=gen, device="cuda")
    rows[0] = sink
    (pk, k), (pv, v) = _pool(keys, entries, page), _pool(rows, entries, page)
    assert k[0, 0] == 6.0 and not bool(k[0, 1:].any())
    some = 3  # sequences with queries of their own, all of the same pages
    q3 = spread * torch.randn(some, n, 4, D, generator=gen, device="cuda")
    q3[..., :16] = 0.0
    q3[..., 0] = top
    q3 = q3.to(q_type)
    q = q3[torch.arange(n_seqs, device="cuda") % some].reshape(n_seqs * n, 4 * D)
    batch = B.PagedBatch(entries.repeat(n_seqs, 1).contiguous(), _i32([n * i for i in range(n_seqs + 1)]), _i32([c] * n_seqs), n_seqs * n, n)
    a, ws = torch.zeros(n_seqs * n, 4 * D, device="cuda", dtype=q_type), B.make_paged_workspace(g)
    B.spark_paged_attention(g, q, B.PagePool(pk, pv), B.SPARK_FULL, batch, a, ws)
    torch.cuda.synchronize()
    assert B.spark_attn_error_word(ws) == 0
    qd = q3.double()
    z = SCALE * torch.einsum("sthd,xd->sthx", qd, k)
    assert bool((z.argmax(-1) == 0).all())
    late = torch.arange(c, device="cuda")[None] > torch.arange(c - n, c, device="cuda")[:, None]
    p = (z - z[..., :1]).masked_fill_(late[None, :, None], float("-inf")).exp_()
    total = p.sum(-1, keepdim=True)
    want = p @ v / total
    ds = (SCALE * (2.0 ** -22 + 2.0 ** -15)) * torch.einsum("sthd,xd->sthx", qd.abs(), k.abs())
    ds += (SCALE * 2.0 ** -25) * (qd.abs().amax(-1, keepdim=True) * k.abs().sum(-1))
    ds[..., 0] = 0.0
    off = p * (1.01 * ds + 2.0 ** -17)
    pv_sum = p @ v.abs()
    single = q_type == F32 or n == 1
    bound = off @ v.abs() + off.sum(-1, keepdim=True) * want.abs() + pv_sum * (2.0 ** -22 if single else 2.0 ** -11)
    cut = 2.0 ** -19 + 1.25 * 2.0 ** -25 * ({F32: 1024, BF16: 2048} if n == 1 else {F32: 2 * 512, BF16: 8192})[q_type]
    bound += 2.0 ** -36 * v.abs().sum(0) + cut * pv_sum
    bound = 1.01 * bound / total + (U[q_type] + (2.0 ** -16 if q_type == F32 else 2.0 ** -13)) * want.abs()
    sel = torch.arange(n_seqs, device="cuda") % some
    worst = ((a.double().view(n_seqs, n, 4, D) - want[sel]).abs() / bound[sel]).max().item()
    assert worst <= 1.0, f"error {worst:.2f} of its bound"


@pytest.mark.parametrize("n_seqs, n, log2", [(s, n, x) for s, n in ((480, 1), (160, 8), (80, 40), (3, 1), (3, 40))
                                             for x in (20, 23, 24, 25, 25.6, 26, 26.6, 27, 27.5, 28, 29, 35, 60) if n == 1 or x < 28])
@pytest.mark.parametrize("q_type", [F32, BF16])
def test_large_scores_leave_probabilities_in_range(B, n_seqs, n, log2, q_type):
    """A key whose scores are far above all others', where fp32's steps of a score pass 1 and 16 (chunks: up to 2^28, to
    base 2): its value, whatever a maximum and what is subtracted from it are rounded to.  Its probability over the sum of
    all is 1, and at least 2^-8: two halves off by 2^-25 are off by 2^-17 of it, one by 2^-11."""
    g, gen, page, c = _geom(B, 1, 512, SCALE), torch.Generator("cuda").manual_seed(10), 64, 700
    entries = torch.randperm(-(-c // page), generator=gen, device="cuda").int()
    keys, rows = torch.zeros(c, 1, D, device="cuda"), torch.rand(c, 1, D, generator=gen, device="cuda")
    keys[:, :, 0], keys[300, :, 0], rows[300] = 4.0, 6.0, 1.5
    (pk, _), (pv, v) = _pool(keys, entries, page), _pool(rows, entries, page)
    # fp32 queries: numbers of all 24 bits, so that products are rounded
    top = 2.0 ** log2 / (SCALE * 6.0 * 1.4426950408889634) * (1.0 + 0.25 * torch.rand(n_seqs * n, 4, generator=gen, device="cuda"))
    q = torch.zeros(n_seqs * n, 4, D, device="cuda")
    q[..., 0] = top
    q = q.to(q_type).reshape(n_seqs * n, 4 * D)
    batch = B.PagedBatch(entries.repeat(n_seqs, 1).contiguous(), _i32([n * i for i in range(n_seqs + 1)]), _i32([c] * n_seqs), n_seqs * n, n)
    a, ws = torch.zeros(n_seqs * n, 4 * D, device="cuda", dtype=q_type), B.make_paged_workspace(g)
    B.spark_paged_attention(g, q, B.PagePool(pk, pv), B.SPARK_FULL, batch, a, ws)
    assert B.spark_attn_error_word(ws) == 0
    err = (a.double().view(-1, 4, D) - v[300]).abs()
    assert bool((err <= v[300] * (U[q_type] + (2.0 ** -11 if q_type == BF16 else 2.0 ** -16))).all()), err.max().item()
