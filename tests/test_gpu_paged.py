"""The paged cache's operators against plain implementations in 64 bits.

Attention tolerances are derived per element from the roundings in the path,
with u the relative rounding of a type (bf16 2^-8, fp32 2^-24):

* a score s = scale * sum_d q_d k_d.  fp32 queries on a bf16 pool are carried
  as two bf16 numbers, off by at most 2^-16 relative; every product is exact
  and 256 of them (two halves: 512) are summed in fp32:
  |ds| <= scale * sum |q k| * (e_q + 2^-15), e_q = 2^-16 for fp32 queries, 0
  for bf16 ones.
* a probability e^(s - m): its relative error is at most 2 |ds| (numerator
  and sum), plus 2^-20 for the exponential, the scaling to base 2 of scores
  of up to 2^6 (2^-24 * 2^6 * ln 2 < 2^-18) and the fp32 sums, plus the
  rounding of the probabilities themselves: 2^-16 for two bf16 halves, 2^-8
  for one.
* the output sum p v / sum p: the same relative error on sum p |v|, fp32 sums
  (within 2^-15), and one rounding to the output's type.

The bound takes the largest |ds| of the row.  fp32 pools use fp32 arithmetic
throughout (e_q = 0, probabilities unrounded).
"""

import numpy as np
import pytest
import torch

import oracle
from decode_attention_block_gb300 import build_lib, synth
from helpers import assert_close, np_weights

pytestmark = pytest.mark.gpu

D = 256
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build_lib.build()
    from decode_attention_block_gb300 import binding
    binding.load()
    return binding


def _geom(B, n_kv=4, window=512, scale=0.0625):
    g = B.spark_geom_default()
    g.n_kv, g.n_q, g.window, g.scale = n_kv, 4 * n_kv, window, scale
    return g


def _i32(x, device="cuda"):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=device)


class Case:
    """Sequences of (context, new tokens) on a pool whose rows outside the
    sequences are NaN, with table entries that no call may use."""

    def __init__(self, seqs, n_kv=4, page=16, dtype=BF16, seed=0, pad=0, extra_pages=3, slack_cols=2):
        r = np.random.default_rng(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.seqs, self.n_kv, self.page, self.dtype = list(seqs), n_kv, page, dtype
        self.ctx = [c for c, _ in seqs]
        self.new = [n for _, n in seqs]
        need = [-(-c // page) for c in self.ctx]
        n_pages = sum(need) + extra_pages
        order = r.permutation(n_pages)
        width = max(max(need), 1) + slack_cols
        table = r.choice([-1, -7, n_pages, 2**31 - 1, -2**31], size=(len(seqs), width))
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = order[at:at + n]
            at += n
        self.table_np = table
        self.table = _i32(table)
        shape = (n_pages, page, n_kv, D)
        self.k = torch.full(shape, float("nan"), device="cuda", dtype=dtype)
        self.v = torch.full(shape, float("nan"), device="cuda", dtype=dtype)
        self.rows_k, self.rows_v = [], []
        for s, c in enumerate(self.ctx):
            k = torch.randn(c, n_kv, D, generator=g, device="cuda").to(dtype)
            v = torch.randn(c, n_kv, D, generator=g, device="cuda").to(dtype)
            self.rows_k.append(k)
            self.rows_v.append(v)
        self.n_tokens = sum(self.new) + pad
        self.q_start = _i32(np.concatenate([[0], np.cumsum(self.new)]))
        self.seq_len = _i32(self.ctx)
        self.max_q = max(1, max(self.new))
        self.g = g

    def where(self, s, upto=None):
        """(page, row) index of positions [0, upto) of sequence s."""
        x = np.arange(self.ctx[s] if upto is None else upto)
        return (torch.tensor(self.table_np[s][x // self.page], device="cuda"),
                torch.tensor(x % self.page, device="cuda"))

    def fill(self, window=0):
        """Put the rows that may be attended to into the pool (the others stay NaN)."""
        for s, (c, n) in enumerate(self.seqs):
            lo = 0 if window == 0 or n == 0 else max(0, c - n + 1 - window)
            p, r = self.where(s)
            self.k[p[lo:], r[lo:]] = self.rows_k[s][lo:]
            self.v[p[lo:], r[lo:]] = self.rows_v[s][lo:]
            if lo >= self.page:  # pages wholly before every window are given back
                self.table[s, : lo // self.page] = -1

    def batch(self, B, n_tokens=None, max_q=None):
        return B.PagedBatch(self.table, self.q_start, self.seq_len, n_tokens or self.n_tokens, max_q or self.max_q)


def _reference(case, q, window, scale, q_type, p_round):
    """out, and the bound of its error, in 64 bits: [tokens, n_q, 256]."""
    n_kv = case.n_kv
    out, bound, t = [], [], 0
    e_q = 2.0**-16 if q_type == F32 and case.dtype == BF16 else 0.0
    u_out = 2.0**-8 if q_type == BF16 else 2.0**-24
    for s, (c, n) in enumerate(case.seqs):
        if n == 0:
            continue
        k = case.rows_k[s].double().repeat_interleave(4, 1)  # query head h reads KV head h / 4
        v = case.rows_v[s].double().repeat_interleave(4, 1)
        qs = q[t:t + n].double().view(n, 4 * n_kv, D)
        pos = torch.arange(c - n, c, device="cuda")[:, None]
        x = torch.arange(c, device="cuda")[None]
        seen = x <= pos
        if window:
            seen &= x > pos - window
        sc = scale * torch.einsum("thd,xhd->htx", qs, k)
        ds = scale * torch.einsum("thd,xhd->htx", qs.abs(), k.abs()) * (e_q + 2.0**-15)
        sc = sc.masked_fill(~seen, -np.inf)
        p = torch.softmax(sc, -1)
        o = torch.einsum("htx,xhd->thd", p, v)
        rel = 2 * ds.masked_fill(~seen, 0).amax(-1) + 2.0**-17 + p_round + 2.0**-15  # [heads, tokens]
        pv = torch.einsum("htx,xhd->thd", p, v.abs())
        out.append(o)
        bound.append(pv * rel.T[:, :, None] * 1.01 + u_out * o.abs() + 1e-30)
        t += n
    return torch.cat(out), torch.cat(bound)


def _check_attention(B, case, q_type=F32, full=True, window=512, scale=0.0625, max_q=None, q_pad=0, stream=None):
    g = _geom(B, case.n_kv, window, scale)
    case.fill(0 if full else window)
    width = 4 * case.n_kv * D
    wide = torch.randn(case.n_tokens, width + q_pad, generator=case.g, device="cuda").to(q_type)
    q = wide[:, q_pad:]
    a = torch.full((case.n_tokens, width), 77.0, device="cuda", dtype=q_type)
    ws = B.make_paged_workspace(g)
    B.spark_paged_attention(g, q, B.PagePool(case.k, case.v), B.SPARK_FULL if full else B.SPARK_SLIDING,
                            case.batch(B, max_q=max_q), a, ws)
    torch.cuda.synchronize()
    assert B.spark_attn_error_word(ws) == 0
    used = sum(case.new)
    assert bool((a[used:] == 77.0).all()), "rows behind the last sequence were written"
    p_round = 0.0 if case.dtype == F32 else 2.0**-16 if q_type == F32 else 2.0**-8
    want, bound = _reference(case, q, 0 if full else window, scale, q_type, p_round)
    err = (a[:used].double().view(want.shape) - want).abs()
    assert bool(torch.isfinite(err).all()), "non-finite output"
    worst = (err / bound).max().item()
    assert worst <= 1.0, f"error {worst:.2f} of its bound"
    return a


SHORT = [(1, 1), (15, 1), (16, 1), (17, 1), (33, 1), (128, 1), (129, 1), (700, 1)]
SETS = {
    "one": [(1, 1)],
    "two": [(2, 2)],
    "decode": SHORT,
    "verify": [(5, 5), (16, 3), (40, 0), (100, 7), (131, 6), (700, 2), (0, 0), (515, 4)],
    "chunk": [(150, 150)],
    "chunk_at": [(300, 45), (161, 33), (129, 32)],
    "mixed": [(400, 1), (0, 0), (260, 130), (1, 1), (77, 64), (530, 3), (640, 31)],
    "long": [(5000, 1)],
    "long_chunk": [(2100, 70)],
    "big_chunk": [(1300, 1100), (700, 257)],
    # mostly long: more than half of the longest on average
    "pairs": [(400, 90), (0, 0), (260, 130), (77, 64), (530, 103), (640, 31), (65, 65), (900, 129)],
    "edges": [(64, 64), (65, 65), (128, 33), (129, 32), (200, 63), (256, 128), (31, 31), (33, 33)],
    "far": [(9000, 40)],     # one group over many CTAs
    "far_short": [(9000, 6)],
}


@pytest.mark.parametrize("q_type", [F32, BF16])
@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("name", list(SETS))
def test_attention_bf16_pool(B, name, full, q_type):
    case = Case(SETS[name], page=64, seed=len(name))
    _check_attention(B, case, q_type, full, window=512 if name != "mixed" else 100)


@pytest.mark.parametrize("q_type", [F32, BF16])
@pytest.mark.parametrize("name", ["one", "two", "decode", "verify", "chunk", "chunk_at", "mixed", "pairs", "edges",
                                  "long_chunk", "far_short"])
@pytest.mark.parametrize("full", [True, False])
def test_attention_f32_pool(B, name, full, q_type):
    _check_attention(B, Case(SETS[name], page=32, dtype=F32, seed=3), q_type, full, window=64)


@pytest.mark.parametrize("n_kv,page", [(1, 16), (3, 48), (5, 80), (8, 256)])
@pytest.mark.parametrize("window", [0, 1, 9, 17, 300])
def test_f32_pool_heads_pages_windows(B, n_kv, page, window):
    for q_type in (F32, BF16):
        _check_attention(B, Case(SETS["mixed"], n_kv=n_kv, page=page, dtype=F32, seed=page, pad=5), q_type, window == 0,
                         window=window or 512, q_pad=8)


@pytest.mark.parametrize("page", [16, 32, 48, 80, 128, 256, 1024])
@pytest.mark.parametrize("name", ["decode", "mixed", "pairs"])
def test_page_sizes(B, page, name):
    _check_attention(B, Case(SETS[name], page=page, seed=page), BF16)
    _check_attention(B, Case(SETS[name], page=page, seed=page + 1), F32, full=False, window=130)


@pytest.mark.parametrize("n_kv", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("name", ["decode", "mixed", "pairs"])
def test_head_counts(B, n_kv, name):
    _check_attention(B, Case(SETS[name], n_kv=n_kv, page=32, seed=n_kv), BF16)
    _check_attention(B, Case(SETS[name], n_kv=n_kv, page=32, seed=n_kv), F32)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 127, 128, 129, 100000])
@pytest.mark.parametrize("q_type", [F32, BF16])
@pytest.mark.parametrize("name", ["mixed", "pairs"])
def test_windows(B, name, window, q_type):
    _check_attention(B, Case(SETS[name], page=16, seed=window), q_type, full=False, window=window)
    _check_attention(B, Case(SETS[name], page=128, seed=window), q_type, full=False, window=window)


@pytest.mark.parametrize("scale", [0.0, 0.01, 0.25, -0.0625])
@pytest.mark.parametrize("name", ["mixed", "pairs"])
def test_scales(B, name, scale):
    _check_attention(B, Case(SETS[name], page=64, seed=9), F32, scale=scale)
    _check_attention(B, Case(SETS[name], page=64, seed=9), BF16, scale=scale)


def test_strided_queries_and_padded_rows(B):
    for q_type in (F32, BF16):
        _check_attention(B, Case(SETS["mixed"], page=64, seed=4, pad=37), q_type, q_pad=2048 + 8, max_q=200)
        _check_attention(B, Case(SETS["pairs"], page=64, seed=4, pad=37), q_type, q_pad=2048 + 8)


@pytest.mark.parametrize("q_type", [F32, BF16])
@pytest.mark.parametrize("name", ["verify", "mixed", "edges", "pairs"])
def test_queries_of_other_sequences_do_not_matter(B, name, q_type):
    """Rows of NaN queries (padding, and every second sequence) next to
    others in a tile: the others' results are bit for bit what they were."""
    case = Case(SETS[name], page=32, seed=12, pad=29)
    g, ws = _geom(B), B.make_paged_workspace(_geom(B))
    case.fill()
    q = torch.randn(case.n_tokens, 4096, generator=case.g, device="cuda").to(q_type)
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    pool = B.PagePool(case.k, case.v)
    B.spark_paged_attention(g, q, pool, B.SPARK_FULL, case.batch(B), a, ws)
    kept = torch.zeros(case.n_tokens, dtype=torch.bool, device="cuda")
    starts = case.q_start.tolist()
    for s in range(0, len(case.seqs), 2):
        kept[starts[s]:starts[s + 1]] = True
    q[~kept] = float("nan")
    B.spark_paged_attention(g, q, pool, B.SPARK_FULL, case.batch(B), b, ws)
    assert B.spark_attn_error_word(ws) == 0
    assert torch.equal(a[kept], b[kept]) and bool(torch.isfinite(a).all())


def test_many_sequences(B):
    r = np.random.default_rng(2)
    seqs = [(int(c), int(min(c, n))) for c, n in zip(r.integers(0, 90, 1024), r.integers(0, 3, 1024))]
    _check_attention(B, Case(seqs, n_kv=1, page=16, seed=6), F32)
    _check_attention(B, Case(seqs, n_kv=1, page=16, seed=6), BF16, full=False, window=20)


def test_nothing_to_do(B):
    """Sequences without new tokens only: nothing is written, nothing reported."""
    for max_q in (1, 20, 64):
        case = Case([(40, 0), (0, 0)], page=16, seed=3, pad=70)
        _check_attention_empty(B, case, max_q)


def _check_attention_empty(B, case, max_q):
    g = _geom(B)
    q = torch.randn(case.n_tokens, 4096, device="cuda")
    a = torch.full_like(q, 5.0)
    ws = B.make_paged_workspace(g)
    batch, pool = case.batch(B, max_q=max_q), B.PagePool(case.k, case.v)
    B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, a, ws)
    k0 = case.k.clone()
    B.spark_paged_append(g, q[:, :1024], q[:, 1024:2048], pool, batch, ws)
    assert B.spark_attn_error_word(ws) == 0
    assert bool((a == 5.0).all()) and torch.equal(case.k.view(torch.int16), k0.view(torch.int16))


def test_pages_far_into_a_pool(B):
    """Page offsets beyond 2^32 bytes, in the append, the attention kernels and
    the copies of a fork."""
    page, n_kv, n_pages = 1024, 8, 1200                       # 4 MB a page: 4.7 GB of K and of V
    free = torch.cuda.mem_get_info()[0]
    if free < 14 << 30:
        pytest.skip("needs 14 GB")
    k = torch.empty(n_pages, page, n_kv, D, device="cuda", dtype=BF16)
    v = torch.empty_like(k)
    pool, g = B.PagePool(k, v), _geom(B, n_kv)
    ws = B.make_paged_workspace(g)
    gen = torch.Generator(device="cuda").manual_seed(1)
    seqs = [(70, 70), (3, 3), (1100, 40)]
    table = _i32([[1199, -1, -1], [1100, -1, -1], [1150, 1198, -1]])
    start, lens = _i32([0, 70, 73, 113]), _i32([70, 3, 1100])
    # the third sequence's first rows come by an append of their own
    x = torch.randn(1060, 2 * n_kv * D, generator=gen, device="cuda").to(BF16)
    B.spark_paged_append(g, x[:, :n_kv * D], x[:, n_kv * D:], pool,
                         B.PagedBatch(table[2:], _i32([0, 1060]), _i32([1060]), 1060, 1060), ws)
    y = torch.randn(113, 2 * n_kv * D, generator=gen, device="cuda").to(BF16)
    B.spark_paged_append(g, y[:, :n_kv * D], y[:, n_kv * D:], pool, B.PagedBatch(table, start, lens, 113, 70), ws)
    assert torch.equal(k[1199, 69].reshape(-1), y[69, :n_kv * D]) and torch.equal(v[1198, 75].reshape(-1), y[112, n_kv * D:])
    case = Case(seqs, n_kv=n_kv, page=16, seed=2)
    rows = [y[:70], y[70:73], torch.cat([x, y[73:]])]
    case.rows_k = [r[:, :n_kv * D].reshape(-1, n_kv, D) for r in rows]
    case.rows_v = [r[:, n_kv * D:].reshape(-1, n_kv, D) for r in rows]
    q = torch.randn(113, 4 * n_kv * D, generator=gen, device="cuda").to(BF16)
    a = torch.zeros_like(q)
    B.spark_paged_attention(g, q, pool, B.SPARK_FULL, B.PagedBatch(table, start, lens, 113, 70), a, ws)
    want, bound = _reference(case, q, 0, 0.0625, BF16, 2.0**-8)
    assert ((a.double().view(want.shape) - want).abs() / bound).max().item() <= 1.0
    one = torch.zeros(1, 4 * n_kv * D, device="cuda", dtype=BF16)      # its last token by the single-token kernel
    B.spark_paged_attention(g, q[112:], pool, B.SPARK_FULL, B.PagedBatch(table[2:], _i32([0, 1]), _i32([1100]), 1, 1), one, ws)
    assert ((one.double().view(1, -1, D) - want[112:]).abs() / bound[112:]).max().item() <= 1.0
    assert B.spark_attn_error_word(ws) == 0
    tws = B.make_pages_workspace(n_pages, 3)
    new = torch.zeros_like(table)
    k[0].fill_(0)
    B.spark_pages_remap(g, [pool], table, _i32([0, 0, -1]), _i32([70, 70, 0]), _i32([70, 70, 0]), new, tws)
    assert B.spark_attn_error_word(tws) == 0 and new.tolist() == [[1199, -1, -1], [0, -1, -1], [-1, -1, -1]]
    assert torch.equal(k[0, :70], k[1199, :70]) and torch.equal(v[0, :70], v[1199, :70]) and not bool(k[0, 70:].any())


def test_large_scores_and_one_dominant_row(B):
    """Scores of hundreds: the running maximum moves from tile to tile."""
    for q_type in (F32, BF16):
        case = Case([(900, 1), (700, 200)], page=64, seed=8)
        for s in range(2):
            ramp = torch.linspace(0.1, 6.0, case.ctx[s], device="cuda")[:, None, None]
            case.rows_k[s] = (case.rows_k[s].float() * ramp).to(BF16)
        g = _geom(B)
        case.fill()
        q = (torch.randn(case.n_tokens, 4096, generator=case.g, device="cuda") * 5).to(q_type)
        a = torch.zeros_like(q)
        ws = B.make_paged_workspace(g)
        B.spark_paged_attention(g, q, B.PagePool(case.k, case.v), B.SPARK_FULL, case.batch(B), a, ws)
        assert B.spark_attn_error_word(ws) == 0
        want, bound = _reference(case, q, 0, 0.0625, q_type, 2.0**-16 if q_type == F32 else 2.0**-8)
        # scores of up to 2^9 or so: their scaling to base 2 alone is off by 2^-24 * 2^9 * 2 ln 2
        err = (a.double().view(want.shape) - want).abs() / (bound + 2.0**-14 * want.abs().amax())
        assert err.max().item() <= 1.0


def test_repeated_and_unordered_calls_agree(B):
    """One workspace, call after call, in any order of batches: bit-identical."""
    g = _geom(B)
    ws = B.make_paged_workspace(g)
    runs = []
    for name in ("decode", "big_chunk", "mixed", "long", "pairs"):
        case = Case(SETS[name], page=64, seed=1)
        case.fill()
        q = torch.randn(case.n_tokens, 4096, generator=case.g, device="cuda")
        runs.append((case, q, torch.zeros_like(q), torch.zeros_like(q)))
    for which, order in ((2, (0, 1, 2, 3, 4)), (3, (4, 3, 1, 0, 2))):
        for i in order:
            case, q = runs[i][:2]
            B.spark_paged_attention(g, q, B.PagePool(case.k, case.v), B.SPARK_FULL, case.batch(B), runs[i][which], ws)
    assert B.spark_attn_error_word(ws) == 0
    for _, _, x, y in runs:
        assert torch.equal(x, y)


def test_bad_entries_raise_the_error_word(B):
    """What only the kernels can see: reported, never followed."""
    def run(change, max_q=None):
        case = Case([(100, 3), (40, 2), (50, 1)], page=16, seed=5)
        case.fill()
        change(case)
        g = _geom(B)
        ws = B.make_paged_workspace(g)
        q = torch.randn(6, 4096, device="cuda")
        a = torch.zeros_like(q)
        kv = torch.ones(6, 1024, device="cuda")
        b = case.batch(B, n_tokens=6, max_q=max_q or 3)
        B.spark_paged_attention(g, q, B.PagePool(case.k, case.v), B.SPARK_FULL, b, a, ws)
        att = B.spark_attn_error_word(ws)
        B.spark_paged_append(g, kv, kv, B.PagePool(case.k, case.v), b, ws)
        return att, B.spark_attn_error_word(ws), a

    def put(name, at, val):
        def change(case):
            getattr(case, name)[at] = val
        return change
    assert run(lambda c: None)[:2] == (0, 0)
    for change in (put("table", (0, 6), -1), put("table", (0, 6), 2**31 - 1), put("table", (1, 2), -5),
                   put("seq_len", 0, 2), put("seq_len", 1, -4), put("seq_len", 2, 2**31 - 1),
                   put("q_start", 1, -3), put("q_start", 3, 7), put("q_start", 2, 1)):
        att, app, a = run(change)
        assert att == 2 and app == 2
    assert run(put("table", (0, 1), -1))[:2] == (2, 0)          # a page that is read only
    assert run(lambda c: None, max_q=2)[:2] == (2, 2)           # a sequence brings more than max_q_len
    # a sequence whose length makes no sense leaves the others' results alone
    good, bad = run(lambda c: None)[2], run(put("seq_len", 0, 1))[2]
    assert bool((bad[:3] == 0).all())


def test_calls_at_once_on_their_own_workspaces(B):
    """Streams side by side, each with its workspace and its kind of batch:
    the results of the same calls one after another."""
    g = _geom(B)
    runs = []
    for i, (name, q_type) in enumerate((("decode", F32), ("mixed", F32), ("pairs", BF16), ("big_chunk", F32),
                                        ("verify", BF16), ("long", BF16), ("edges", F32))):
        case = Case(SETS[name], page=(16, 64)[i % 2], dtype=F32 if name == "edges" else BF16, seed=20 + i)
        case.fill()
        q = torch.randn(case.n_tokens, 4096, generator=case.g, device="cuda").to(q_type)
        ws = B.make_paged_workspace(g)
        want, got = torch.zeros_like(q), torch.zeros_like(q)
        runs.append((q, B.PagePool(case.k, case.v), case.batch(B), want, got, ws, torch.cuda.Stream(), case))
    for q, pool, batch, want, _, ws, _, _ in runs:
        B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, want, ws)
    torch.cuda.synchronize()
    for _ in range(5):
        for q, pool, batch, _, got, ws, st, _ in runs:
            B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, got, ws, stream=st)
    torch.cuda.synchronize()
    for _, _, _, want, got, ws, _, _ in runs:
        assert B.spark_attn_error_word(ws) == 0 and torch.equal(want, got)


@pytest.mark.parametrize("q_type,dtype", [(F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("page", [16, 64])
def test_bad_pages_under_long_chunks(B, page, q_type, dtype):
    """Entries outside the pool under long chunks: reported, and the other
    sequence's results are what they were."""
    case = Case([(200, 90), (130, 70)], page=page, dtype=dtype, seed=15)
    case.fill()
    g, ws, pool = _geom(B), B.make_paged_workspace(_geom(B)), B.PagePool(case.k, case.v)
    q = torch.randn(160, 4096, generator=case.g, device="cuda").to(q_type)
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    B.spark_paged_attention(g, q, pool, B.SPARK_FULL, case.batch(B), a, ws)
    assert B.spark_attn_error_word(ws) == 0
    keep = case.table.clone()
    for entry in (-1, case.k.shape[0], 2**31 - 1, -2**31):
        case.table.copy_(keep)
        case.table[0, 1] = entry
        b.zero_()
        B.spark_paged_attention(g, q, pool, B.SPARK_FULL, case.batch(B), b, ws)
        assert B.spark_attn_error_word(ws) == 2
        assert torch.equal(a[90:], b[90:])
        B.spark_attn_workspace_init(ws)


@pytest.mark.parametrize("q_type,dtype", [(F32, BF16), (BF16, BF16), (F32, F32)])
def test_captured_long_chunks_replay_with_new_lengths(B, q_type, dtype):
    g = _geom(B)
    case = Case([(300, 130), (200, 70)], page=16, dtype=dtype, seed=16)
    case.fill()
    pool, ws = B.PagePool(case.k, case.v), B.make_paged_workspace(g)
    q = torch.randn(200, 4096, generator=case.g, device="cuda").to(q_type)
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    batch = case.batch(B)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, a, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, a, ws)
    for lens, new in (((300, 200), (130, 70)), ((33, 199), (33, 1)), ((290, 2), (0, 2)), ((129, 64), (128, 64))):
        case.seq_len.copy_(_i32(lens))
        case.q_start.copy_(_i32([0, new[0], sum(new)]))
        a.fill_(3.0)
        b.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, b, ws)
        torch.cuda.synchronize()
        assert torch.equal(a, b) and bool((a[sum(new):] == 3.0).all())
    assert B.spark_attn_error_word(ws) == 0


def test_captured_calls_replay_with_new_lengths(B):
    g = _geom(B)
    case = Case([(200, 4), (90, 1)], page=16, seed=12)
    case.fill()
    pool, ws = B.PagePool(case.k, case.v), B.make_paged_workspace(g)
    q = torch.randn(5, 4096, generator=case.g, device="cuda")
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    batch = case.batch(B)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, a, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, a, ws)
    for lens, new in (((200, 90), (4, 1)), ((33, 90), (1, 3)), ((150, 2), (0, 2))):
        case.seq_len.copy_(_i32(lens))
        case.q_start.copy_(_i32([0, new[0], sum(new)]))
        a.fill_(3.0)
        b.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, b, ws)
        torch.cuda.synchronize()
        assert torch.equal(a, b) and bool((a[sum(new):] == 3.0).all())
    assert B.spark_attn_error_word(ws) == 0


def test_another_stream_orders_the_work(B):
    g = _geom(B)
    case = Case(SETS["mixed"], page=64, seed=14)
    case.fill()
    ws = B.make_paged_workspace(g)
    q = torch.randn(case.n_tokens, 4096, generator=case.g, device="cuda")
    want = torch.zeros_like(q)
    B.spark_paged_attention(g, q, B.PagePool(case.k, case.v), B.SPARK_FULL, case.batch(B), want, ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    late, got = torch.zeros_like(q), torch.zeros_like(q)
    with torch.cuda.stream(st):
        torch.mm(torch.randn(4096, 4096, device="cuda"), torch.randn(4096, 4096, device="cuda"))
        late.copy_(q)
    B.spark_paged_attention(g, late, B.PagePool(case.k, case.v), B.SPARK_FULL, case.batch(B), got, ws, stream=st)
    st.synchronize()
    assert torch.equal(got, want)


# ---------------------------------------------------------------------------
# the write of new rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("x_type", [BF16, F32])
@pytest.mark.parametrize("page,n_kv,name", [(16, 4, "mixed"), (48, 1, "verify"), (64, 8, "decode"), (1024, 3, "chunk_at")])
def test_append(B, page, n_kv, name, x_type, dtype):
    case = Case(SETS[name], n_kv=n_kv, page=page, dtype=dtype, seed=1, pad=5)
    g = _geom(B, n_kv)
    ws = B.make_paged_workspace(g)
    row = n_kv * D
    x = torch.randn(case.n_tokens, 3 * row, generator=case.g, device="cuda").to(x_type)
    k0, v0 = case.k.clone(), case.v.clone()
    t = 0
    for s, (c, n) in enumerate(case.seqs):
        p, r = case.where(s)
        k0[p[c - n:], r[c - n:]] = x[t:t + n, row:2 * row].reshape(n, n_kv, D).to(dtype)
        v0[p[c - n:], r[c - n:]] = x[t:t + n, 2 * row:].reshape(n, n_kv, D).to(dtype)
        t += n
    B.spark_paged_append(g, x[:, row:2 * row], x[:, 2 * row:], B.PagePool(case.k, case.v), case.batch(B), ws)
    assert B.spark_attn_error_word(ws) == 0
    iv = torch.int16 if dtype == BF16 else torch.int32
    assert torch.equal(case.k.view(iv), k0.view(iv)) and torch.equal(case.v.view(iv), v0.view(iv))


# ---------------------------------------------------------------------------
# page tables
# ---------------------------------------------------------------------------

def _remap_oracle(table, parent, keep, new, page, n_pages):
    """(new table, [(src, dst, rows)]), or None where the call is refused."""
    n, width = table.shape
    whole, part = set(), {}
    for s in range(n):
        if not -1 <= parent[s] < n or not 0 <= keep[s] <= new[s] or (parent[s] < 0 and keep[s]) or new[s] > width * page:
            return None
        for i in range(-(-keep[s] // page)):
            p = table[parent[s], i]
            if not 0 <= p < n_pages:
                return None
            if (i + 1) * page <= keep[s]:
                whole.add(int(p))
            else:
                part.setdefault(int(p), s)
    free = [p for p in range(n_pages) if p not in whole and p not in part]
    out, moves = np.full_like(table, -1), []
    for s in range(n):
        kept = -(-keep[s] // page)
        for i in range(-(-new[s] // page)):
            if i < kept:
                p = int(table[parent[s], i])
                if keep[s] % page and i == kept - 1 and (p in whole or part[p] != s):
                    if not free:
                        return None
                    moves.append((p, free[0], int(keep[s] % page)))
                    p = free.pop(0)
            else:
                if not free:
                    return None
                p = free.pop(0)
            out[s, i] = p
    return out, moves


def _scattered(r, lens, page, n_pages, width):
    order = r.permutation(n_pages)
    table, at = np.full((len(lens), width), -1, dtype=np.int64), 0
    for s, c in enumerate(lens):
        m = -(-c // page)
        table[s, :m] = order[at:at + m]
        at += m
    return table


def _pools(B, layers, n_pages, page, n_kv, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(layers, 2, n_pages, page, n_kv, D, generator=g, device="cuda").to(dtype)
    return x, [B.PagePool(x[i, 0], x[i, 1]) for i in range(layers)]


def _run_remap(B, table, parent, keep, new, page, n_pages, layers=2, n_kv=2, dtype=BF16, seed=0):
    x, pools = _pools(B, layers, n_pages, page, n_kv, dtype, seed)
    before = x.clone()
    ws = B.make_pages_workspace(n_pages, len(parent))
    old, out = _i32(table), torch.full(table.shape, -99, dtype=torch.int32, device="cuda")
    B.spark_pages_remap(_geom(B, n_kv), pools, old, _i32(parent), _i32(keep), _i32(new), out, ws)
    word = B.spark_attn_error_word(ws)
    assert np.array_equal(old.cpu().numpy(), np.asarray(table, dtype=np.int32))
    want = _remap_oracle(np.asarray(table), parent, keep, new, page, n_pages)
    if want is None:
        assert word in (2, 4) and bool((out == -99).all()) and torch.equal(x, before)
        return word
    assert word == 0
    assert np.array_equal(out.cpu().numpy(), want[0])
    for src, dst, rows in want[1]:
        before[:, :, dst, :rows] = before[:, :, src, :rows]
    assert torch.equal(x, before)
    return 0


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("page", [16, 48])
def test_remap_random(B, seed, page):
    r = np.random.default_rng(seed)
    n = int(r.integers(1, 60))
    lens = r.integers(0, 20 * page, n)
    width = 24
    n_pages = int(sum(-(-lens // page)) + r.integers(0, 12 * n + 2))
    table = _scattered(r, lens, page, n_pages, width) if n_pages else np.full((n, width), -1)
    n_pages = max(1, n_pages)
    parent = r.integers(-1, n, n)
    keep = np.array([0 if p < 0 else r.integers(0, lens[p] + 1) for p in parent])
    new = keep + r.integers(0, 3 * page, n)
    _run_remap(B, table, parent.tolist(), keep.tolist(), new.tolist(), page, n_pages, seed=seed)


def test_remap_forks_share_whole_pages_and_copy_the_last(B):
    page, n_pages, width = 16, 40, 6
    table = np.full((5, width), -1)
    table[0, :3] = [30, 7, 12]
    table[1, :2] = [3, 39]
    # slots 0..3 all continue sequence 0 (40 rows: 2 whole pages, 8 rows); 4 takes its first page and a half
    for dtype, layers, n_kv in ((BF16, 3, 4), (F32, 1, 1)):
        assert _run_remap(B, table, [0, 0, 0, 0, 0], [40, 40, 40, 40, 24], [41, 41, 90, 40, 25], page, n_pages,
                          layers=layers, n_kv=n_kv, dtype=dtype) == 0
    # all ended; one begins on the lowest pages
    assert _run_remap(B, table, [-1] * 5, [0] * 5, [0, 33, 0, 0, 16], page, n_pages) == 0
    # swapped, cut to nothing, cut at a page's end
    assert _run_remap(B, table, [1, 0, 0, 0, 1], [32, 40, 0, 16, 0], [32, 40, 0, 16, 96], page, n_pages) == 0


def test_remap_is_all_or_nothing(B):
    page, n_pages, width = 16, 8, 6
    table = np.full((3, width), -1)
    table[0, :3] = [1, 5, 2]
    table[1, :3] = [0, 4, 7]
    ok = ([0, 1, -1], [40, 48, 0], [48, 48, 32])
    assert _run_remap(B, table, *ok, page, n_pages) == 0                               # exactly the two free pages
    assert _run_remap(B, table, [0, 1, -1], [40, 48, 0], [48, 48, 33], page, n_pages) == 4   # three wanted
    assert _run_remap(B, table, [0, 1, 0], [40, 48, 40], [48, 49, 49], page, n_pages) == 4
    for change in (dict(p=(0, 3)), dict(p=(0, -2)), dict(k=(0, -1)), dict(k=(0, 49)), dict(k=(2, 5)), dict(n=(1, 97)),
                   dict(n=(1, 2**31 - 1)), dict(k=(0, 2**31 - 1))):
        par, keep, new = (list(x) for x in ok)
        for key, arr in (("p", par), ("k", keep), ("n", new)):
            if key in change:
                arr[change[key][0]] = change[key][1]
        assert _run_remap(B, table, par, keep, new, page, n_pages) == 2, change
    for entry in (-1, 8, 2**31 - 1):
        bad = table.copy()
        bad[0, 1] = entry
        assert _run_remap(B, bad, *ok, page, n_pages) == 2
    bad = table.copy()
    bad[0, 3] = 12345                                                                  # not kept: never looked at
    assert _run_remap(B, bad, *ok, page, n_pages) == 0


def test_remap_at_its_limits(B):
    """1024 slots; a table wider than a block; many more pages than the plan's
    threads; both forms of the plan (pools and tables that fit one CTA's
    shared memory, and larger ones)."""
    r = np.random.default_rng(1)
    for n_pages in (20011, 24576, 24577, 90001):
        table = _scattered(r, r.integers(0, 33, 1024), 16, n_pages, 3)
        keep = np.array([0 if row[0] < 0 else 5 for row in table])
        parent = np.where(keep > 0, np.arange(1024), -1)
        _run_remap(B, table, parent.tolist(), keep.tolist(), (keep + 20).tolist(), 16, n_pages, layers=1, n_kv=1)
    for width in (5000, 32768, 32769):
        wide = _scattered(r, [16 * 4000 + 3, 0], 16, 5000, width)
        _run_remap(B, wide, [0, 0], [16 * 4000 + 3, 16 * 3999 + 1], [16 * 4100, 16 * 3999 + 1], 16, 5000, layers=1, n_kv=1)
    # too few pages, and a bad entry, in the larger form
    assert _run_remap(B, wide, [0, 0], [16 * 4000 + 3] * 2, [16 * 4999] * 2, 16, 5000, layers=1, n_kv=1) == 4
    wide[0, 5] = 5000
    assert _run_remap(B, wide, [0, 0], [16 * 4000 + 3] * 2, [16 * 4001] * 2, 16, 5000, layers=1, n_kv=1) == 2


@pytest.mark.parametrize("seed", range(13))
def test_compact(B, seed):
    r = np.random.default_rng(seed)
    page, n_kv, layers = (16, 2, 3) if seed % 2 and seed < 10 else (32 if seed < 10 else 16, 1, 1)
    n = int(r.integers(1, 40))
    lens = r.integers(0, 12 * page, n)
    need = int(sum(-(-lens // page)))
    n_pages = max(1, need + int(r.integers(0, 3 * need + 2)) * (seed != 4))
    if seed >= 10:
        n_pages = 30000                                         # the plan's larger form
    table = _scattered(r, lens, page, n_pages, 13)
    if n > 2 and seed % 3 == 0:
        table[1] = table[0]                                     # shared pages
    live = np.unique(table[table >= 0])
    m = len(live)
    src, dst = live[live >= m], np.setdiff1d(np.arange(m), live)
    to = np.arange(n_pages)
    to[src] = dst
    want = np.where(table >= 0, to[table], -1)
    x, pools = _pools(B, layers, n_pages, page, n_kv, BF16, seed)
    after = x.clone()
    if m:
        after[:, :, torch.tensor(dst, device="cuda")] = x[:, :, torch.tensor(src, device="cuda")]
    ws = B.make_pages_workspace(n_pages, n)
    old = _i32(table)
    out = torch.zeros_like(old) if seed % 2 else old            # apart, or in place
    n_live = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    B.spark_pages_compact(_geom(B, n_kv), pools, old, out, n_live, ws)
    assert B.spark_attn_error_word(ws) == 0
    assert int(n_live) == m and np.array_equal(out.cpu().numpy(), want)
    assert torch.equal(x[:, :, :m], after[:, :, :m]) and torch.equal(x, after)


def test_compact_refuses_bad_entries(B):
    x, pools = _pools(B, 1, 20, 16, 1, BF16, 0)
    before = x.clone()
    ws = B.make_pages_workspace(20, 2)
    for entry in (-2, 20, 2**31 - 1):
        table = _i32([[19, -1, 3], [entry, 7, -1]])
        out = torch.full_like(table, -99)
        n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
        B.spark_pages_compact(_geom(B, 1), pools, table, out, n_live, ws)
        assert B.spark_attn_error_word(ws) == 2
        assert int(n_live) == -1 and bool((out == -99).all()) and torch.equal(x, before)


# ---------------------------------------------------------------------------
# the block, and the operators as a server runs them
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("is_full", [True, False])
@pytest.mark.parametrize("dtype,hidden", [("bf16", 2560), ("f32", 256)])
def test_block_matches_the_contiguous_cache(B, is_full, dtype, hidden):
    """spark_attn_paged on pages against spark_attn_prefill and the oracle on
    a contiguous cache: three sequences, a chunk, a few tokens, one token."""
    spec = [(600, 40), (90, 3), (700, 1)]
    geom = _geom(B)
    geom.hidden = hidden
    wl = synth.Workload("paged", "", dtype, [c for c, _ in spec], [synth.LayerSpec(is_full, 0)], seed=77, hidden=hidden)
    td = wl.torch_dtype
    w = synth.make_weights(wl, 0, "cuda")
    case = Case([(c, n) for c, n in spec], page=32, dtype=td, seed=3)
    case.fill()
    n_tok = case.n_tokens
    h = torch.randn(n_tok, hidden, generator=case.g, device="cuda")
    positions = [p for c, n in spec for p in range(c - n, c)]
    lw = B.LayerWeights(**w)
    cls = B.SPARK_FULL if is_full else B.SPARK_SLIDING
    ws, pws = B.make_workspace(geom, n_tok), B.make_paged_workspace(geom)
    out = torch.zeros_like(h)
    B.spark_attn_paged(geom, h, lw, B.PagePool(case.k, case.v), cls, case.batch(B), positions, out, ws, pws)
    assert B.spark_attn_error_word(ws) == 0 and B.spark_attn_error_word(pws) == 0
    t = 0
    for s, (c, n) in enumerate(spec):
        kc, vc = case.rows_k[s][None].clone(), case.rows_v[s][None].clone()
        k_np, v_np = synth.to_numpy(kc), synth.to_numpy(vc)
        ref = torch.zeros(n, hidden, device="cuda")
        wsp = B.make_workspace(geom, n)
        B.spark_attn_prefill(geom, h[t:t + n].contiguous(), lw, B.KvLayer(kc, vc, 0), cls, c - n, ref, wsp)
        assert B.spark_attn_error_word(wsp) == 0
        assert_close((out[t:t + n] - h[t:t + n]).cpu(), (ref - h[t:t + n]).cpu(), f"sequence {s}")
        p, r = case.where(s)
        # the rows written: the projections may take another kernel at another batch size
        assert_close(case.k[p, r].double().cpu(), kc[0].double().cpu(), f"K of sequence {s}")
        assert_close(case.v[p, r].double().cpu(), vc[0].double().cpu(), f"V of sequence {s}")
        if n == 1:
            res = oracle.decode_step(oracle.OracleGeometry(hidden=hidden), synth.to_numpy(h[t:t + 1]).astype(np.float64),
                                     np_weights(w), k_np, v_np, is_full, [c - 1], 0)
            assert_close((out[t:t + 1] - h[t:t + 1]).cpu().double().numpy()[0], res["o"][0], "oracle")
        t += n


def test_block_in_place_and_with_padded_rows(B):
    geom = _geom(B)
    wl = synth.Workload("paged", "", "bf16", [50], [synth.LayerSpec(True, 0)], seed=78)
    lw = B.LayerWeights(**synth.make_weights(wl, 0, "cuda"))
    outs = []
    for in_place, pad in ((False, 0), (True, 0), (False, 3)):
        case = Case([(50, 2), (70, 6)], page=16, seed=3, pad=pad)
        case.fill()
        h = torch.randn(8, 2560, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
        h = torch.cat([h, torch.ones(pad, 2560, device="cuda")])
        out = h if in_place else torch.zeros_like(h)
        ws, pws = B.make_workspace(geom, 8 + pad), B.make_paged_workspace(geom)
        B.spark_attn_paged(geom, h, lw, B.PagePool(case.k, case.v), B.SPARK_FULL, case.batch(B),
                           [48, 49] + list(range(64, 70)) + [0] * pad, out, ws, pws)
        assert B.spark_attn_error_word(pws) == 0
        outs.append(out[:8])
    assert torch.equal(outs[0], outs[1])
    assert_close(outs[2].cpu(), outs[0].cpu(), "padded")


def test_serving_run(B):
    """Two prompts, a fork, rejected drafts, an ended sequence and a compaction
    in two layers: every step's logits scores equal those of a run on
    contiguous caches."""
    geom = _geom(B)
    page, n_pages, width, vocab = 16, 24, 6, 1000
    wl = synth.Workload("serve", "", "bf16", [80], [synth.LayerSpec(True, 0), synth.LayerSpec(False, 0)], seed=79)
    layers = [B.LayerWeights(**synth.make_weights(wl, i, "cuda")) for i in range(2)]
    classes = [B.SPARK_FULL, B.SPARK_SLIDING]
    head = synth.make_head(3, 2560, vocab, torch.bfloat16, "cuda")
    x, pools = _pools(B, 2, n_pages, page, 4, BF16, 1)
    x.fill_(float("nan"))
    tables = [torch.full((3, width), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    ws, pws = B.make_workspace(geom, 64), B.make_paged_workspace(geom)
    tws, sws, hws = B.make_pages_workspace(n_pages, 3), B.make_logprobs_workspace(64, 4), B.make_mlp_workspace(geom, 0, 64)
    gen = torch.Generator(device="cuda").manual_seed(4)
    history = [[], [], []]                       # each slot's residual inputs, for the contiguous run

    def step(parent, keep, feed):
        """parent, keep per slot; feed: new residual rows per slot."""
        nonlocal history
        n = [f.shape[0] for f in feed]
        new = [k + m for k, m in zip(keep, n)]
        B.spark_pages_remap(geom, pools, tables[0], _i32(parent), _i32(keep), _i32(new), tables[1], tws)
        tables.reverse()
        history = [(history[p][:k] if p >= 0 else []) + list(f) for p, k, f in zip(parent, keep, feed)]
        batch = B.PagedBatch(tables[0], _i32(np.concatenate([[0], np.cumsum(n)])), _i32(new), sum(n), max(n))
        pos = [p for k, e in zip(keep, new) for p in range(k, e)]
        h = torch.cat(feed)
        for w, p, c in zip(layers, pools, classes):
            B.spark_attn_paged(geom, h, w, p, c, batch, pos, h, ws, pws)
        logits = torch.zeros(sum(n), vocab, device="cuda")
        B.spark_head_logits(geom, h, head["norm_w"], head["embed"], logits, hws)
        res = _scores(B, logits, _i32(np.arange(sum(n)) * 7 % vocab), 4, sws)
        assert [B.spark_attn_error_word(t) for t in (ws, pws, tws, sws, hws)] == [0] * 5
        # the same rows on contiguous caches, each sequence from its start
        at = 0
        for s, m in enumerate(n):
            if m == 0:
                continue
            hh = torch.stack(history[s])
            wss = B.make_workspace(geom, len(hh))
            for w, c in zip(layers, classes):
                kc = torch.zeros(1, len(hh), 4, D, device="cuda", dtype=BF16)
                B.spark_attn_prefill(geom, hh, w, B.KvLayer(kc, torch.zeros_like(kc), 0), c, 0, hh, wss)
            ref = torch.zeros(len(hh), vocab, device="cuda")
            B.spark_head_logits(geom, hh, head["norm_w"], head["embed"], ref, B.make_mlp_workspace(geom, 0, len(hh)))
            assert_close(logits[at:at + m].cpu(), ref[-m:].cpu(), f"slot {s}")
            lp = torch.log_softmax(logits[at:at + m].double(), -1)
            tg = (torch.arange(at, at + m, device="cuda") * 7) % vocab
            assert torch.allclose(res["logprob"][at:at + m].double(), lp[torch.arange(m), tg], atol=1e-5, rtol=1e-5)
            at += m

    def rows(m):
        return torch.randn(m, 2560, generator=gen, device="cuda")
    step([-1, -1, -1], [0, 0, 0], [rows(37), rows(16), rows(0)])
    step([0, 1, 0], [37, 16, 37], [rows(1), rows(5), rows(1)])       # slot 2 forks slot 0
    step([0, 1, 2], [38, 18, 38], [rows(1), rows(1), rows(2)])       # slot 1's last drafts rejected
    step([0, -1, 2], [39, 0, 40], [rows(1), rows(3), rows(1)])       # slot 1 ends, another begins
    n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spark_pages_compact(geom, pools, tables[0], tables[0], n_live, tws)
    used = tables[0][tables[0] >= 0].unique()
    assert int(n_live) == len(used) and int(used.max()) == len(used) - 1
    step([0, 1, 2], [40, 3, 41], [rows(1), rows(1), rows(1)])


# ---------------------------------------------------------------------------
# token scores
# ---------------------------------------------------------------------------

def _scores(B, logits, targets, k, ws=None):
    n = logits.shape[0]
    out = {"logprob": torch.full((n,), 9.0, device="cuda"), "entropy": torch.full((n,), 9.0, device="cuda"),
           "top_ids": torch.full((n, k), -9, dtype=torch.int32, device="cuda"),
           "top_logprobs": torch.full((n, k), 9.0, device="cuda")}
    ws = B.make_logprobs_workspace(n, k) if ws is None else ws
    B.spark_token_logprobs(logits, targets, out["logprob"], out["entropy"], out["top_ids"], out["top_logprobs"], ws)
    torch.cuda.synchronize()
    out["word"] = B.spark_attn_error_word(ws)
    return out


def _check_scores(got, logits, targets, k):
    """Sums of vocab fp32 terms in a tree: their relative error is within
    2^-24 (depth + the 64 terms of a thread's tiles + the exponential's 2^-22
    and its argument's |x - m| 2^-23); 2^-17 covers it for |x - m| < 32 (what
    lies further below the maximum weighs less than e^-32).  A log probability
    then is off by that plus 2^-23 of its parts; the entropy by 32 times it
    (its terms are weighted by |x - m|)."""
    x = logits.double()
    m = x.amax(-1, keepdim=True)
    lp = x - m - (x - m).exp().sum(-1, keepdim=True).log()
    rows = torch.arange(len(x), device="cuda")
    t = targets.long()
    want = torch.where(t >= 0, lp[rows, t.clamp(min=0)], 0.0)
    tol = 2.0**-17 + 2.0**-22 * (x.abs().amax(-1).nan_to_num(0, 0, 0).clamp(max=1e6) + want.abs().nan_to_num(0, 0, 0))
    g = got["logprob"].double()
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(g), inf) and bool(((g - want).abs()[~inf] <= tol[~inf]).all())
    p = lp.exp()
    h = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    assert bool(((got["entropy"].double() - h).abs() <= 2.0**-12 * 0.25 + 2.0**-20 * h.abs()).all())
    ids = torch.sort(logits.float(), dim=-1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(got["top_ids"].long(), ids)
    top = lp.gather(1, ids)
    fin = torch.isfinite(top)
    assert torch.equal(torch.isfinite(got["top_logprobs"]), fin)
    assert bool(((got["top_logprobs"].double() - top).abs()[fin] <= (tol + 2.0**-20 * 40)[:, None].expand_as(top)[fin]).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,vocab,k", [(1, 1, 1), (1, 1, 0), (3, 2, 2), (2, 31, 31), (5, 257, 5), (1, 4097, 20),
                                       (7, 8191, 32), (64, 1000, 1), (1, 131072, 20), (2, 131071, 32), (33, 50001, 5),
                                       (700, 5003, 3), (1, 262144, 0), (2100, 64, 4),
                                       # rows in parts: 65536 and up
                                       (1, 65535, 20), (3, 65536, 32), (5, 65539, 1), (33, 70001, 6), (128, 66000, 9),
                                       (129, 65537, 2), (1, 1000003, 32)])
def test_logprobs(B, n, vocab, k, dtype):
    g = torch.Generator(device="cuda").manual_seed(n + vocab)
    x = (torch.randn(n, vocab, generator=g, device="cuda") * 3).to(dtype)
    t = torch.randint(-1, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
    got = _scores(B, x, t, k)
    assert got["word"] == 0
    _check_scores(got, x, t, k)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ld,off,vocab", [(5007, 0, 5000), (5008, 3, 5000), (5001, 1, 5000), (6000, 7, 5000),
                                          (70009, 0, 70001), (70001, 1, 69999), (66000, 5, 65536)])
def test_logprobs_strides_and_alignment(B, ld, off, vocab, dtype):
    x = (torch.randn(9, ld, device="cuda") * 2).to(dtype)
    v = x[:, off:off + vocab]
    t = torch.arange(9, dtype=torch.int32, device="cuda") * 500
    x[:, :off] = float("inf")                       # outside the rows: never looked at
    x[:, off + vocab:] = float("nan")
    got = _scores(B, v, t, 7)
    assert got["word"] == 0
    _check_scores(got, v, t, 7)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("v", [9000, 81000])
def test_logprobs_ties_orders_and_masks(B, v, dtype):
    i = torch.arange(v, device="cuda", dtype=F32)
    neg = torch.full((v,), -float("inf"), device="cuda")
    rows = [torch.zeros(v, device="cuda"),                                  # all equal: the lowest indices
            -torch.zeros(v, device="cuda") + torch.where(i % 2 == 0, 0.0, -0.0),  # -0 and 0 are equal
            i / v, -i / v, (i * 7919 % v) / v,                              # ascending, descending, mixed
            torch.where(i % (v // 9) == 999, 0.5, neg),                     # nine tokens left
            torch.where(i == 8888, 2.0, neg),                               # one left
            torch.where((i == 8998) | (i == 8990), 0.0, torch.where(i == 4100, -0.0, neg)),  # three, equal, far apart
            torch.where(i % (7 * v // 90) == 3, 1.0, 0.0),                  # thirteen above a plateau
            torch.where(i < 4000, torch.finfo(dtype).min, 1.0),             # the type's lowest value as a mask
            torch.where(i == 5, 80.0, torch.randn(v, device="cuda"))]       # all but certain
    x = torch.stack(rows).to(dtype)
    t = _i32([8999, 0, 8999, 0, 17, 999, 0, 4100, 3, 3, 5])
    got = _scores(B, x, t, 16)
    assert got["word"] == 0
    _check_scores(got, x, t, 16)
    assert got["logprob"][6].item() == -float("inf") and got["entropy"][6].item() == 0.0
    assert abs(got["entropy"][0].item() - np.log(v)) < 1e-5


@pytest.mark.parametrize("v", [6000, 66001])
def test_logprobs_rows_without_a_distribution(B, v):
    base = torch.randn(v, device="cuda")
    inf, nan = float("inf"), float("nan")
    x = torch.stack([base] * 5)
    x[1] = -inf
    x[2, 77] = inf
    x[3, 5000] = nan
    got = _scores(B, x, _i32([1, 2, 77, 4, -1]), 4)
    assert got["word"] == 0
    for r in (1, 2, 3):
        assert np.isnan(got["logprob"][r].item()) and np.isnan(got["entropy"][r].item())
        assert bool(torch.isnan(got["top_logprobs"][r]).all())
    assert got["logprob"][4].item() == 0.0
    assert got["top_ids"][1].tolist() == [0, 1, 2, 3] and got["top_ids"][2][0].item() == 77
    order = torch.sort(torch.nan_to_num(x[3], nan=-1e30), descending=True, stable=True)[1][:4]
    assert got["top_ids"][3].tolist() == order.tolist()
    _check_scores({k: g[[0, 4]] for k, g in got.items() if k != "word"}, x[[0, 4]], _i32([1, -1]), 4)
    bad = _scores(B, x[:1].repeat(3, 1), _i32([v, -2, 5]), 0)
    assert bad["word"] == 2 and bool(torch.isnan(bad["logprob"][:2]).all()) and bool(torch.isfinite(bad["logprob"][2]))


def test_logprobs_captured_on_a_shared_workspace(B):
    ws = B.make_logprobs_workspace(4, 3)
    outs, graphs, ins = [], [], []
    for n, v in ((1, 100000), (4, 70000)):
        x = torch.randn(n, v, device="cuda")
        t = torch.zeros(n, dtype=torch.int32, device="cuda")
        o = [torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"),
             torch.zeros(n, 3, dtype=torch.int32, device="cuda"), torch.zeros(n, 3, device="cuda")]
        B.spark_token_logprobs(x, t, *o, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.spark_token_logprobs(x, t, *o, ws)
        outs.append(o), graphs.append(graph), ins.append((x, t))
    for k in range(3):
        for x, t in ins:
            x.normal_()
            t.fill_(k)
        graphs[k % 2].replay()
        graphs[(k + 1) % 2].replay()
        torch.cuda.synchronize()
        for (x, t), o in zip(ins, outs):
            _check_scores(dict(zip(("logprob", "entropy", "top_ids", "top_logprobs"), o)), x, t, 3)
    assert B.spark_attn_error_word(ws) == 0
