"""Pages held in 4 bits, and the append with the rotation on the way, against
plain implementations in 64 bits.

Rows: the codes and scales of an append are compared bit for bit with the
format's definition on the same fp32 numbers; a rotated key's are those of the
exact rotation rounded to fp32.  Other rotated elements are within 1.5 ulp of the
exact rotation in fp32 (Kahan's a c - b s with fma: w = b s rounded, e = w - b s
exact, f = a c - w rounded once, f + e rounded once; Jeannerod, Louvet and Muller
2013 prove 1.5 ulp, an ulp being at most 2^-23 of the value: 3 * 2^-24), then
rounded to their type (bf16 2^-8).

Attention over 4-bit pages, per element, with M the largest magnitude of a
token's and head's queries:
* a query, scaled so that M is in [1, 2), is two fp16 numbers (11 bits each,
  steps of 2^-24 at the least): off by 2^-22 |q| + 2^-25 M at most.  bf16 queries
  of chunks are one fp16 number: off by 2^-25 M.
* elements of K and V are fp16 numbers as they are, products exact, 256 (512) of
  them summed in fp32 (within 2^-15 of the sum of magnitudes):
  |ds| <= scale (sum |q k| (2^-22 + 2^-15) + 2^-25 M sum |k|).
* a probability e^(s - m): at most 2 |ds| relative (numerator and sum), 2^-17 for
  the exponential, its scaling to base 2 and the sums, and its rounding: two fp16
  numbers 2^-22, one (bf16 queries, chunks) 2^-11, and 2^-25 absolute, where the
  sum of the probabilities is at least 1.
* the output: fp32 sums (2^-15) and one rounding to its type.
"""

import numpy as np
import pytest
import torch

import fp4_ref
from decode_attention_block_gb300 import synth
from test_gpu_paged import B, BF16, D, F32, SETS, Case, _geom, _i32, _remap_oracle, _scattered  # noqa: F401

pytestmark = pytest.mark.gpu
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


class Fp4Case(Case):
    """As Case: blocks whose rows outside the sequences are 0xFF (NaN)."""

    def __init__(self, seqs, n_kv=4, page=16, seed=0, pad=0, spread=1.0):
        super().__init__(seqs, n_kv, page, BF16, seed, pad)
        shape = (self.k.shape[0], page // 16, n_kv, fp4_ref.BLOCK)
        self.k, self.v = (torch.full(shape, 0xFF, dtype=torch.uint8, device="cuda") for _ in "kv")
        self.code_k, self.code_v = [], []
        for rows, codes in ((self.rows_k, self.code_k), (self.rows_v, self.code_v)):
            for s, x in enumerate(rows):
                if spread != 1.0:  # groups of very different sizes
                    x = x.float() * spread ** torch.randn(x.shape[0], n_kv, 16, 1, generator=self.g, device="cuda").expand(
                        x.shape[0], n_kv, 16, 16).flatten(-2)
                codes.append(fp4_ref.quantize(x))
                rows[s] = fp4_ref.values(*codes[-1])

    def fill(self, window=0):
        for s, (c, n) in enumerate(self.seqs):
            lo = 0 if window == 0 or n == 0 else max(0, c - n + 1 - window)
            pos = torch.arange(lo, c, device="cuda")
            if len(pos):
                entries = torch.tensor(self.table_np[s], device="cuda")
                for pool, codes in ((self.k, self.code_k), (self.v, self.code_v)):
                    fp4_ref.write(pool, entries, self.page, pos, codes[s][0][lo:], codes[s][1][lo:])
            if lo >= self.page:
                self.table[s, : lo // self.page] = -1


def _reference(case, q, window, scale, q_type, single):
    n_kv = case.n_kv
    out, bound, t = [], [], 0
    for s, (c, n) in enumerate(case.seqs):
        if n == 0:
            continue
        k = case.rows_k[s].double().repeat_interleave(4, 1)
        v = case.rows_v[s].double().repeat_interleave(4, 1)
        qs = q[t:t + n].double().view(n, 4 * n_kv, D)
        pos, x = torch.arange(c - n, c, device="cuda")[:, None], torch.arange(c, device="cuda")[None]
        seen = x <= pos
        if window:
            seen &= x > pos - window
        sc = scale * torch.einsum("thd,xhd->htx", qs, k)
        ds = abs(scale) * (torch.einsum("thd,xhd->htx", qs.abs(), k.abs()) * (2.0 ** -22 + 2.0 ** -15) +
                           2.0 ** -25 * qs.abs().amax(-1).T[:, :, None] * k.abs().sum(-1).T[:, None])
        p = torch.softmax(sc.masked_fill(~seen, -np.inf), -1)
        o = torch.einsum("htx,xhd->thd", p, v)
        p_round = 2.0 ** -11 if q_type == BF16 and not single else 2.0 ** -22
        rel = 2 * ds.masked_fill(~seen, 0).amax(-1) + 2.0 ** -17 + p_round + 2.0 ** -15
        pv = torch.einsum("htx,xhd->thd", p, v.abs())
        out.append(o)
        bound.append(pv * rel.T[:, :, None] * 1.01 + 2.0 ** -25 * torch.einsum("tx,xhd->thd", seen.double(), v.abs()) +
                     U[q_type] * o.abs() + 1e-30)
        t += n
    return torch.cat(out), torch.cat(bound)


def _check(B, case, q_type=F32, full=True, window=512, scale=0.0625, max_q=None, q_pad=0, q_scale=None):
    g = _geom(B, case.n_kv, window, scale)
    case.fill(0 if full else window)
    width = 4 * case.n_kv * D
    q = torch.randn(case.n_tokens, width + q_pad, generator=case.g, device="cuda")
    if q_scale is not None:
        q *= q_scale
    q = q.to(q_type)[:, q_pad:]
    a = torch.full((case.n_tokens, width), 77.0, device="cuda", dtype=q_type)
    ws = B.make_paged_workspace(g)
    B.spark_paged_attention(g, q, B.PagePool(case.k, case.v), B.SPARK_FULL if full else B.SPARK_SLIDING,
                            case.batch(B, max_q=max_q), a, ws)
    torch.cuda.synchronize()
    assert B.spark_attn_error_word(ws) == 0
    used = sum(case.new)
    assert bool((a[used:] == 77.0).all()), "rows behind the last sequence were written"
    want, bound = _reference(case, q, 0 if full else window, scale, q_type, (max_q or case.max_q) == 1)
    err = (a[:used].double().view(want.shape) - want).abs()
    assert bool(torch.isfinite(err).all()), "non-finite output"
    worst = (err / bound).max().item()
    assert worst <= 1.0, f"error {worst:.2f} of its bound"
    return a


# ---------------------------------------------------------------------------
# rows into pages and out of them
# ---------------------------------------------------------------------------

def _special_rows(x):
    """Rows of zeros, of ties, tiny and huge ones, and ones with an infinity or a NaN."""
    n = len(x)
    if n < 9:
        return x
    x[0] = 0.0
    x[1] = 2.0 ** -30                                        # below half a step of the scales
    x[2] *= 2.0 ** -13                                       # scales in steps of 2^-17
    x[3] *= 5e4                                              # beyond the largest scale
    ties = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -0.0],
                        device=x.device)
    x[4] = (ties * 1.125).repeat(x.shape[1] // 16)           # scale 1.125: every quotient a border
    x[5] = (ties * 1.0625).repeat(x.shape[1] // 16)          # scale 1.0625: between two scales
    x[6, 3], x[6, 40] = float("inf"), float("nan")
    x[7] = -60000.0
    x[8] = 1e30
    return x


def _compare_rows(case, before, rows_k, rows_v):
    """Pools after an append of rows (fp32, as they are quantised): the groups' bytes, and all other bytes as before."""
    for pool, old, rows in ((case.k, before[0], rows_k), (case.v, before[1], rows_v)):
        rest, want = pool.clone(), old.clone()
        t = 0
        for s, (c, n) in enumerate(case.seqs):
            if n == 0:
                continue
            pos = torch.arange(c - n, c, device="cuda")
            entries = torch.tensor(case.table_np[s], device="cuda")
            code, scale = fp4_ref.quantize(rows[t:t + n].reshape(n, case.n_kv, D))
            got_code, got_scale = fp4_ref.read(pool, entries, case.page, pos, case.n_kv)
            assert torch.equal(got_scale, scale)
            fine = (scale != 0xFF).repeat_interleave(16, -1)
            assert torch.equal(got_code[fine], code[fine])
            for x in (rest, want):
                fp4_ref.write(x, entries, case.page, pos, torch.zeros_like(code), torch.zeros_like(scale))
            t += n
        assert torch.equal(rest, want), "other bytes were written"


@pytest.mark.parametrize("x_type", [BF16, F32])
@pytest.mark.parametrize("page,n_kv,name", [(16, 4, "mixed"), (48, 1, "verify"), (64, 8, "decode"), (1024, 3, "chunk_at")])
def test_append(B, page, n_kv, name, x_type):
    case = Fp4Case(SETS[name], n_kv=n_kv, page=page, seed=1, pad=5)
    g, row = _geom(B, n_kv), n_kv * D
    ws = B.make_paged_workspace(g)
    x = _special_rows(torch.randn(case.n_tokens, 3 * row, generator=case.g, device="cuda")).to(x_type)
    before = case.k.clone(), case.v.clone()
    B.spark_paged_append(g, x[:, row:2 * row], x[:, 2 * row:], B.PagePool(case.k, case.v), case.batch(B), ws)
    assert B.spark_attn_error_word(ws) == 0
    _compare_rows(case, before, x[:, row:2 * row], x[:, 2 * row:])


@pytest.mark.parametrize("layer", ["full", "sliding"])
def test_rope_table(B, layer):
    g = _geom(B)
    cls = B.SPARK_FULL if layer == "full" else B.SPARK_SLIDING
    for r in (64, 2, 62, 256):
        g.full_rotary_dim = r
        r = r if layer == "full" else 256
        theta = g.full_theta if layer == "full" else g.sliding_theta
        n = 70001
        rope = torch.full((n + 1, r // 2, 2), 9.0, device="cuda")
        B.spark_rope_table(g, cls, rope[:n])
        ang = torch.arange(n, dtype=torch.float64)[:, None] * theta ** (-2.0 * torch.arange(r // 2, dtype=torch.float64) / r)
        want = torch.stack([ang.cos(), ang.sin()], -1)
        # half an ulp of numbers up to 1, and angles off by a few 2^-53 of up to 70000
        assert ((rope[:n].cpu().double() - want).abs().max().item()) <= 2.0 ** -25 + 70000 * 2.0 ** -50
        assert bool((rope[n] == 9.0).all())


def _turned(x, cs):
    """Rows [n, heads, 256] in 64 bits, rotated by cs [n, r / 2, 2]."""
    x, c, s = x.double().clone(), cs[:, None, :, 0].double(), cs[:, None, :, 1].double()
    h = c.shape[-1]
    a, b = x[..., :h].clone(), x[..., h:2 * h].clone()
    x[..., :h], x[..., h:2 * h] = a * c - b * s, b * c + a * s
    return x


@pytest.mark.parametrize("pool", ["fp4", BF16, F32])
@pytest.mark.parametrize("x_type", [BF16, F32])
@pytest.mark.parametrize("name,page,n_kv,r,how", [
    ("mixed", 16, 4, 64, "out"), ("verify", 48, 1, 256, "in place"), ("decode", 64, 8, 2, "out"), ("one", 32, 4, 64, "in place"),
    ("chunk_at", 1024, 3, 62, "keys"), ("two", 16, 2, 100, "in place"), ("edges", 32, 5, 16, "out")])
def test_rope_append(B, name, page, n_kv, r, how, x_type, pool):
    if pool == "fp4":
        case = Fp4Case(SETS[name], n_kv=n_kv, page=page, seed=2, pad=3)
    else:
        case = Case(SETS[name], n_kv=n_kv, page=page, dtype=pool, seed=2, pad=3)
    g, row = _geom(B, n_kv), n_kv * D
    g.full_rotary_dim = r
    ws = B.make_paged_workspace(g)
    rope = torch.zeros(max(case.ctx), r // 2, 2, device="cuda")
    B.spark_rope_table(g, B.SPARK_FULL, rope)
    x = torch.randn(case.n_tokens, 6 * row + 8, generator=case.g, device="cuda").to(x_type)
    old = x.clone()
    q, k, v = x[:, :4 * row], x[:, 4 * row:5 * row], x[:, 5 * row:6 * row]
    q_out = {"out": torch.full_like(q, 5.0), "in place": q, "keys": None}[how]
    before = case.k.clone(), case.v.clone()
    B.spark_paged_rope_append(g, None if how == "keys" else q, k, v, B.SPARK_FULL, rope, B.PagePool(case.k, case.v),
                              case.batch(B), q_out, ws)
    assert B.spark_attn_error_word(ws) == 0
    used = sum(case.new)
    pos = torch.cat([torch.arange(c - n, c, device="cuda") for c, n in case.seqs])
    q0, k0, v0 = (t[:used].reshape(used, -1, D) for t in (old[:, :4 * row], old[:, 4 * row:5 * row], old[:, 5 * row:6 * row]))
    # what is not written is as it was
    assert torch.equal(x[:, 4 * row:], old[:, 4 * row:])
    if how != "in place":
        assert torch.equal(x, old)
    if how != "keys":
        want = _turned(q0, rope[pos])
        got = q_out[:used].double().view(want.shape)
        assert bool(((got - want).abs() <= (U[x_type] + 3 * 2.0 ** -24) * want.abs() * (1 + 2.0 ** -20) + 1e-40).all())
        assert torch.equal(q_out[used:], old[used:, :4 * row] if how == "in place" else torch.full_like(q_out[used:], 5.0))
    want = _turned(k0, rope[pos])
    if pool == "fp4":
        _compare_rows(case, before, want.float(), v0.float())
        return
    t = 0
    for s, (c, n) in enumerate(case.seqs):
        p, w = case.where(s)
        got = case.k[p[c - n:], w[c - n:]].double()
        assert bool(((got - want[t:t + n]).abs() <= (U[pool] + 3 * 2.0 ** -24) * want[t:t + n].abs() * (1 + 2.0 ** -20) + 1e-40).all())
        assert torch.equal(case.v[p[c - n:], w[c - n:]], v0[t:t + n].to(pool))
        case.k[p[c - n:], w[c - n:]] = before[0][p[c - n:], w[c - n:]]
        case.v[p[c - n:], w[c - n:]] = before[1][p[c - n:], w[c - n:]]
        t += n
    iv = torch.int16 if pool == BF16 else torch.int32
    assert torch.equal(case.k.view(iv), before[0].view(iv)) and torch.equal(case.v.view(iv), before[1].view(iv))


def test_rope_append_of_a_sliding_layer_and_short_tables(B):
    g = _geom(B)
    case = Fp4Case([(40, 3), (90, 2), (7, 7)], seed=3)
    rope = torch.zeros(90, 128, 2, device="cuda")
    B.spark_rope_table(g, B.SPARK_SLIDING, rope)
    ws, x = B.make_paged_workspace(g), torch.randn(12, 6144, generator=case.g, device="cuda")
    args = x[:, :4096], x[:, 4096:5120], x[:, 5120:], B.SPARK_SLIDING
    before, q_out = (case.k.clone(), case.v.clone()), torch.zeros(12, 4096, device="cuda")
    B.spark_paged_rope_append(g, *args, rope, B.PagePool(case.k, case.v), case.batch(B), q_out, ws)
    assert B.spark_attn_error_word(ws) == 0
    pos = torch.tensor([37, 38, 39, 88, 89, 0, 1, 2, 3, 4, 5, 6], device="cuda")
    _compare_rows(case, before, _turned(args[1].reshape(12, 4, D), rope[pos]).float(), args[2].float())
    # positions behind the table: reported and left out
    case.k.copy_(before[0])
    case.v.copy_(before[1])
    q_out.fill_(3.0)
    B.spark_paged_rope_append(g, *args, rope[:89], B.PagePool(case.k, case.v), case.batch(B), q_out, ws)
    assert B.spark_attn_error_word(ws) == 2
    assert bool((q_out[4] == 3.0).all()) and not bool((q_out[3] == 3.0).any())
    code, _ = fp4_ref.read(case.k, case.table[1], 16, torch.tensor([89], device="cuda"), 4)
    assert bool((code == 15).all())


@pytest.mark.parametrize("pool", ["fp4", BF16, F32])
@pytest.mark.parametrize("x_type", [BF16, F32])
@pytest.mark.parametrize("name,page,n_kv", [("mixed", 16, 4), ("verify", 48, 1), ("decode", 64, 8), ("chunk_at", 1024, 3)])
def test_read(B, name, page, n_kv, x_type, pool):
    case = (Fp4Case(SETS[name], n_kv=n_kv, page=page, seed=4, pad=6) if pool == "fp4" else
            Case(SETS[name], n_kv=n_kv, page=page, dtype=pool, seed=4, pad=6))
    case.fill()
    g = _geom(B, n_kv)
    ws = B.make_paged_workspace(g)
    x = torch.full((case.n_tokens, 2 * n_kv * D + 8), 3.0, device="cuda", dtype=x_type)
    k, v = x[:, :n_kv * D], x[:, n_kv * D:2 * n_kv * D]
    B.spark_paged_read(g, B.PagePool(case.k, case.v), case.batch(B), k, v, ws)
    assert B.spark_attn_error_word(ws) == 0
    used = sum(case.new)
    for got, rows in ((k, case.rows_k), (v, case.rows_v)):
        want = torch.cat([r[c - n:] for r, (c, n) in zip(rows, case.seqs)]).reshape(used, -1)
        assert torch.equal(got[:used], want.to(x_type))
    assert bool((x[used:] == 3.0).all()) and bool((x[:, 2 * n_kv * D:] == 3.0).all())


@pytest.mark.parametrize("x_type", [BF16, F32])
@pytest.mark.parametrize("n_kv,page,most", [(1, 16, 70), (3, 48, 70), (4, 16, 9000), (8, 64, 70)])
def test_long_reads(B, n_kv, page, most, x_type):
    """As many tokens as a long prompt's, of a few long sequences or of many short ones, the empty among them."""
    rng = np.random.default_rng(n_kv)
    seqs, tokens = [], 0
    while tokens < 9100:
        n = int(rng.integers(0, most + 1)) if most < 9000 else (9000, 0, 7, 400)[len(seqs) % 4]
        seqs.append((n + int(rng.integers(0, 40)), n))
        tokens += n
    case = Fp4Case(seqs, n_kv=n_kv, page=page, seed=5, pad=37)
    case.fill()
    g = _geom(B, n_kv)
    ws = B.make_paged_workspace(g)
    k, v = (torch.full((case.n_tokens, n_kv * D), 3.0, device="cuda", dtype=x_type) for _ in "kv")
    B.spark_paged_read(g, B.PagePool(case.k, case.v), case.batch(B), k, v, ws)
    assert B.spark_attn_error_word(ws) == 0
    used = sum(case.new)
    want = [torch.cat([r[c - n:] for r, (c, n) in zip(rows, case.seqs)]).reshape(used, -1).to(x_type)
            for rows in (case.rows_k, case.rows_v)]
    for got, w in zip((k, v), want):
        assert torch.equal(got[:used], w) and bool((got[used:] == 3.0).all())
    # an entry outside the pool: its rows are left out, and no others
    s = max(range(len(seqs)), key=lambda i: seqs[i][1])
    c, n = seqs[s]
    col = (c - 1) // page
    case.table[s, col] = case.k.shape[0]
    k.fill_(3.0), v.fill_(3.0)
    B.spark_paged_read(g, B.PagePool(case.k, case.v), case.batch(B), k, v, ws)
    assert B.spark_attn_error_word(ws) == 2
    lost = torch.zeros(case.n_tokens, dtype=torch.bool, device="cuda")
    at = sum(m for _, m in seqs[:s]) + torch.arange(n, device="cuda")
    lost[at[torch.arange(c - n, c, device="cuda") >= col * page]] = True
    assert bool(lost.any())
    for got, w in zip((k, v), want):
        assert bool((got[lost] == 3.0).all()) and torch.equal(got[:used][~lost[:used]], w[~lost[:used]])


def test_bad_entries_of_row_calls(B):
    """Reported, never followed; the other sequences' rows are written."""
    g = _geom(B)
    ws, rope = B.make_paged_workspace(g), torch.zeros(200, 32, 2, device="cuda")
    B.spark_rope_table(g, B.SPARK_FULL, rope)
    for at, val in ((("table", (0, 6)), -1), (("table", (0, 6)), 2 ** 31 - 1), (("table", (1, 2)), -5), (("seq_len", 0), 2),
                    (("seq_len", 1), -4), (("seq_len", 2), 2 ** 31 - 1), (("q_start", 1), -3), (("q_start", 3), 7),
                    (("q_start", 2), 1)):
        for pool in ("fp4", BF16):
            seqs = [(100, 3), (40, 2), (50, 1)]
            case = Fp4Case(seqs, seed=5) if pool == "fp4" else Case(seqs, seed=5)
            case.fill()
            getattr(case, at[0])[at[1]] = val
            x, out = torch.randn(6, 6144, device="cuda"), torch.zeros(6, 4096, device="cuda")
            b = case.batch(B, n_tokens=6, max_q=3)
            pages = B.PagePool(case.k, case.v)
            B.spark_paged_read(g, pages, b, out[:, :1024], out[:, 1024:2048], ws)
            assert B.spark_attn_error_word(ws) == 2
            B.spark_paged_rope_append(g, x[:, :4096], x[:, 4096:5120], x[:, 5120:], B.SPARK_FULL, rope, pages, b, out, ws)
            assert B.spark_attn_error_word(ws) == 2


def test_captured_append_and_attention_replay_for_the_next_token(B):
    """Lengths on the device: one graph, a token more at every replay."""
    g = _geom(B)
    case = Fp4Case([(61, 1), (16, 1), (130, 1)], page=32, seed=6)
    case.fill()
    rope = torch.zeros(160, 32, 2, device="cuda")
    B.spark_rope_table(g, B.SPARK_FULL, rope)
    pool, ws, batch = B.PagePool(case.k, case.v), B.make_paged_workspace(g), case.batch(B)
    x, a = torch.randn(3, 6144, generator=case.g, device="cuda"), torch.zeros(3, 4096, device="cuda")
    q = torch.zeros_like(a)

    def step():
        B.spark_paged_rope_append(g, x[:, :4096], x[:, 4096:5120], x[:, 5120:], B.SPARK_FULL, rope, pool, batch, q, ws)
        B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, a, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.normal_(generator=case.g)
        case.seq_len.copy_(_i32([61 + i, 16 + i, 130 + i]))
        graph.replay()
        torch.cuda.synchronize()
        k, v, b = case.k.clone(), case.v.clone(), a.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.equal(k, case.k) and torch.equal(v, case.v)
        for s, n in enumerate([61 + i, 16 + i, 130 + i]):
            case.rows_k[s], case.rows_v[s] = (fp4_ref.values(*fp4_ref.read(pl, case.table[s], 32, torch.arange(n, device="cuda"), 4))
                                              for pl in (case.k, case.v))
        now = type("Now", (), dict(seqs=[(61 + i, 1), (16 + i, 1), (130 + i, 1)], n_kv=4, rows_k=case.rows_k, rows_v=case.rows_v))
        want, bound = _reference(now, q, 0, 0.0625, F32, True)
        assert bool(((a.double().view(want.shape) - want).abs() <= bound).all())
    assert B.spark_attn_error_word(ws) == 0


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("q_type", [F32, BF16])
@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("name", list(SETS))
def test_attention(B, name, full, q_type):
    _check(B, Fp4Case(SETS[name], page=64, seed=len(name)), q_type, full, window=512 if name != "mixed" else 100)


@pytest.mark.parametrize("page", [16, 32, 48, 80, 128, 256, 1024])
@pytest.mark.parametrize("name", ["decode", "mixed", "pairs"])
def test_page_sizes(B, page, name):
    _check(B, Fp4Case(SETS[name], page=page, seed=page), BF16)
    _check(B, Fp4Case(SETS[name], page=page, seed=page + 1), F32, full=False, window=130)


@pytest.mark.parametrize("n_kv", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("name", ["decode", "mixed", "pairs"])
def test_head_counts(B, n_kv, name):
    _check(B, Fp4Case(SETS[name], n_kv=n_kv, page=32, seed=n_kv), BF16)
    _check(B, Fp4Case(SETS[name], n_kv=n_kv, page=32, seed=n_kv), F32)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 127, 128, 129, 100000])
@pytest.mark.parametrize("q_type", [F32, BF16])
@pytest.mark.parametrize("name", ["decode", "mixed", "pairs"])
def test_windows(B, name, window, q_type):
    _check(B, Fp4Case(SETS[name], page=16, seed=window), q_type, full=False, window=window)
    _check(B, Fp4Case(SETS[name], page=128, seed=window), q_type, full=False, window=window)


@pytest.mark.parametrize("scale", [0.0, 0.01, 0.25, -0.0625])
@pytest.mark.parametrize("name", ["decode", "mixed", "pairs"])
def test_scales(B, name, scale):
    _check(B, Fp4Case(SETS[name], page=64, seed=9), F32, scale=scale)
    _check(B, Fp4Case(SETS[name], page=64, seed=9), BF16, scale=scale)


@pytest.mark.parametrize("q_type", [F32, BF16])
@pytest.mark.parametrize("name", ["decode", "mixed", "pairs"])
def test_groups_and_queries_of_all_sizes(B, name, q_type):
    _check(B, Fp4Case(SETS[name], page=64, seed=10, spread=2.0), q_type)
    for q_scale, scale in ((1e-30, 0.0625), (0.0, 0.0625), (1e20, 0.0625e-20), (3e-5, 2000.0)):
        _check(B, Fp4Case(SETS[name], page=64, seed=11), q_type, scale=scale, q_scale=q_scale)


@pytest.mark.parametrize("q_type", [F32, BF16])
def test_strided_queries_and_padded_rows(B, q_type):
    _check(B, Fp4Case(SETS["mixed"], page=64, seed=4, pad=37), q_type, q_pad=2048 + 8, max_q=200)
    _check(B, Fp4Case(SETS["pairs"], page=64, seed=4, pad=37), q_type, q_pad=2048 + 8)
    _check(B, Fp4Case(SETS["decode"], page=64, seed=4, pad=37), q_type, q_pad=2048 + 8)


def test_many_sequences(B):
    r = np.random.default_rng(2)
    seqs = [(int(c), int(min(c, n))) for c, n in zip(r.integers(0, 90, 1024), r.integers(0, 3, 1024))]
    _check(B, Fp4Case(seqs, n_kv=1, seed=6), F32)
    _check(B, Fp4Case(seqs, n_kv=1, seed=6), BF16, full=False, window=20)
    _check(B, Fp4Case([(c, min(1, n)) for c, n in seqs], n_kv=1, seed=6), F32)


@pytest.mark.parametrize("max_q", [1, 20, 64])
def test_nothing_to_do(B, max_q):
    case = Fp4Case([(40, 0), (0, 0)], seed=3, pad=70)
    g, q = _geom(B), torch.randn(70, 4096, device="cuda")
    a, ws = torch.full_like(q, 5.0), B.make_paged_workspace(_geom(B))
    batch, pool, k0 = case.batch(B, max_q=max_q), B.PagePool(case.k, case.v), case.k.clone()
    B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, a, ws)
    B.spark_paged_append(g, q[:, :1024], q[:, 1024:2048], pool, batch, ws)
    B.spark_paged_read(g, pool, batch, a[:, :1024], a[:, 1024:2048], ws)
    assert B.spark_attn_error_word(ws) == 0 and bool((a == 5.0).all()) and torch.equal(case.k, k0)


@pytest.mark.parametrize("q_type", [F32, BF16])
@pytest.mark.parametrize("name", ["decode", "verify", "mixed", "edges", "pairs"])
def test_queries_of_other_sequences_do_not_matter(B, name, q_type):
    case = Fp4Case(SETS[name], page=32, seed=12, pad=29)
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


def test_large_scores_and_one_dominant_row(B):
    for q_type in (F32, BF16):
        for seqs in ([(900, 1), (700, 200)], [(900, 1), (333, 1)]):
            case = Fp4Case(seqs, page=64, seed=8)
            for s in range(2):
                ramp = torch.linspace(0.1, 6.0, case.ctx[s], device="cuda")[:, None, None]
                case.code_k[s] = fp4_ref.quantize(case.rows_k[s] * ramp)
                case.rows_k[s] = fp4_ref.values(*case.code_k[s])
            g = _geom(B)
            case.fill()
            q = (torch.randn(case.n_tokens, 4096, generator=case.g, device="cuda") * 5).to(q_type)
            a, ws = torch.zeros_like(q), B.make_paged_workspace(g)
            B.spark_paged_attention(g, q, B.PagePool(case.k, case.v), B.SPARK_FULL, case.batch(B), a, ws)
            assert B.spark_attn_error_word(ws) == 0
            want, bound = _reference(case, q, 0, 0.0625, q_type, case.max_q == 1)
            # scores of up to 2^9 or so: their scaling to base 2 alone is off by 2^-24 * 2^9 * 2 ln 2
            err = (a.double().view(want.shape) - want).abs() / (bound + 2.0 ** -14 * want.abs().amax())
            assert err.max().item() <= 1.0


@pytest.mark.parametrize("n_seqs, n, c, q_type", [(480, 1, 400000, F32), (160, 8, 50000, F32), (80, 40, 50000, F32),
                                                  (160, 8, 50000, BF16), (80, 40, 50000, BF16)])
def test_long_sums_keep_their_bits(B, n_seqs, n, c, q_type):
    """Sums of positive values over a whole long sequence per share: what the matrix instructions cut off (up to 2^-23 of
    the sum a step, towards zero) may come to 2^-15 of it for fp32 queries, 2^-14 for bf16 ones, whatever the length.
    Scores are tiny (2 |ds| below 2^-20), probabilities as above (the sum of a row's rounded to nearest: sqrt(12500) 2^-24
    is within the 2^-17)."""
    g, gen = _geom(B, 1, 512, 0.0625), torch.Generator("cuda").manual_seed(5)
    page = 256
    entries = torch.randperm(-(-c // page), generator=gen, device="cuda").int()
    pools, vals = [], []
    for make in (torch.randn, torch.rand):
        code, sc = fp4_ref.quantize(make(c, 1, D, generator=gen, device="cuda"))
        pool = torch.full((len(entries), page // 16, 1, fp4_ref.BLOCK), 0xFF, dtype=torch.uint8, device="cuda")
        fp4_ref.write(pool, entries, page, torch.arange(c, device="cuda"), code, sc)
        pools.append(pool)
        vals.append(fp4_ref.values(code, sc)[:, 0])
        del code, sc
    some = 3  # sequences with queries of their own, all of the same pages
    q3 = (torch.randn(some, n, 4, D, generator=gen, device="cuda") * 2.0 ** -10).to(q_type)
    q = q3[torch.arange(n_seqs, device="cuda") % some].reshape(n_seqs * n, 4 * D)
    batch = B.PagedBatch(entries.repeat(n_seqs, 1).contiguous(), _i32([n * i for i in range(n_seqs + 1)]), _i32([c] * n_seqs), n_seqs * n, n)
    a, ws = torch.zeros(n_seqs * n, 4 * D, device="cuda", dtype=q_type), B.make_paged_workspace(g)
    B.spark_paged_attention(g, q, B.PagePool(*pools), B.SPARK_FULL, batch, a, ws)
    torch.cuda.synchronize()
    assert B.spark_attn_error_word(ws) == 0
    z = 0.0625 * torch.einsum("sthd,xd->sthx", q3.double(), vals[0])
    late = torch.arange(c, device="cuda")[None] > torch.arange(c - n, c, device="cuda")[:, None]
    want = torch.softmax(z.masked_fill(late[None, :, None], -np.inf), -1) @ vals[1]
    rel = 2.0 ** -20 + 2.0 ** -17 + (2.0 ** -22 + 2.0 ** -15 if q_type == F32 else 2.0 ** -11 + 2.0 ** -14 + 2.0 ** -8)
    want = want[torch.arange(n_seqs, device="cuda") % some]
    err = (a.double().view(n_seqs, n, 4, D) - want).abs()
    worst = (err / want).max().item()
    assert worst <= rel, f"{worst:.2g} of the output, bound {rel:.2g}"


@pytest.mark.parametrize("n_seqs, n, c, q_type", [(480, 1, 40000, F32), (480, 1, 40000, BF16), (160, 8, 12000, F32), (80, 40, 12000, F32),
                                                  (160, 8, 30000, BF16), (80, 40, 30000, BF16)])
@pytest.mark.parametrize("rising", [True, False])
def test_long_sums_under_maxima_that_move(B, n_seqs, n, c, q_type, rising):
    """Scores that rise by some 24 over a third of a long sequence and stay there, or stay and fall: sums put aside under an
    earlier maximum count for less, or for all."""
    g, gen = _geom(B, 1, 512, 0.0625), torch.Generator("cuda").manual_seed(6)
    page = 128
    entries = torch.randperm(-(-c // page), generator=gen, device="cuda").int()
    x = torch.arange(c, device="cuda", dtype=torch.float32)
    ramp = (3.0 * x / c).clamp(max=1.0)
    ramp = ramp if rising else ramp.flip(0)
    way = torch.randn(D, generator=gen, device="cuda").sign()
    keys = (way * ramp[:, None] + 0.05 * torch.randn(c, D, generator=gen, device="cuda"))[:, None]
    pools, vals = [], []
    for rows in (keys, torch.rand(c, 1, D, generator=gen, device="cuda")):
        code, sc = fp4_ref.quantize(rows)
        pool = torch.full((len(entries), page // 16, 1, fp4_ref.BLOCK), 0xFF, dtype=torch.uint8, device="cuda")
        fp4_ref.write(pool, entries, page, torch.arange(c, device="cuda"), code, sc)
        pools.append(pool)
        vals.append(fp4_ref.values(code, sc)[:, 0])
    q = (1.5 * way + 0.1 * torch.randn(n * 4, D, generator=gen, device="cuda")).to(q_type).reshape(n, 4 * D)
    batch = B.PagedBatch(entries.repeat(n_seqs, 1).contiguous(), _i32([n * i for i in range(n_seqs + 1)]), _i32([c] * n_seqs), n_seqs * n, n)
    a, ws = torch.zeros(n_seqs * n, 4 * D, device="cuda", dtype=q_type), B.make_paged_workspace(g)
    B.spark_paged_attention(g, q.repeat(n_seqs, 1), B.PagePool(*pools), B.SPARK_FULL, batch, a, ws)
    torch.cuda.synchronize()
    assert B.spark_attn_error_word(ws) == 0
    qd = q.double().view(n, 4, D)
    z = 0.0625 * torch.einsum("thd,xd->thx", qd, vals[0])
    late = torch.arange(c, device="cuda")[None] > torch.arange(c - n, c, device="cuda")[:, None]
    want = torch.softmax(z.masked_fill(late[:, None], -np.inf), -1) @ vals[1]
    ds = 0.0625 * (torch.einsum("thd,xd->thx", qd.abs(), vals[0].abs()) * (2.0 ** -22 + 2.0 ** -15) +
                   2.0 ** -25 * qd.abs().amax(-1, keepdim=True) * vals[0].abs().sum(-1)).amax(-1, keepdim=True)
    rel = 2 * ds + 2.0 ** -17 + (2.0 ** -22 + 2.0 ** -15 if q_type == F32 else 2.0 ** -11 + 2.0 ** -14 + 2.0 ** -8)
    err = ((a.double().view(n_seqs, n, 4, D) - want).abs() / want - 2.0 ** -25 * vals[1].sum(0) / want).clamp(min=0)
    worst = (err / rel).max().item()
    assert worst <= 1.0, f"error {worst:.2f} of its bound"


def test_repeated_and_unordered_calls_agree(B):
    g = _geom(B)
    ws, runs = B.make_paged_workspace(g), []
    for name in ("decode", "big_chunk", "mixed", "long", "pairs"):
        case = Fp4Case(SETS[name], page=64, seed=1)
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


def test_calls_at_once_on_their_own_workspaces(B):
    g, runs = _geom(B), []
    for i, (name, q_type) in enumerate((("decode", F32), ("mixed", F32), ("pairs", BF16), ("big_chunk", F32), ("long", BF16))):
        case = Fp4Case(SETS[name], page=(16, 64)[i % 2], seed=20 + i)
        case.fill()
        q = torch.randn(case.n_tokens, 4096, generator=case.g, device="cuda").to(q_type)
        runs.append((q, B.PagePool(case.k, case.v), case.batch(B), torch.zeros_like(q), torch.zeros_like(q),
                     B.make_paged_workspace(g), torch.cuda.Stream(), case))
    for q, pool, batch, want, _, ws, _, _ in runs:
        B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, want, ws)
    torch.cuda.synchronize()
    for _ in range(5):
        for q, pool, batch, _, got, ws, st, _ in runs:
            B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, got, ws, stream=st)
    torch.cuda.synchronize()
    for _, _, _, want, got, ws, _, _ in runs:
        assert B.spark_attn_error_word(ws) == 0 and torch.equal(want, got)


@pytest.mark.parametrize("q_type", [F32, BF16])
@pytest.mark.parametrize("new", [(1, 1), (4, 2), (90, 70)])
def test_bad_pages(B, new, q_type):
    """Entries outside the pool: reported, and the other sequence's results are what they were."""
    case = Fp4Case([(200, new[0]), (130, new[1])], page=16, seed=15)
    case.fill()
    g, ws, pool = _geom(B), B.make_paged_workspace(_geom(B)), B.PagePool(case.k, case.v)
    q = torch.randn(sum(new), 4096, generator=case.g, device="cuda").to(q_type)
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    B.spark_paged_attention(g, q, pool, B.SPARK_FULL, case.batch(B), a, ws)
    assert B.spark_attn_error_word(ws) == 0
    keep = case.table.clone()
    for entry in (-1, case.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        case.table.copy_(keep)
        case.table[0, 1] = entry
        b.zero_()
        B.spark_paged_attention(g, q, pool, B.SPARK_FULL, case.batch(B), b, ws)
        assert B.spark_attn_error_word(ws) == 2
        assert torch.equal(a[new[0]:], b[new[0]:])


@pytest.mark.parametrize("q_type", [F32, BF16])
@pytest.mark.parametrize("seqs", [[(300, 130), (200, 70)], [(200, 1), (90, 1)], [(200, 5), (90, 3)]])
def test_captured_calls_replay_with_new_lengths(B, seqs, q_type):
    g = _geom(B)
    case = Fp4Case(seqs, seed=16)
    case.fill()
    pool, ws = B.PagePool(case.k, case.v), B.make_paged_workspace(g)
    q = torch.randn(case.n_tokens, 4096, generator=case.g, device="cuda").to(q_type)
    a, b, batch = torch.zeros_like(q), torch.zeros_like(q), case.batch(B)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, a, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, a, ws)
    for cut in (0, 3, 40):
        lens = [c - cut for c, _ in seqs]
        new = [max(0, n - cut) if n > 1 else n for _, n in seqs]
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


def test_pages_far_into_a_pool(B):
    """Byte offsets beyond 2^32 in the append, the read, attention and a fork's copies."""
    page, n_kv, n_pages = 1024, 8, 4000                       # 1.2 MB a page: 4.7 GB of K and of V
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("needs 14 GB")
    k = torch.empty(n_pages, page // 16, n_kv, fp4_ref.BLOCK, device="cuda", dtype=torch.uint8)
    v = torch.empty_like(k)
    pool, g = B.PagePool(k, v), _geom(B, n_kv)
    ws, gen = B.make_paged_workspace(g), torch.Generator(device="cuda").manual_seed(1)
    table, start, lens = _i32([[3999, -1], [3900, 3998]]), _i32([0, 70, 110]), _i32([70, 1100])
    x = torch.randn(1060, 2 * n_kv * D, generator=gen, device="cuda")
    B.spark_paged_append(g, x[:, :n_kv * D], x[:, n_kv * D:], pool, B.PagedBatch(table[1:], _i32([0, 1060]), _i32([1060]), 1060, 1060), ws)
    y = torch.randn(110, 2 * n_kv * D, generator=gen, device="cuda")
    batch = B.PagedBatch(table, start, lens, 110, 70)
    B.spark_paged_append(g, y[:, :n_kv * D], y[:, n_kv * D:], pool, batch, ws)
    rows = [y[:70], torch.cat([x, y[70:]])]
    case = type("Rows", (), dict(seqs=[(70, 70), (1100, 40)], n_kv=n_kv))
    case.rows_k, case.rows_v = ([fp4_ref.values(*fp4_ref.quantize(r[:, i * n_kv * D:(i + 1) * n_kv * D].reshape(-1, n_kv, D)))
                                 for r in rows] for i in (0, 1))
    got_k, got_v = torch.zeros(110, n_kv * D, device="cuda"), torch.zeros(110, n_kv * D, device="cuda")
    B.spark_paged_read(g, pool, batch, got_k, got_v, ws)
    assert torch.equal(got_k[70:].double(), case.rows_k[1][1060:].flatten(1)) and torch.equal(got_v[:70].double(), case.rows_v[0].flatten(1))
    q = torch.randn(110, 4 * n_kv * D, generator=gen, device="cuda")
    a = torch.zeros_like(q)
    B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, a, ws)
    want, bound = _reference(case, q, 0, 0.0625, F32, False)
    assert ((a.double().view(want.shape) - want).abs() / bound).max().item() <= 1.0
    one = torch.zeros(1, 4 * n_kv * D, device="cuda")
    B.spark_paged_attention(g, q[109:], pool, B.SPARK_FULL, B.PagedBatch(table[1:], _i32([0, 1]), _i32([1100]), 1, 1), one, ws)
    assert ((one.double().view(1, -1, D) - want[109:]).abs() / bound[109:]).max().item() <= 1.0
    assert B.spark_attn_error_word(ws) == 0
    tws, new = B.make_pages_workspace(n_pages, 2), torch.zeros_like(table)
    B.spark_pages_remap(g, [pool], table, _i32([0, 0]), _i32([70, 70]), _i32([70, 70]), new, tws)
    assert B.spark_attn_error_word(tws) == 0 and new.tolist() == [[3999, -1], [0, -1]]
    assert torch.equal(k[0, :5], k[3999, :5]) and torch.equal(v[0, :5], v[3999, :5])


# ---------------------------------------------------------------------------
# page tables and the block
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("page", [16, 48])
def test_remap_and_compact(B, seed, page):
    """What every slot keeps reads as it did, in every layer."""
    r = np.random.default_rng(seed)
    n, n_kv, layers = int(r.integers(1, 30)), 3, 2
    lens = r.integers(1, 8 * page, n)
    n_pages = int(sum(-(-lens // page)) + 4 * n + 2)
    table = _scattered(r, lens, page, n_pages, 12)
    parent = r.integers(-1, n, n)
    keep = np.array([0 if p < 0 else r.integers(0, lens[p] + 1) for p in parent])
    new = keep + r.integers(0, 2 * page, n)
    g = _geom(B, n_kv)
    x = torch.randint(0, 256, (layers, 2, n_pages, page // 16, n_kv, fp4_ref.BLOCK), device="cuda", dtype=torch.uint8)
    pools, before = [B.PagePool(p[0], p[1]) for p in x], x.clone()
    ws, out = B.make_pages_workspace(n_pages, n), torch.full(table.shape, -99, dtype=torch.int32, device="cuda")
    B.spark_pages_remap(g, pools, _i32(table), _i32(parent), _i32(keep), _i32(new), out, ws)
    want = _remap_oracle(table, parent, keep, new, page, n_pages)
    assert B.spark_attn_error_word(ws) == 0 and np.array_equal(out.cpu().numpy(), want[0])

    def kept(pools_now, tables, slot, m):
        pos = torch.arange(m, device="cuda")
        return [torch.cat([t.flatten() for t in fp4_ref.read(pools_now[i, j], tables[slot], page, pos, n_kv)])
                for i in range(layers) for j in (0, 1)]
    old = torch.tensor(table, device="cuda")
    for s in range(n):
        if keep[s]:
            for a, b in zip(kept(x, out.long(), s, int(keep[s])), kept(before, old, int(parent[s]), int(keep[s]))):
                assert torch.equal(a, b)
    # and all pages in use to the front
    had, n_live = x.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    packed = torch.zeros_like(out)
    B.spark_pages_compact(g, pools, out, packed, n_live, ws)
    assert B.spark_attn_error_word(ws) == 0
    used = set(out[out >= 0].tolist())
    assert int(n_live) == len(used) and set(packed[packed >= 0].tolist()) == set(range(len(used)))
    for a, b in zip(packed[packed >= 0].tolist(), out[out >= 0].tolist()):
        assert torch.equal(x[:, :, a], had[:, :, b])


@pytest.mark.parametrize("name", ["decode", "mixed"])
@pytest.mark.parametrize("full", [True, False])
def test_block_on_4_bit_pages(B, name, full):
    """The block against its stages: the fused projection's k and v rows in 4
    bits, attention over the pages, gate and o_proj."""
    g = _geom(B)
    cls = B.SPARK_FULL if full else B.SPARK_SLIDING
    wl = synth.Workload("fp4", "", "bf16", [1], [synth.LayerSpec(full, 0 if full else 512)], seed=3)
    w = B.LayerWeights(**synth.make_weights(wl, 0, "cuda"))
    case = Fp4Case(SETS[name], page=32, seed=5)
    case.fill()
    n = case.n_tokens
    positions = [p for c, m in case.seqs for p in range(c - m, c)]
    h = torch.randn(n, g.hidden, generator=case.g, device="cuda")
    ws, pws = B.make_workspace(g, n), B.make_paged_workspace(g)
    # the stages, on copies of the pages
    pool2 = B.PagePool(case.k.clone(), case.v.clone())
    rows = [torch.zeros(n, 1, 4, D, device="cuda") for _ in "kv"]
    q, gl, a, want = (torch.zeros(n, m, device="cuda") for m in (4096, 16, 4096, g.hidden))
    staged = B.KvLayer(*(torch.zeros(n, 1024, 4, D, device="cuda") for _ in "kv"), 0) if n <= 8 else None
    out = torch.zeros_like(h)
    B.spark_attn_paged(g, h, w, B.PagePool(case.k, case.v), cls, case.batch(B), positions, out, ws, pws)
    assert B.spark_attn_error_word(ws) == 0 and B.spark_attn_error_word(pws) == 0
    # k and v of the fused projection from the same call on an fp32 pool
    f32 = Case(SETS[name], page=32, dtype=F32, seed=5)
    f32.k.zero_()
    f32.v.zero_()
    scratch = torch.zeros_like(h)
    B.spark_attn_paged(g, h, w, B.PagePool(f32.k, f32.v), cls, f32.batch(B), positions, scratch, ws, pws)
    B.spark_paged_read(g, B.PagePool(f32.k, f32.v), f32.batch(B), rows[0].view(n, -1), rows[1].view(n, -1), pws)
    B.spark_paged_append(g, rows[0].view(n, -1), rows[1].view(n, -1), pool2, case.batch(B), pws)
    assert torch.equal(pool2.k, case.k) and torch.equal(pool2.v, case.v)
    if staged is not None:  # q and the gate by their own entry point
        B.spark_dbg_qkv_rope(g, h, w, staged, cls, positions, q, gl, ws)
        B.spark_paged_attention(g, q, pool2, cls, case.batch(B), a, pws)
        B.spark_dbg_gate_oproj(g, a, gl, h, w, want, ws)
        assert torch.equal(out, want)
    assert bool(torch.isfinite(out).all())
