"""The paged cache's operators where their forms meet: pools around the sizes
at which a plan's shared memory needs more than the default, batches of more
sequences than a warp has lanes, sequences that no row of an append belongs
to, the block in a replayed graph.  References, bounds and their derivation:
``test_gpu_paged.py``."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from decode_attention_block_gb300 import synth
from test_gpu_paged import B, BF16, D, F32, SETS, Case, _check_attention, _geom, _i32, _pools, _run_remap, _scattered  # noqa: F401

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


# ---------------------------------------------------------------------------
# page plans
# ---------------------------------------------------------------------------

def _run_compact(B, table, page, n_pages):
    live = np.unique(table[table >= 0])
    m = len(live)
    src, dst = live[live >= m], np.setdiff1d(np.arange(m), live)
    to = np.arange(n_pages)
    to[src] = dst
    x, pools = _pools(B, 1, n_pages, page, 1, BF16, n_pages)
    after = x.clone()
    after[:, :, torch.tensor(dst, device="cuda")] = x[:, :, torch.tensor(src, device="cuda")]
    ws = B.make_pages_workspace(n_pages, len(table))
    out, n_live = _i32(table), torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spark_pages_compact(_geom(B, 1), pools, out, out, n_live, ws)
    assert B.spark_attn_error_word(ws) == 0 and int(n_live) == m
    assert np.array_equal(out.cpu().numpy(), np.where(table >= 0, to[table], -1))
    assert torch.equal(x, after)


def plans_of(sizes):
    """Remap and compact on pools of these sizes."""
    from decode_attention_block_gb300 import binding as B
    r = np.random.default_rng(7)
    for n_pages in sizes:
        lens = r.integers(0, 400, 20)
        table = _scattered(r, lens, 16, n_pages, 30)
        _run_remap(B, table, list(range(20)), lens.tolist(), (lens + 17).tolist(), 16, n_pages, layers=1, n_kv=1)
        _run_compact(B, table, 16, n_pages)


@pytest.mark.parametrize("sizes", [(4095, 4096, 4097), (5080, 5086, 5087, 5088, 5500), (6143, 6144, 6145)])
def test_plans_around_the_default_shared_memory(B, sizes):
    """In a process of their own: what one call raises for a kernel stays
    raised for the calls after it."""
    code = f"import sys; sys.path[:0] = [{HERE!r}, {os.path.dirname(HERE)!r}]; import test_gpu_paged_limits as t; t.plans_of({sizes!r})"
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]


def test_pages_kept_whole_and_in_part_at_once(B):
    """Every page of a sequence kept whole by some of 300 slots and in part by
    others: whole wins, whoever comes first."""
    page, n_pages, width = 16, 700, 12
    table = np.full((300, width), -1)
    table[17, :10] = np.random.default_rng(3).permutation(n_pages)[:10]
    keep = [(7 * s) % 160 + 1 for s in range(300)]
    for parents in ([17] * 300, [17 if s % 3 else -1 for s in range(300)]):
        kept = [k if p >= 0 else 0 for k, p in zip(keep, parents)]
        assert _run_remap(B, table, parents, kept, [k + 1 for k in kept], page, n_pages, layers=1, n_kv=1) == 0


# ---------------------------------------------------------------------------
# appends
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("start", [(0, 6, 4, 4), (0, 6, 6, 9), (0, 6, 6, 5), (0, 6, -1, -1), (0, 2, 6, 2**31 - 1)])
def test_append_reports_sequences_that_no_row_belongs_to(B, start):
    """Starts that decrease or pass the rows of the call are reported by the
    append too, where the search of no row ends in them."""
    case = Case([(100, 6), (40, 0), (50, 0)], page=16, seed=5)
    case.q_start = _i32(start)
    g, ws, pool = _geom(B), B.make_paged_workspace(_geom(B)), B.PagePool(case.k, case.v)
    kv = torch.ones(6, 1024, device="cuda")
    B.spark_paged_append(g, kv, kv, pool, case.batch(B, n_tokens=6, max_q=6), ws)
    assert B.spark_attn_error_word(ws) == 2
    case.q_start = _i32((0, 6, 6, 6))
    B.spark_paged_append(g, kv, kv, pool, case.batch(B, n_tokens=6, max_q=6), ws)
    assert B.spark_attn_error_word(ws) == 0


def test_append_reports_one_sequence_of_many(B):
    """1024 sequences, one of them with an end behind the rows of the call."""
    case = Case([(3, 1)] * 1024, n_kv=1, page=16, seed=5)
    g, ws, pool = _geom(B, 1), B.make_paged_workspace(_geom(B, 1)), B.PagePool(case.k, case.v)
    kv = torch.ones(1024, D, device="cuda")
    B.spark_paged_append(g, kv, kv, pool, case.batch(B), ws)
    assert B.spark_attn_error_word(ws) == 0
    case.q_start[1023:] = _i32([1024, 1025])          # the last but one takes the last row
    B.spark_paged_append(g, kv, kv, pool, case.batch(B, max_q=2), ws)
    assert B.spark_attn_error_word(ws) == 2


# ---------------------------------------------------------------------------
# more sequences than a warp has lanes
# ---------------------------------------------------------------------------

def _many(n, lo, hi, ctx, seed, long=0):
    """n sequences of lo .. hi new tokens at up to ctx positions, every seventh
    and the last two without new tokens, `long` of them ten times as long."""
    r = np.random.default_rng(seed)
    c, m = r.integers(1, ctx, n), r.integers(lo, hi + 1, n)
    c[r.permutation(n)[:long]] *= 10
    c = np.maximum(c, m)
    m[::7], m[-2:] = 0, 0
    return [(int(a), int(b)) for a, b in zip(c, m)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,n_kv,ctx,long", [(33, 4, 700, 3), (64, 1, 900, 5), (64, 4, 700, 3), (1024, 1, 90, 9),
                                             (1024, 4, 60, 0)])
def test_many_sequences_of_single_tokens(B, n, n_kv, ctx, long, dtype):
    seqs = _many(n, 1, 1, ctx, n + n_kv, long)
    _check_attention(B, Case(seqs, n_kv=n_kv, page=16, dtype=dtype, seed=n), F32)
    _check_attention(B, Case(seqs, n_kv=n_kv, page=48, dtype=dtype, seed=n), BF16, full=False, window=100)


@pytest.mark.parametrize("n,hi,n_kv,ctx", [(33, 20, 4, 500), (64, 9, 1, 900), (1024, 3, 1, 60)])
def test_many_sequences_on_an_f32_pool(B, n, hi, n_kv, ctx):
    seqs = _many(n, 2, hi, ctx, n, 2)
    _check_attention(B, Case(seqs, n_kv=n_kv, page=32, dtype=F32, seed=n, pad=3), F32)
    _check_attention(B, Case(seqs, n_kv=n_kv, page=16, dtype=F32, seed=n, pad=3), BF16, full=False, window=70)


@pytest.mark.parametrize("q_type", [F32, BF16])
@pytest.mark.parametrize("n,lo,hi,n_kv", [(33, 60, 90, 4), (40, 200, 300, 1), (130, 34, 40, 1)])
def test_many_long_chunks(B, n, lo, hi, n_kv, q_type):
    """Mostly long ones: pairs of CTAs."""
    seqs = _many(n, lo, hi, 600, n + lo, 1)
    case = Case(seqs, n_kv=n_kv, page=64, seed=n)
    assert 2 * case.n_tokens > n * case.max_q and case.max_q > 32
    _check_attention(B, case, q_type)
    _check_attention(B, Case(seqs, n_kv=n_kv, page=16, seed=n), q_type, full=False, window=130)


@pytest.mark.parametrize("q_type", [F32, BF16])
def test_results_repeat_bit_for_bit(B, q_type):
    """Whatever ran before, and beside them: every kernel, twenty times."""
    g, ws = _geom(B), B.make_paged_workspace(_geom(B))
    runs = []
    for name, dtype in (("decode", BF16), ("long", BF16), ("mixed", BF16), ("big_chunk", BF16), ("far", BF16),
                        ("edges", F32), ("decode", F32)):
        case = Case(SETS[name], page=64, seed=len(name), dtype=dtype)
        case.fill()
        q = torch.randn(case.n_tokens, 4096, generator=case.g, device="cuda").to(q_type)
        runs.append((q, B.PagePool(case.k, case.v), case.batch(B), torch.zeros_like(q), case))
    first = None
    r = np.random.default_rng(1)
    for _ in range(20):
        for i in r.permutation(len(runs)):
            q, pool, batch, a, _ = runs[i]
            B.spark_paged_attention(g, q, pool, B.SPARK_FULL, batch, a.fill_(7.0), ws)
        now = [a.clone() for _, _, _, a, _ in runs]
        first = first or now
        assert all(torch.equal(x, y) for x, y in zip(first, now))
    assert B.spark_attn_error_word(ws) == 0


# ---------------------------------------------------------------------------
# the block in a graph
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("is_full", [True, False])
def test_a_captured_block_replays_with_new_lengths_and_its_own_positions(B, is_full):
    """Tables, starts, lengths and rows are read at the replay, the rope
    positions are those of the capture."""
    geom = _geom(B, window=100)
    wl = synth.Workload("paged", "", "bf16", [50], [synth.LayerSpec(is_full, 0)], seed=80)
    lw = B.LayerWeights(**synth.make_weights(wl, 0, "cuda"))
    cls = B.SPARK_FULL if is_full else B.SPARK_SLIDING
    case = Case([(300, 5), (200, 3)], page=16, seed=21)
    for s, c in enumerate(case.ctx):        # every row: the replays end sequences elsewhere
        p, r = case.where(s)
        case.k[p, r], case.v[p, r] = case.rows_k[s], case.rows_v[s]
    k0, v0 = case.k.clone(), case.v.clone()
    ws, pws = B.make_workspace(geom, 8), B.make_paged_workspace(geom)
    pool, batch = B.PagePool(case.k, case.v), case.batch(B, max_q=8)
    h = torch.randn(8, 2560, generator=case.g, device="cuda")
    out, ref = torch.zeros_like(h), torch.zeros_like(h)
    positions = list(range(295, 300)) + list(range(197, 200))

    def call(to, pos):
        B.spark_attn_paged(geom, h, lw, pool, cls, batch, pos, to, ws, pws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out, positions)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, positions)
    for lens, new in (((300, 200), (5, 3)), ((130, 64), (1, 7)), ((299, 17), (8, 0))):
        case.seq_len.copy_(_i32(lens))
        case.q_start.copy_(_i32([0, new[0], sum(new)]))
        h.normal_(generator=case.g)
        got = []
        for replay in (True, False):
            case.k.copy_(k0), case.v.copy_(v0)
            graph.replay() if replay else call(ref, positions)
            torch.cuda.synchronize()
            got.append((case.k.clone(), case.v.clone()))
        iv = torch.int16
        assert torch.equal(out, ref)
        assert all(torch.equal(x.view(iv), y.view(iv)) for x, y in zip(*got))
    # other positions are another result: what a replay cannot take up
    call(ref, [p + 1 for p in positions])
    assert not torch.equal(out, ref)
    assert B.spark_attn_error_word(ws) == 0 and B.spark_attn_error_word(pws) == 0
