"""Beam search's selection and reordering against plain implementations, and
steps of it together with 4-bit pages.

A score is compared within 2^-24 of itself (its rounding to fp32) and 2^-18 for
the log of the sum: a thread adds up to 32 tiles of 16 exponentials of 131072
logits (40 roundings of 2^-24), an exponential is off by 2^-22 and its argument,
up to 30 where it counts, by 30 * 2^-24.  Where offers of two beams are nearer than
twice that, either order is right: also where the oracle has them equal, if their
rows are other sequences of logits (the same numbers in another order are summed
in another order, each sum within its own error of the oracle's).  Offers of one
beam, and of beams with the same row, share an error: equal ones keep the order.
"""

import numpy as np
import pytest
import torch

import fp4_ref
from test_gpu_paged import B, BF16, D, F32, _geom, _i32  # noqa: F401

pytestmark = pytest.mark.gpu
INF = float("inf")
NAMES = ("new_score", "token", "parent", "new_done", "keep_len", "new_len")


def _oracle(logits, score, done, length, W, eos):
    """Per group: all offers in order [(score, slot, token)], in 64 bits."""
    x = logits.double().cpu().numpy()
    out = []
    for g in range(len(x) // W):
        offers = []
        for s in range(g * W, (g + 1) * W):
            sc = float(score[s])
            if not np.isfinite(sc):
                continue
            if done[s]:
                offers.append((sc, s, eos))
                continue
            row = x[s]
            m = row.max() if len(row) else -INF
            if not np.isfinite(m):           # a NaN, a +inf, or nothing but -inf
                continue
            z = row - m - np.log(np.exp(row - m).sum())
            at = np.argsort(-z, kind="stable")[:W]
            offers += [(sc + z[t], s, int(t)) for t in at if z[t] > -INF]
        offers.sort(key=lambda o: (-o[0], o[1], o[2]))
        out.append(offers)
    return out


def _lists(n):
    out = {k: torch.full((n,), -9, dtype=torch.int32, device="cuda") for k in NAMES}
    out["new_score"] = torch.full((n,), 9.0, device="cuda")
    return out


def _select(B, logits, score, done, length, W, eos, ws, out=None, stream=None):
    out = out or _lists(len(score))
    B.spark_beam_select(logits, score, done, length, W, eos, *(out[k] for k in NAMES), ws, stream=stream)
    return out


def _check(B, logits, score, W, eos=-1, done=None, length=None):
    n = len(score)
    done_l = [0] * n if done is None else done.tolist()
    length = torch.arange(3, 3 + n, dtype=torch.int32, device="cuda") if length is None else length
    ws = B.make_beam_workspace(n // W, W)
    out = _select(B, logits, score, done, length, W, eos, ws)
    again = _select(B, logits, score, done, length, W, eos, ws)
    assert B.spark_attn_error_word(ws) == 0
    for k in NAMES:
        assert torch.equal(out[k], again[k]), k
    got = {k: v.tolist() for k, v in out.items()}
    for g, offers in enumerate(_oracle(logits, score, done_l, length, W, eos)):
        for i in range(W):
            s = g * W + i
            if i >= len(offers):
                assert got["new_score"][s] == -INF and got["token"][s] == -1 and got["parent"][s] == -1
                assert got["new_done"][s] == 1 and got["keep_len"][s] == got["new_len"][s] == 0
                continue
            want, slot, token = offers[i]
            tol = 2.0 ** -18 + 2.0 ** -24 * abs(want)
            assert abs(got["new_score"][s] - want) <= tol
            near = [o for o in offers if abs(o[0] - want) <= 2 * tol and
                    (o[0] != want or not torch.equal(logits[o[1]], logits[slot]))]
            mine = (got["parent"][s], got["token"][s])
            assert mine == (slot, token) or mine in [(o[1], o[2]) for o in near]
            slot, token = mine
            assert got["keep_len"][s] == int(length[slot])
            assert got["new_len"][s] == int(length[slot]) + (0 if done_l[slot] else 1)
            assert got["new_done"][s] == int(bool(done_l[slot]) or token == eos)
        chosen = [(got["parent"][g * W + i], got["token"][g * W + i]) for i in range(min(W, len(offers)))]
        assert len(set(chosen)) == len(chosen)
    return out


def _random(n, vocab, dtype=F32, seed=0, pad=0, spread=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(n, vocab + pad, generator=g, device="cuda") * spread).to(dtype)
    return x[:, pad:], -30.0 * torch.rand(n, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("groups,W,vocab,pad", [
    (1, 1, 1, 0), (1, 1, 131072, 0), (1, 4, 131072, 0), (3, 5, 50257, 3), (7, 8, 4096, 0), (2, 32, 131071, 1), (1, 32, 40000, 0),
    (32, 32, 1001, 7), (5, 3, 2, 0), (2, 32, 17, 1), (128, 8, 300, 0), (1024, 1, 513, 0), (1, 32, 8193, 5), (64, 16, 33, 0)])
def test_random(B, groups, W, vocab, pad, dtype):
    logits, score = _random(groups * W, vocab, dtype, seed=groups + W, pad=pad)
    _check(B, logits, score, W)
    score = -20.0 + 0.01 * score    # beams close to one another: offers of all of them
    _check(B, logits, score, W)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("groups,W,vocab", [(1, 4, 131072), (9, 5, 20011), (2, 32, 5000), (3, 2, 7)])
def test_ended_beams_and_slots_out_of_use(B, groups, W, vocab, dtype):
    r = np.random.default_rng(groups)
    n = groups * W
    logits, score = _random(n, vocab, dtype, seed=7)
    logits = logits.clone()
    for eos in (0, vocab - 1, 1):
        logits[:, eos] += 9.0                      # ends are likely
        for p in (0.2, 0.7, 1.0):
            done = _i32(r.random(n) < p)
            sc = -8.0 + 0.2 * score
            _check(B, logits, sc, W, eos, done)
            sc[torch.tensor(r.random(n) < 0.4, device="cuda")] = -INF
            _check(B, logits, sc, W, eos, done)
    # before the first step: one beam of each group
    first = torch.where(torch.arange(n, device="cuda") % W == 0, 0.0, -INF)
    _check(B, logits, first, W, 0, _i32(np.zeros(n)))
    _check(B, logits, torch.full((n,), -INF, device="cuda"), W, 0, _i32(np.zeros(n)))


def test_scores_that_are_no_numbers(B):
    logits, score = _random(8, 5000, seed=3)
    for bad in (INF, float("nan")):
        score[1] = bad
        done = _i32([0, 0, 0, 1, 0, 1, 0, 0])
        score[5] = bad                             # an ended beam without a score offers nothing
        _check(B, logits, score, 4, 9, done)


@pytest.mark.parametrize("W,vocab", [(4, 131072), (5, 1000), (32, 9000)])
def test_masks_and_rows_without_a_distribution(B, W, vocab):
    n = 3 * W
    logits, score = _random(n, vocab, seed=5)
    logits = logits.clone()
    logits[0, 3:] = -INF                           # three tokens left
    logits[1] = -INF                               # nothing left
    logits[2, vocab // 2] = float("nan")
    logits[3, vocab - 1] = INF
    logits[W, 1:] = torch.finfo(F32).min           # a mask of the type's lowest value
    logits[W + 1, :vocab - 1] = -INF               # only the last token
    logits[2 * W:] = -INF                          # a group without an offer
    _check(B, logits, -1.0 + 0.01 * score, W)
    # equal scores everywhere: the lower beam, then the lower token
    for value in (0.0, -1e30, 3.5):
        out = _check(B, torch.full((n, vocab), value, device="cuda"), torch.full((n,), -2.0, device="cuda"), W)
        assert out["parent"].tolist() == [W * (i // W) for i in range(n)] and out["token"].tolist() == list(range(W)) * 3


def test_equal_logits_within_and_across_beams(B):
    g = torch.Generator(device="cuda").manual_seed(1)
    for W, vocab in ((8, 70000), (32, 3001), (4, 131072)):
        row = torch.randint(0, 9, (vocab,), generator=g, device="cuda").float()
        _check(B, row.expand(2 * W, vocab).contiguous(), torch.full((2 * W,), -5.0, device="cuda"), W)
        shuffled = torch.stack([row[torch.randperm(vocab, generator=g, device="cuda")] for _ in range(2 * W)])
        _check(B, shuffled, torch.full((2 * W,), -5.0, device="cuda"), W)
        _check(B, shuffled.sort(-1)[0], torch.full((2 * W,), -5.0, device="cuda"), W)


def test_dominated_and_far_apart_scores(B):
    logits, score = _random(12, 30000, seed=9, spread=40.0)
    _check(B, logits, score * 100, 6)
    _check(B, logits * 1e4, score, 6)


def test_zeros_of_either_sign_are_equal(B):
    logits, score = _random(4, 1000, seed=11)
    out = _check(B, logits, torch.tensor([-0.0, 0.0, 0.0, -0.0], device="cuda"), 4, 9, _i32([1] * 4))
    assert out["parent"].tolist() == [0, 1, 2, 3]
    # all of a row's weight on one token: a live beam's score stays 0
    logits[1:3] = -INF
    logits[1:3, 5] = -0.0
    out = _check(B, logits, torch.tensor([-1.0, 0.0, -0.0, -0.0], device="cuda"), 4, 9, _i32([1, 0, 0, 1]))
    assert out["parent"].tolist() == [1, 2, 3, 0] and out["token"].tolist() == [5, 5, 9, 9]


def test_what_fp32_cannot_hold_is_no_offer(B):
    """Next to a logit of 3e38 one of -3e38 has a log probability of -6e38."""
    logits = torch.full((6, 70000), -3e38, device="cuda")
    logits[:, 3] = 3e38
    logits[:3, 69999] = 3e38
    out = _lists(6)
    ws = B.make_beam_workspace(2, 3)
    _select(B, logits, torch.full((6,), -1.0, device="cuda"), None, _i32([4] * 6), 3, -1, ws, out)
    assert out["token"].tolist() == [3, 69999, 3, 3, 3, 3] and out["parent"].tolist() == [0, 0, 1, 3, 4, 5]
    half = -1.0 - np.log(2.0)
    assert np.allclose(out["new_score"].tolist(), [half] * 3 + [-1.0] * 3, atol=2.0 ** -18)
    _select(B, logits[3:], torch.tensor([-1.0, -INF, -INF], device="cuda"), None, _i32([4] * 3), 3, -1, ws, first := _lists(3))
    assert first["parent"].tolist() == [0, -1, -1] and first["new_score"].tolist()[1:] == [-INF, -INF]
    assert B.spark_attn_error_word(ws) == 0


def test_outputs_in_place_of_inputs(B):
    for n, W, vocab in ((64, 8, 9001), (4, 4, 131072)):
        logits, score = _random(n, vocab, seed=2)
        done, length = _i32(np.arange(n) % 5 == 0), _i32(np.arange(n) + 1)
        ws = B.make_beam_workspace(n // W, W)
        want = _select(B, logits, score, done, length, W, 3, ws)
        sc, dn, ln = score.clone(), done.clone(), length.clone()
        out = {**_lists(n), "new_score": sc, "new_done": dn, "new_len": ln}
        _select(B, logits, sc, dn, ln, W, 3, ws, out)
        for k in NAMES:
            assert torch.equal(out[k], want[k]), k
        # without lengths, without an end
        lists = _lists(n)
        B.spark_beam_select(logits, score, None, None, W, -1, lists["new_score"], lists["token"], lists["parent"], None, None,
                            None, ws)
        full = _select(B, logits, score, None, length, W, -1, ws)
        for k in ("new_score", "token", "parent"):
            assert torch.equal(lists[k], full[k])
        assert B.spark_attn_error_word(ws) == 0


def test_captured_selection_and_streams(B):
    logits, score = _random(20, 60000, seed=4)
    length = _i32(np.arange(20))
    ws, ws2 = B.make_beam_workspace(4, 5), B.make_beam_workspace(4, 5)
    out, side = _lists(20), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _select(B, logits, score, None, length, 5, -1, ws, out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _select(B, logits, score, None, length, 5, -1, ws, out)
    for i in range(3):
        score.copy_(-30.0 * torch.rand(20, device="cuda"))
        logits.normal_()
        graph.replay()
        other = _select(B, logits, score, None, length, 5, -1, ws2)
        torch.cuda.synchronize()
        for k in NAMES:
            assert torch.equal(out[k], other[k]), k


# ---------------------------------------------------------------------------
# reordering
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n,width", [(1, 1), (7, 130), (64, 1023), (1024, 5), (3, 50001)])
def test_reorder(B, n, width):
    r = np.random.default_rng(n)
    parent = r.integers(-1, n, n)
    keep = np.where(parent < 0, 0, r.integers(0, width + 1, n))
    new = keep + np.where(keep < width, r.integers(0, 2, n), 0)
    token = _i32(r.integers(0, 99, n))
    ws = B.make_beam_workspace(1, 1)
    hist = torch.randint(0, 1000, (n, width), dtype=torch.int32, device="cuda")
    rows = [torch.randn(n, width, device="cuda"), torch.randn(n, 2 * width, device="cuda").to(BF16),
            torch.randn(n, 3, 4 * width, device="cuda"), torch.randn(n, width, 2, device="cuda")]
    states = [B.BeamState(hist, torch.full_like(hist, -7), positions=True, push=token)]
    states += [B.BeamState(x, torch.full_like(x, -7)) for x in rows[:3]]
    states.append(B.BeamState(rows[3], torch.full_like(rows[3], -7), positions=True))
    B.spark_beam_reorder(_i32(parent), _i32(keep), _i32(new), states, ws)
    assert B.spark_attn_error_word(ws) == 0
    for i, st in enumerate(states):
        want = torch.full_like(st.src, -7)
        for s in range(n):
            if parent[s] >= 0:
                m = keep[s] if st.positions else None
                want[s, :m] = st.src[parent[s], :m]
                if i == 0 and new[s] > keep[s]:
                    want[s, keep[s]] = token[s]
        assert torch.equal(st.dst, want), i
    # whole rows need no lengths
    B.spark_beam_reorder(_i32(parent), None, None, states[1:4], ws)
    assert B.spark_attn_error_word(ws) == 0


def test_reorder_reports_what_has_no_room(B):
    hist = torch.arange(40, dtype=torch.int32, device="cuda").view(4, 10)
    token = _i32([7, 7, 7, 7])

    def run(parent, keep, new, push=True):
        st = B.BeamState(hist, torch.full_like(hist, -1), positions=True, push=token if push else None)
        ws = B.make_beam_workspace(2, 2)
        B.spark_beam_reorder(_i32(parent), _i32(keep), _i32(new), [st], ws)
        return B.spark_attn_error_word(ws), st.dst
    ok = [1, 0, 3, -1], [9, 10, 0, 0], [10, 10, 1, 0]
    word, dst = run(*ok)
    assert word == 0 and dst[0].tolist() == list(range(10, 19)) + [7] and dst[1].tolist() == list(range(10))
    assert dst[2].tolist() == [7] + [-1] * 9 and dst[3].tolist() == [-1] * 10
    for which, at, value in ((0, 0, 4), (0, 1, -2), (0, 2, 2 ** 31 - 1), (1, 0, 11), (1, 1, -1), (1, 1, 2 ** 31 - 1), (2, 0, 8),
                             (2, 1, 11)):
        args = [list(x) for x in ok]
        args[which][at] = value
        word, bad = run(*args)
        assert word == 2, (which, at, value)
        for s in range(4):
            assert bad[s].tolist() == ([-1] * 10 if s == at else dst[s].tolist())
    assert run(ok[0], ok[1], [99, 99, 99, 99], push=False)[0] == 0      # nothing is written behind


# ---------------------------------------------------------------------------
# steps of beam search on 4-bit pages
# ---------------------------------------------------------------------------

class Searcher:
    """A one-layer model with random weights that searches with beams: the
    library's calls of a step, all lengths and tables on the device."""

    def __init__(self, B, groups=3, W=4, vocab=601, page=16, steps=12, seed=0):
        self.B, self.W, self.n, self.vocab, self.page = B, W, groups * W, vocab, page
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.geom, n = _geom(B), self.n
        self.embed = torch.randn(vocab, 64, generator=g, device="cuda")
        self.w_qkv = torch.randn(64, 6144, generator=g, device="cuda") * 0.125
        self.w_out = torch.randn(4096, vocab, generator=g, device="cuda") * 0.05
        width, n_pages = 6, 6 * n
        shape = (n_pages, page // 16, 4, fp4_ref.BLOCK)
        self.k, self.v = (torch.full(shape, 0xFF, dtype=torch.uint8, device="cuda") for _ in "kv")
        self.pool = B.PagePool(self.k, self.v)
        self.rope = torch.zeros(96, 32, 2, device="cuda")
        B.spark_rope_table(self.geom, B.SPARK_FULL, self.rope)
        z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.table, self.new_table = torch.full((n, width), -1, dtype=torch.int32, device="cuda"), z(n, width)
        self.length, self.done, self.token, self.parent = z(n), z(n), z(n), z(n)
        self.keep_len = z(n)
        self.score = torch.where(torch.arange(n, device="cuda") % W == 0, 0.0, -INF)
        self.hist, self.new_hist = z(n, 96), z(n, 96)
        self.logits = torch.randn(n, vocab, generator=g, device="cuda") * 2
        self.q, self.a = torch.zeros(n, 4096, device="cuda"), torch.zeros(n, 4096, device="cuda")
        self.batch = B.PagedBatch(self.table, _i32(np.arange(n + 1)), z(n), n, 1)
        self.bws, self.pws, self.tws = B.make_beam_workspace(groups, W), B.make_paged_workspace(self.geom), B.make_pages_workspace(n_pages, n)
        self.moves = [B.BeamState(self.hist, self.new_hist, positions=True, push=self.token)]

    def step(self):
        B, g = self.B, self.geom
        B.spark_beam_select(self.logits, self.score, self.done, self.length, self.W, 5, self.score, self.token, self.parent,
                            self.done, self.keep_len, self.length, self.bws)
        B.spark_beam_reorder(self.parent, self.keep_len, self.length, self.moves, self.bws)
        B.spark_pages_remap(g, [self.pool], self.table, self.parent, self.keep_len, self.length, self.new_table, self.tws)
        self.hist.copy_(self.new_hist)
        self.table.copy_(self.new_table)
        self.batch.seq_len.copy_(self.length)
        x = self.embed[self.token.clamp(min=0).long()] @ self.w_qkv
        # (an ended beam brings its last token again: its rows and its logits change nothing that counts)
        B.spark_paged_rope_append(g, x[:, :4096], x[:, 4096:5120], x[:, 5120:], B.SPARK_FULL, self.rope, self.pool, self.batch,
                                  self.q, self.pws)
        B.spark_paged_attention(g, self.q, self.pool, B.SPARK_FULL, self.batch, self.a, self.pws)
        torch.matmul(self.a, self.w_out, out=self.logits)

    def words(self):
        return [self.B.spark_attn_error_word(w) for w in (self.bws, self.pws, self.tws)]


def test_steps_of_beam_search_on_4_bit_pages(B):
    """Every step against an oracle that keeps each beam's tokens and recomputes
    its keys, values and attention from them."""
    m = Searcher(B)
    n, W = m.n, m.W
    beams = [[] for _ in range(n)]
    for step in range(20):
        logits, score, done, length = m.logits.clone(), m.score.clone(), m.done.clone(), m.length.clone()
        m.step()
        torch.cuda.synchronize()
        assert m.words() == [0, 0, 0]
        offers = _oracle(logits, score, done.tolist(), length, W, 5)
        parent, token = m.parent.tolist(), m.token.tolist()
        for s in range(n):
            want = offers[s // W][s % W]
            assert abs(float(m.score[s]) - want[0]) <= 2.0 ** -18 + 2.0 ** -24 * abs(want[0])
            assert (parent[s], token[s]) == want[1:]
        beams = [beams[parent[s]] + ([] if done[parent[s]] else [token[s]]) for s in range(n)]
        assert [m.hist[s, :len(b)].tolist() for s, b in enumerate(beams)] == beams
        assert m.length.tolist() == [len(b) for b in beams]
        if step % 4 == 3:
            for s, b in enumerate(beams):
                x = (m.embed[torch.tensor(b, device="cuda")] @ m.w_qkv).double()
                cs = m.rope[:len(b)].double()
                turned = x[:, :5120].view(len(b), 20, D).clone()
                p, q = turned[..., :32].clone(), turned[..., 32:64].clone()
                c, sn = cs[:, None, :, 0], cs[:, None, :, 1]
                turned[..., :32], turned[..., 32:64] = p * c - q * sn, q * c + p * sn
                pos = torch.arange(len(b), device="cuda")
                k, v = (fp4_ref.values(*fp4_ref.read(pl, m.table[s], m.page, pos, 4)) for pl in (m.k, m.v))
                # (the products of a batch of another size are summed in another order: a code may differ by a step)
                near = (fp4_ref.values(*fp4_ref.quantize(turned[:, 16:].float())) - k).abs()
                assert near.max() <= 0.5 * k.abs().max() and (near > 0).double().mean() < 0.01
                sc = 0.0625 * torch.einsum("hd,xhd->hx", turned[-1, :16], k.repeat_interleave(4, 1))
                o = torch.einsum("hx,xhd->hd", torch.softmax(sc, -1), v.repeat_interleave(4, 1))
                want = o.flatten() @ m.w_out.double()
                assert (m.logits[s].double() - want).abs().max() <= 1e-3 * want.abs().max() + 1e-3


def test_captured_steps_replay(B):
    """One step's graph, replayed: the tables, lengths, tokens and scores of steps enqueued one by one."""
    a, b = Searcher(B, seed=3), Searcher(B, seed=3)
    for m in (a, b):
        m.step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    keep = [t.clone() for t in (b.table, b.length, b.done, b.score, b.hist, b.logits, b.k, b.v, b.token, b.batch.seq_len)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.step()
    side.synchronize()
    with torch.cuda.graph(graph):
        b.step()
    for t, old in zip((b.table, b.length, b.done, b.score, b.hist, b.logits, b.k, b.v, b.token, b.batch.seq_len), keep):
        t.copy_(old)
    for _ in range(10):
        a.step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.parent, b.parent) and torch.equal(a.token, b.token) and torch.equal(a.score, b.score)
        assert torch.equal(a.table, b.table) and torch.equal(a.length, b.length) and torch.equal(a.logits, b.logits)
    assert a.words() == [0, 0, 0] and b.words() == [0, 0, 0]
