"""Cases of the paged-cache operators and of the token scores, in their plain
form (elementary torch operations in fp32) and through the library.

  append    k and v rows of new tokens into a paged cache
  attention grouped-query attention of every sequence's new tokens (one, a few
            drafted ones, a chunk of a prompt) over its pages
  remap     the page tables of a step: sequences kept, forked, cut, freed, grown
  compact   the pages in use moved to the front of the pool
  logprobs  log probabilities of given tokens, entropy, top alternatives
"""

import math

import numpy as np
import torch

own = False

HEAD = 256      # head_dim
GROUP = 4       # query heads per KV head
WINDOW = 512    # sliding layers
SCALE = 0.0625  # 256^-0.5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one sequence, one new token at position 700: the smallest decode call
        dict(name="attention b1 pos700", op="attention", q="f32", kv="bf16", n_kv=4, page=64, full=True, seqs=1,
             ctx_lo=701, ctx_hi=701, q_lo=1, q_hi=1, long=0, lens=1),
        # 64 sequences decoding at ragged contexts: the default serving step's full layer
        dict(name="attention b64 ctx512-32768", op="attention", q="bf16", kv="bf16", n_kv=4, page=64, full=True,
             seqs=64, ctx_lo=512, ctx_hi=32768, q_lo=1, q_hi=1, long=0, lens=2),
        # a long prompt's chunk over the history before it
        dict(name="attention chunk 4096 at 4096", op="attention", q="bf16", kv="bf16", n_kv=4, page=128, full=True,
             seqs=1, ctx_lo=8192, ctx_hi=8192, q_lo=4096, q_hi=4096, long=0, lens=3),
        # continuous batching: 4 sequences bring chunks of prompts, the others verify up to 7 drafted tokens;
        # odd lengths, small pages, fp32 queries as the block's projections leave them
        dict(name="attention mixed b32", op="attention", q="f32", kv="bf16", n_kv=4, page=16, full=True, seqs=32,
             ctx_lo=300, ctx_hi=6000, q_lo=1, q_hi=7, long=4, long_hi=517, lens=4),
        # the rows of one decode step of 64 sequences
        dict(name="append b64", op="append", x="f32", kv="bf16", n_kv=4, page=64, seqs=64, ctx_lo=512, ctx_hi=2048,
             q_lo=1, q_hi=1, lens=5),
        # the rows of prompts, from the fused projection's fp32 output
        dict(name="append 8 prompts", op="append", x="f32", kv="bf16", n_kv=4, page=16, seqs=8, ctx_lo=1500,
             ctx_hi=4000, q_lo=700, q_hi=1500, lens=6),
        # one decode step's page tables: most sequences grow by a token, some end, some begin
        dict(name="remap step b64", op="remap", layers=36, n_kv=4, page=16, seqs=64, ctx_lo=20, ctx_hi=180, kind="step",
             spare=128, lens=7),
        # parallel sampling: every 8th sequence is forked into the seven slots behind it, in 36 layers
        dict(name="remap fork 16x8", op="remap", layers=36, n_kv=4, page=32, seqs=128, ctx_lo=40, ctx_hi=900,
             kind="fork", spare=160, lens=8),
        # a pool a quarter full after a burst of requests, a few layers
        dict(name="compact 300 of 1200", op="compact", layers=4, n_kv=4, page=16, seqs=24, ctx_lo=100, ctx_hi=300,
             pool=1200, lens=9),
        # half a pool of 36 layers
        dict(name="compact half of 900 x36", op="compact", layers=36, n_kv=4, page=16, seqs=40, ctx_lo=60, ctx_hi=300,
             pool=900, lens=10),
        # one sequence's sampled token, with 20 alternatives
        dict(name="logprobs 1", op="logprobs", x="f32", rows=1, vocab=131072, top=20),
        # the scores of a chunk of a prompt (an odd number of rows)
        dict(name="logprobs 511", op="logprobs", x="f32", rows=511, vocab=131072, top=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "remap", "compact", "logprobs"])
    n_kv = rng.choice([1, 2, 3, 4, 4, 4, 5, 8])
    lens = rng.randrange(1 << 30)
    if op == "attention":
        kind = rng.choice(["decode", "verify", "chunk", "mixed"])
        c = dict(op=op, q=rng.choice(["f32", "bf16"]), kv=rng.choice(["bf16", "bf16", "bf16", "f32"]), n_kv=n_kv,
                 page=rng.choice([16, 32, 48, 64, 80, 128, 256]), full=rng.random() < 0.7, long=0, lens=lens)
        if kind == "decode":
            c.update(seqs=_log(rng, 1, 64), q_lo=1, q_hi=1)
            c.update(ctx_lo=rng.randrange(1, 500), ctx_hi=_log(rng, 600, 32768 if c["seqs"] < 33 else 8000))
        elif kind == "verify":
            c.update(seqs=_log(rng, 1, 40), q_lo=rng.randrange(0, 3), q_hi=rng.randrange(3, 17))
            c.update(ctx_lo=rng.randrange(17, 500), ctx_hi=_log(rng, 600, 12000))
        elif kind == "chunk":
            n = _log(rng, 33, 1500)
            c.update(seqs=rng.randrange(1, 4), q_lo=max(1, n // 2), q_hi=n, ctx_lo=n, ctx_hi=n + rng.randrange(0, 2500))
        else:
            c.update(seqs=rng.randrange(3, 33), q_lo=rng.randrange(0, 2), q_hi=rng.randrange(2, 9),
                     long=rng.randrange(1, 4), long_hi=_log(rng, 40, 700))
            c.update(ctx_lo=rng.randrange(9, 300), ctx_hi=_log(rng, 800, 6000))
        if c["kv"] == "f32":  # a test and debugging type: shorter
            c["ctx_hi"] = max(c["ctx_lo"], min(c["ctx_hi"], 1500))
        return c
    if op == "append":
        hi = _log(rng, 1, 1500)
        return dict(op=op, x=rng.choice(["f32", "bf16"]), kv=rng.choice(["bf16", "bf16", "f32"]), n_kv=n_kv,
                    page=rng.choice([16, 32, 48, 64, 128]), seqs=rng.randrange(1, 33), ctx_lo=hi, ctx_hi=hi + 2500,
                    q_lo=rng.randrange(0, hi + 1), q_hi=hi, lens=lens)
    if op == "remap":
        seqs = _log(rng, 2, 256)
        return dict(op=op, layers=rng.choice([1, 2, 9, 36]), n_kv=n_kv, page=rng.choice([16, 32, 64]), seqs=seqs,
                    ctx_lo=rng.randrange(1, 40), ctx_hi=_log(rng, 50, 20000 // seqs + 60),
                    kind=rng.choice(["step", "fork", "mixed"]), spare=2 * seqs + rng.randrange(0, 64), lens=lens)
    if op == "compact":
        seqs = rng.randrange(1, 40)
        hi = _log(rng, 40, 400)
        return dict(op=op, layers=rng.choice([1, 2, 9, 36]), n_kv=n_kv, page=rng.choice([16, 32]), seqs=seqs,
                    ctx_lo=rng.randrange(1, 40), ctx_hi=hi, pool=seqs * (hi // 16 + 1) + rng.randrange(0, 200), lens=lens)
    return dict(op=op, x=rng.choice(["f32", "bf16"]), rows=_log(rng, 1, 500), vocab=_log(rng, 1000, 131072) | 1,
                top=rng.choice([0, 1, 5, 20, 32]), lens=lens)


def _lengths(c):
    """(context, new tokens) of every sequence: what the case's numbers stand for."""
    r = np.random.RandomState(c["lens"] & 0x7FFFFFFF)
    ctx = r.randint(c["ctx_lo"], c["ctx_hi"] + 1, size=c["seqs"])
    if "q_lo" not in c:
        return ctx, None
    new = r.randint(c["q_lo"], c["q_hi"] + 1, size=c["seqs"])
    if c.get("long"):
        at = r.permutation(c["seqs"])[: c["long"]]
        new[at] = r.randint(max(1, c["long_hi"] // 2), c["long_hi"] + 1, size=len(at))
    new = np.minimum(new, ctx)
    if new.sum() == 0:
        new[0] = 1
    return ctx, new


def _remap_lists(c):
    """parent, keep and new length of every slot, and the old lengths."""
    ctx, _ = _lengths(c)
    r = np.random.RandomState((c["lens"] + 1) & 0x7FFFFFFF)
    n = c["seqs"]
    parent, keep = np.arange(n), ctx.copy()
    new = ctx + 1
    kind = c["kind"]
    if kind in ("step", "mixed"):
        ended = r.rand(n) < 0.1
        parent[ended], keep[ended] = -1, 0
        new[ended] = r.randint(0, 40, size=int(ended.sum()))
        cut = ~ended & (r.rand(n) < 0.2)  # rejected drafts
        keep[cut] = np.maximum(0, ctx[cut] - r.randint(0, 6, size=int(cut.sum())))
        new[cut] = keep[cut] + 5
    if kind == "fork" or kind == "mixed":
        f = 8 if kind == "fork" else 3
        for s in range(n):
            if s % f and (kind == "fork" or r.rand() < 0.5):
                p = s - s % f
                parent[s], keep[s], new[s] = p, ctx[p], ctx[p] + 1
    return ctx, parent, keep, new


def _pages_of(rows, page):
    return -(-rows // page)


def work(case):
    c = case
    op = c["op"]
    row = c.get("n_kv", 0) * HEAD  # elements of one K (or V) row
    if op == "attention":
        ctx, new = _lengths(c)
        es, qs = (2 if c["kv"] == "bf16" else 4), (2 if c["q"] == "bf16" else 4)
        rows = pairs = 0
        for n, q in zip(ctx.tolist(), new.tolist()):
            if q == 0:
                continue
            first = n - q
            seen = np.arange(first, n) + 1
            if not c["full"]:
                seen = np.minimum(seen, WINDOW)
            pairs += int(seen.sum())
            rows += n - (0 if c["full"] else max(0, first + 1 - WINDOW))
        return {"bytes": 2 * rows * row * es + 2 * int(new.sum()) * GROUP * row * qs,
                "flops": 4 * HEAD * GROUP * c["n_kv"] * pairs}
    if op == "append":
        _, new = _lengths(c)
        return {"bytes": 2 * int(new.sum()) * row * ((4 if c["x"] == "f32" else 2) + (4 if c["kv"] == "f32" else 2)),
                "flops": 0}
    if op == "remap":
        ctx, parent, keep, new = _remap_lists(c)
        page = c["page"]
        holders = {}
        for s in range(c["seqs"]):
            if keep[s] % page:
                holders.setdefault((int(parent[s]), int(keep[s]) // page), []).append(s)
        full = {(int(parent[s]), i) for s in range(c["seqs"]) for i in range(int(keep[s]) // page)}
        rows = 0
        for key, who in holders.items():
            rows += sum(int(keep[s]) % page for s in who if key in full or s != min(who))
        width = int(_pages_of(max(int(ctx.max()), int(new.max())), page))
        return {"bytes": 8 * c["seqs"] * width + 2 * rows * 2 * c["layers"] * row * 2, "flops": 0}
    if op == "compact":
        ctx, _ = _lengths(c)
        live = int(_pages_of(ctx, c["page"]).sum())
        moved = max(0, live * (c["pool"] - live)) / c["pool"]  # of a random placement, on average
        return {"bytes": 8 * live + 2 * moved * 2 * c["layers"] * c["page"] * row * 2, "flops": 0}
    es = 4 if c["x"] == "f32" else 2
    return {"bytes": c["rows"] * (c["vocab"] * es + 12 + 8 * c["top"]), "flops": 6 * c["rows"] * c["vocab"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _dev(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def _tables(ctx, page, pool, g, width=None):
    """Page tables [sequences, width] of random pages of a pool (-1: none)."""
    need = _pages_of(ctx, page)
    width = int(need.max()) if width is None else width
    at = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    n = torch.tensor(need, device="cuda")
    start = torch.cumsum(n, 0) - n
    return torch.where(col < n[:, None], at[(start[:, None] + col).clamp(max=pool - 1)], -1)


def prepare(case, seed):
    c = case
    op = c["op"]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": c}
    if op == "logprobs":
        x = torch.randn(c["rows"], c["vocab"], generator=g, device="cuda").mul_(2.5)
        s["logits"] = x.to(_DT[c["x"]])
        s["targets"] = torch.randint(0, c["vocab"], (c["rows"],), generator=g, device="cuda", dtype=torch.int32)
    else:
        n_kv, page = c["n_kv"], c["page"]
        s["window"] = WINDOW
    if op in ("attention", "append"):
        ctx, new = _lengths(c)
        pool = int(_pages_of(ctx, page).sum()) + 3
        shape = (pool, page, n_kv, HEAD)
        dt = _DT[c["kv"]]
        s["k"] = torch.randn(shape, generator=g, device="cuda", dtype=dt)
        s["v"] = torch.randn(shape, generator=g, device="cuda", dtype=dt)
        s["table"] = _tables(ctx, page, pool, g)
        s["q_start"] = _dev(np.concatenate([[0], np.cumsum(new)]))
        s["seq_len"] = _dev(ctx)
        s["tokens"], s["max_q"], s["max_ctx"] = int(new.sum()), int(new.max()), int(ctx.max())
        if op == "attention":
            s["q"] = torch.randn(s["tokens"], GROUP * n_kv * HEAD, generator=g, device="cuda").to(_DT[c["q"]])
            s["out"] = torch.zeros_like(s["q"])
        else:  # the fused projection's rows: q | k | v
            s["qkv"] = torch.randn(s["tokens"], (GROUP + 2) * n_kv * HEAD, generator=g, device="cuda").to(_DT[c["x"]])
    elif op in ("remap", "compact"):
        if op == "remap":
            ctx, parent, keep, new = _remap_lists(c)
            pool = int(_pages_of(ctx, page).sum()) + int(_pages_of(new, page).sum() - _pages_of(keep, page).sum()) + c["spare"]
            width = int(_pages_of(max(int(ctx.max()), int(new.max())), page))
            s["parent"], s["keep"], s["new"] = _dev(parent), _dev(keep), _dev(new)
        else:
            ctx, _ = _lengths(c)
            pool, width = c["pool"], None
        s["table"] = _tables(ctx, page, pool, g, width)
        s["out_table"] = torch.zeros_like(s["table"])
        # every layer's K and V pages: [layer][k, v][page][row][head][dim]
        s["pools"] = torch.randn((c["layers"], 2, pool, page, n_kv, HEAD), generator=g, device="cuda",
                                 dtype=torch.bfloat16)
        s["n_live"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        _keep_handles(s)
    return s


def _keep_handles(s):
    """What a program keeps between calls: geometry, descriptors, workspaces, output buffers."""
    from decode_attention_block_gb300 import binding as B
    c = s["case"]
    s["B"] = B
    geom = s["geom"] = B.spark_geom_default()
    if c["op"] == "logprobs":
        n, k = c["rows"], c["top"]
        s["logprob"] = torch.zeros(n, device="cuda")
        s["entropy"] = torch.zeros(n, device="cuda")
        s["top_ids"] = torch.zeros(n, k, dtype=torch.int32, device="cuda")
        s["top_logprobs"] = torch.zeros(n, k, device="cuda")
        s["ws"] = B.make_logprobs_workspace(n, k)
        return
    geom.n_kv, geom.n_q = c["n_kv"], GROUP * c["n_kv"]
    if c["op"] in ("attention", "append"):
        s["pool"] = B.PagePool(s["k"], s["v"])
        s["batch"] = B.PagedBatch(s["table"], s["q_start"], s["seq_len"], s["tokens"], s["max_q"])
        s["ws"] = B.make_paged_workspace(geom)
    else:
        s["page_pools"] = [B.PagePool(p[0], p[1]) for p in s["pools"]]
        s["ws"] = B.make_pages_workspace(s["pools"].shape[2], s["table"].shape[0])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_attention(s):
    B = s["B"]
    cls = B.SPARK_FULL if s["case"]["full"] else B.SPARK_SLIDING
    B.spark_paged_attention(s["geom"], s["q"], s["pool"], cls, s["batch"], s["out"], s["ws"])
    return s["out"]


def _own_append(s):
    q, kv = GROUP * s["case"]["n_kv"] * HEAD, s["case"]["n_kv"] * HEAD
    x = s["qkv"]
    s["B"].spark_paged_append(s["geom"], x[:, q:q + kv], x[:, q + kv:], s["pool"], s["batch"], s["ws"])
    return {"k": s["k"], "v": s["v"]}


def _own_remap(s):
    s["B"].spark_pages_remap(s["geom"], s["page_pools"], s["table"], s["parent"], s["keep"], s["new"], s["out_table"],
                             s["ws"])
    return {"table": s["out_table"], "pools": s["pools"]}


def _own_compact(s):
    s["B"].spark_pages_compact(s["geom"], s["page_pools"], s["table"], s["out_table"], s["n_live"], s["ws"])
    return {"table": s["out_table"], "n_live": s["n_live"], "pools": s["pools"]}


def _own_logprobs(s):
    s["B"].spark_token_logprobs(s["logits"], s["targets"], s["logprob"], s["entropy"], s["top_ids"],
                                s["top_logprobs"], s["ws"])
    return {k: s[k] for k in ("logprob", "entropy", "top_ids", "top_logprobs")}


_OWN = {"attention": _own_attention, "append": _own_append, "remap": _own_remap, "compact": _own_compact,
        "logprobs": _own_logprobs}


def _plain_attention(s):
    c, page = s["case"], s["case"]["page"]
    n_kv, n, t = c["n_kv"], s["table"].shape[0], s["tokens"]
    pos = torch.arange(s["max_ctx"], device="cuda")
    pages = s["table"][:, pos // page].clamp(min=0).long()
    k = s["k"][pages, pos % page].float()  # [n, ctx, n_kv, 256]
    v = s["v"][pages, pos % page].float()
    q0, length = s["q_start"][:-1].long(), s["seq_len"].long()
    new = s["q_start"][1:].long() - q0
    i = torch.arange(s["max_q"], device="cuda")
    tok = torch.where(i < new[:, None], q0[:, None] + i, t)  # t: a row for those that are not there
    q = s["q"].float().view(t, n_kv, GROUP, HEAD)[tok.clamp(max=t - 1)]
    at = (length - new)[:, None] + i  # position of each token
    seen = pos <= at[:, :, None]
    if not c["full"]:
        seen &= pos > at[:, :, None] - s["window"]
    seen &= pos < length[:, None, None]
    # rows that no token sees may hold anything
    v = torch.where(seen.any(1)[:, :, None, None], v, 0.0)
    sc = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(n, n_kv, GROUP * s["max_q"], HEAD), k.permute(0, 2, 3, 1))
    sc = sc.view(n, n_kv, GROUP, s["max_q"], -1).mul_(SCALE)
    sc.masked_fill_(~seen[:, None, None], float("-inf"))
    sc.sub_(sc.amax(-1, keepdim=True)).exp_()
    sc.div_(sc.sum(-1, keepdim=True))
    o = torch.matmul(sc.view(n, n_kv, GROUP * s["max_q"], -1), v.permute(0, 2, 1, 3))
    o = o.view(n, n_kv, GROUP, s["max_q"], HEAD).permute(0, 3, 1, 2, 4).reshape(n * s["max_q"], -1)
    out = torch.zeros(t + 1, n_kv * GROUP * HEAD, device="cuda")
    out[tok.reshape(-1)] = o
    return out[:t].to(s["q"].dtype)


def _plain_append(s):
    c, page = s["case"], s["case"]["page"]
    q, kv = GROUP * c["n_kv"] * HEAD, c["n_kv"] * HEAD
    t = torch.arange(s["tokens"], device="cuda")
    ends = s["q_start"][1:].long()
    seq = (ends <= t[:, None]).sum(1)
    pos = s["seq_len"].long()[seq] - (ends[seq] - t)
    at = s["table"][seq, pos // page].long(), pos % page
    x = s["qkv"]
    s["k"][at] = x[:, q:q + kv].reshape(-1, c["n_kv"], HEAD).to(s["k"].dtype)
    s["v"][at] = x[:, q + kv:].reshape(-1, c["n_kv"], HEAD).to(s["v"].dtype)
    return {"k": s["k"], "v": s["v"]}


def _plain_remap(s):
    page, table, pools = s["case"]["page"], s["table"].long(), s["pools"]
    n, width = table.shape
    total = pools.shape[2]
    parent, keep, new = s["parent"].long(), s["keep"].long(), s["new"].long()
    slot, col = torch.arange(n, device="cuda"), torch.arange(width, device="cuda")
    full, rest = keep // page, keep % page
    kept, wanted = (keep + page - 1) // page, (new + page - 1) // page
    old = table[parent.clamp(min=0)]
    used = torch.zeros(total + 1, dtype=torch.bool, device="cuda")
    used[torch.where(col < full[:, None], old, total)] = True
    last = torch.where(rest > 0, old.gather(1, full.clamp(max=width - 1)[:, None])[:, 0], total)
    first = torch.full((total + 1,), n, device="cuda").scatter_reduce_(0, last, slot, "amin")
    # a page that a slot has in part is its own: it stays with the first of those that have it so, if nobody has it whole
    copied = (rest > 0) & (used[last] | (first[last] != slot))
    need = copied + wanted - kept
    begin = torch.cumsum(need, 0) - need
    live = used[:total] | (first[:total] < n)
    free = torch.argsort(live.to(torch.int8), stable=True)  # the free pages, lowest first
    fresh = free[(begin[:, None] + col - kept[:, None] + copied[:, None]).clamp(0, total - 1)]
    out = torch.where(col < kept[:, None], old, torch.where(col < wanted[:, None], fresh, -1))
    to = free[begin.clamp(max=total - 1)]
    out = torch.where((col == full[:, None]) & copied[:, None], to[:, None], out)
    who = copied.nonzero()[:, 0]
    rows = torch.arange(page, device="cuda") < rest[who][:, None]
    w, r = rows.nonzero(as_tuple=True)
    pools[:, :, to[who][w], r] = pools[:, :, last[who][w], r]
    return {"table": out.to(torch.int32), "pools": pools}


def _plain_compact(s):
    table, pools = s["table"].long(), s["pools"]
    total = pools.shape[2]
    live = torch.zeros(total + 1, dtype=torch.bool, device="cuda")
    live[torch.where(table >= 0, table, total)] = True
    live = live[:total]
    n_live = live.sum()
    at = torch.arange(total, device="cuda")
    src = (live & (at >= n_live)).nonzero()[:, 0]
    dst = (~live & (at < n_live)).nonzero()[:, 0]
    to = at.clone()
    to[src] = dst
    pools[:, :, dst] = pools[:, :, src]
    return {"table": torch.where(table >= 0, to[table.clamp(min=0)], -1).to(torch.int32),
            "n_live": n_live.to(torch.int32).view(1), "pools": pools}


def _plain_logprobs(s):
    x, k = s["logits"].float(), s["case"]["top"]
    d = x - x.amax(-1, keepdim=True)
    e = d.exp()
    z = e.sum(-1)
    lz = z.log()
    lp = d.gather(1, s["targets"].long()[:, None])[:, 0] - lz
    h = lz - torch.where(e > 0, e * d, 0.0).sum(-1) / z
    ids = torch.sort(x, dim=-1, descending=True, stable=True)[1][:, :k]
    return {"logprob": lp, "entropy": h, "top_ids": ids.to(torch.int32), "top_logprobs": d.gather(1, ids) - lz[:, None]}


_PLAIN = {"attention": _plain_attention, "append": _plain_append, "remap": _plain_remap, "compact": _plain_compact,
          "logprobs": _plain_logprobs}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    c = case
    if c["op"] == "logprobs":
        s = prepare(c, seed)
        lp, h, top = [], [], []
        for row, t in zip(s["logits"], s["targets"].tolist()):
            p = row.double()
            ln = torch.log_softmax(p, 0)
            lp.append(ln[t])
            h.append(-(ln.exp() * ln).nan_to_num(0.0).sum())
            top.append(torch.topk(ln, c["top"])[0])
        return {"logprob": torch.stack(lp), "entropy": torch.stack(h), "top_ids": None, "top_logprobs": torch.stack(top)}
    if c["op"] != "attention":
        return None
    if work(c)["flops"] > 6e11:
        return None
    s = prepare(c, seed)
    page, n_kv = c["page"], c["n_kv"]
    ctx, new = s["seq_len"].tolist(), np.diff(s["q_start"].cpu().numpy()).tolist()
    out = torch.zeros(s["tokens"], n_kv, GROUP, HEAD, dtype=torch.float64, device="cuda")
    t = 0
    for b, (n, m) in enumerate(zip(ctx, new)):
        if m == 0:
            continue
        p = s["table"][b, : -(-n // page)].long()
        k = s["k"][p].reshape(-1, n_kv, HEAD)[:n].double()
        v = s["v"][p].reshape(-1, n_kv, HEAD)[:n].double()
        q = s["q"][t:t + m].double().view(m, n_kv, GROUP, HEAD)
        back = torch.arange(n - m, n, device="cuda")[:, None] - torch.arange(n, device="cuda")
        allowed = (back >= 0) if c["full"] else (back >= 0) & (back < WINDOW)
        for j in range(n_kv):
            for h in range(GROUP):
                z = (q[:, j, h] @ k[:, j].T) / math.sqrt(HEAD)
                w = torch.softmax(z.masked_fill(~allowed, -math.inf), -1)
                out[t:t + m, j, h] = w @ v[:, j]
        t += m
    return out.view(s["tokens"], -1)
