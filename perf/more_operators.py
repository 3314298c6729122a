"""Cases of the 4-bit paged cache, of the rotating append and of beam search,
in their plain form (elementary torch operations) and through the library.

  rope       un-rotated q, k, v of new tokens: q rotated, k rotated and v into
             their pages (4-bit pages: their rows read back)
  attention  grouped-query attention of every sequence's new tokens over pages
             held in 4 bits
  read       rows of sequences out of their pages
  beam       the best continuations of beams over the vocabulary, and the
             beams' histories and states in their new order
"""

import math

import numpy as np
import torch

own = False

HEAD = 256      # head_dim
GROUP = 4       # query heads per KV head
WINDOW = 512    # sliding layers
SCALE = 0.0625  # 256^-0.5
FULL_ROPE, FULL_THETA = 64, 5e6   # full layers rotate 64 dims
SLIDE_THETA = 1e4                 # sliding ones all 256
HIDDEN = 2560
EOS = 2
# 4-bit pages: blocks of 16 positions of a KV head, 16 rows of 128 bytes of
# codes (16-byte chunk c of row r at c ^ _TURN[r]), 16 rows of 16 scales
BLOCK = 2304
_TURN = [(r & 1) | ((r >> 2 & 3) << 1) for r in range(16)]
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one sequence's decode step in a full layer: the smallest append
        dict(name="rope b1", op="rope", x="f32", kv="bf16", n_kv=4, page=64, full=True, seqs=1, ctx_lo=701, ctx_hi=701,
             q_lo=1, q_hi=1, lens=1),
        # a decode step of 64 sequences into 4-bit pages
        dict(name="rope b64 4-bit", op="rope", x="f32", kv="fp4", n_kv=4, page=64, full=True, seqs=64, ctx_lo=512,
             ctx_hi=32768, q_lo=1, q_hi=1, lens=2),
        # chunks of prompts in a sliding layer (all 256 dims rotated), bf16 activations
        dict(name="rope 8 prompts 4-bit", op="rope", x="bf16", kv="fp4", n_kv=4, page=16, full=False, seqs=8, ctx_lo=1500,
             ctx_hi=4000, q_lo=700, q_hi=1500, lens=3),
        # one sequence, one new token at position 700: the smallest decode call
        dict(name="attention b1 pos700", op="attention", q="f32", n_kv=4, page=64, full=True, seqs=1, ctx_lo=701,
             ctx_hi=701, q_lo=1, q_hi=1, long=0, lens=4),
        # 64 sequences decoding at ragged contexts: the default serving step's full layer
        dict(name="attention b64 ctx512-32768", op="attention", q="bf16", n_kv=4, page=64, full=True, seqs=64, ctx_lo=512,
             ctx_hi=32768, q_lo=1, q_hi=1, long=0, lens=5),
        # continuous batching: 4 sequences bring chunks of prompts, the others verify up to 7 drafted tokens;
        # odd lengths, small pages, fp32 queries as the block's projections leave them
        dict(name="attention mixed b32", op="attention", q="f32", n_kv=4, page=16, full=True, seqs=32, ctx_lo=300,
             ctx_hi=6000, q_lo=1, q_hi=7, long=4, long_hi=517, lens=6),
        # a long prompt's chunk over the history before it
        dict(name="attention chunk 4096 at 4096", op="attention", q="bf16", n_kv=4, page=128, full=True, seqs=1,
             ctx_lo=8192, ctx_hi=8192, q_lo=4096, q_hi=4096, long=0, lens=7),
        # the last positions of a few sequences, to look at
        dict(name="read b5", op="read", x="f32", kv="fp4", n_kv=4, page=64, seqs=5, ctx_lo=100, ctx_hi=2000, q_lo=1,
             q_hi=9, lens=8),
        # whole prefixes leave 4-bit pages for another cache
        dict(name="read 9 prefixes", op="read", x="bf16", kv="fp4", n_kv=4, page=32, seqs=9, ctx_lo=1500, ctx_hi=9000,
             whole=True, lens=9),
        # one request of 4 beams
        dict(name="beam 1x4", op="beam", x="f32", groups=1, beams=4, vocab=131072, max_len=512, first=False, ended=0.0,
             lens=10),
        # a batch's first step: one live beam a request
        dict(name="beam first 17x5 bf16", op="beam", x="bf16", groups=17, beams=5, vocab=50257, max_len=300, first=True,
             ended=0.0, lens=11),
        # a batch of requests, some beams at their end
        dict(name="beam 32x8", op="beam", x="f32", groups=32, beams=8, vocab=131072, max_len=1024, first=False, ended=0.1,
             lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "rope", "rope", "read", "beam", "beam"])
    n_kv = rng.choice([1, 2, 3, 4, 4, 4, 5, 8])
    lens = rng.randrange(1 << 30)
    if op == "beam":
        beams = _log(rng, 1, 32)
        return dict(op=op, x=rng.choice(["f32", "bf16"]), groups=_log(rng, 1, 256 // beams), beams=beams,
                    vocab=_log(rng, 1000, 131072) | 1, max_len=_log(rng, 8, 2000), first=rng.random() < 0.2,
                    ended=rng.choice([0.0, 0.1, 0.5]), lens=lens)
    if op == "rope":
        hi = _log(rng, 1, 1500)
        return dict(op=op, x=rng.choice(["f32", "bf16"]), kv=rng.choice(["fp4", "fp4", "bf16", "f32"]), n_kv=n_kv,
                    page=rng.choice([16, 32, 48, 64, 128]), full=rng.random() < 0.5, seqs=rng.randrange(1, 33), ctx_lo=hi,
                    ctx_hi=hi + 2500, q_lo=rng.randrange(0, hi + 1), q_hi=hi, lens=lens)
    if op == "read":
        hi = _log(rng, 1, 3000)
        return dict(op=op, x=rng.choice(["f32", "bf16"]), kv=rng.choice(["fp4", "fp4", "bf16", "f32"]), n_kv=n_kv,
                    page=rng.choice([16, 48, 64]), seqs=rng.randrange(1, 20), ctx_lo=hi, ctx_hi=hi + 1000,
                    q_lo=rng.randrange(0, hi + 1), q_hi=hi, lens=lens)
    kind = rng.choice(["decode", "verify", "chunk", "mixed"])
    c = dict(op=op, q=rng.choice(["f32", "bf16"]), n_kv=n_kv, page=rng.choice([16, 32, 48, 64, 80, 128, 256]),
             full=rng.random() < 0.7, long=0, lens=lens)
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
    return c


def _lengths(c):
    """(context, new tokens) of every sequence: what the case's numbers stand for."""
    r = np.random.RandomState(c["lens"] & 0x7FFFFFFF)
    ctx = r.randint(c["ctx_lo"], c["ctx_hi"] + 1, size=c["seqs"])
    if c.get("whole"):
        return ctx, ctx.copy()
    new = r.randint(c["q_lo"], c["q_hi"] + 1, size=c["seqs"])
    if c.get("long"):
        at = r.permutation(c["seqs"])[: c["long"]]
        new[at] = r.randint(max(1, c["long_hi"] // 2), c["long_hi"] + 1, size=len(at))
    new = np.minimum(new, ctx)
    if new.sum() == 0:
        new[0] = 1
    return ctx, new


def _beams(c):
    """length, whether it has ended, and whether it is in use, of every beam."""
    r = np.random.RandomState(c["lens"] & 0x7FFFFFFF)
    n = c["groups"] * c["beams"]
    length = r.randint(1, c["max_len"], size=n)
    live = np.ones(n, dtype=bool)
    if c["first"]:
        length[:] = np.repeat(length[:: c["beams"]], c["beams"])
        live[:] = np.arange(n) % c["beams"] == 0
    return length, (r.rand(n) < c["ended"]) & (not c["first"]), live


def _pages_of(rows, page):
    return -(-rows // page)


def _row_bytes(c):
    """Bytes of one position's K (or V) of all heads."""
    return c["n_kv"] * {"fp4": HEAD // 2 + HEAD // 16, "bf16": 2 * HEAD, "f32": 4 * HEAD}[c["kv"]]


def work(case):
    c = case
    if c["op"] == "beam":
        length, ended, live = _beams(c)
        es = 4 if c["x"] == "f32" else 2
        rows = int((live & ~ended).sum())
        n = c["groups"] * c["beams"]
        moved = 8 * int(length.sum()) + 8 * HIDDEN * n
        return {"bytes": rows * c["vocab"] * es + 32 * n + moved, "flops": 4 * rows * c["vocab"]}
    ctx, new = _lengths(c)
    t = int(new.sum())
    if c["op"] == "attention":
        rows = pairs = 0
        for n, q in zip(ctx.tolist(), new.tolist()):
            if q == 0:
                continue
            seen = np.arange(n - q, n) + 1
            if not c["full"]:
                seen = np.minimum(seen, WINDOW)
            pairs += int(seen.sum())
            rows += n - (0 if c["full"] else max(0, n - q + 1 - WINDOW))
        return {"bytes": 2 * rows * c["n_kv"] * 144 + 2 * t * GROUP * c["n_kv"] * HEAD * (2 if c["q"] == "bf16" else 4),
                "flops": 4 * HEAD * GROUP * c["n_kv"] * pairs}
    xs = 4 if c["x"] == "f32" else 2
    if c["op"] == "read":
        return {"bytes": 2 * t * (_row_bytes(c) + c["n_kv"] * HEAD * xs), "flops": 0}
    half = (FULL_ROPE if c["full"] else HEAD) // 2
    b = t * c["n_kv"] * HEAD * xs * (2 * GROUP + 2) + 2 * t * _row_bytes(c) + 8 * half * t
    if c["kv"] == "fp4":  # read back in bf16
        b += 2 * t * (_row_bytes(c) + 2 * c["n_kv"] * HEAD)
    return {"bytes": b, "flops": 6 * t * half * (GROUP + 1) * c["n_kv"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype).cuda()


def _tables(ctx, page, pool, g):
    """Page tables [sequences, width] of random pages of a pool (-1: none)."""
    need = _pages_of(ctx, page)
    width = int(need.max())
    at = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    n = torch.tensor(need, device="cuda")
    start = torch.cumsum(n, 0) - n
    return torch.where(col < n[:, None], at[(start[:, None] + col).clamp(max=pool - 1)], -1)


def _fp4_blocks(n, g):
    """n blocks of rows of normally distributed values."""
    x = torch.randn(n, 16, HEAD, generator=g, device="cuda")
    code, scale = _quantize(x)
    blocks = torch.zeros(n, BLOCK, dtype=torch.uint8, device="cuda")
    turn = _dev(_TURN, torch.int64)
    place = torch.arange(8, device="cuda") ^ turn[:, None]                            # [16, 8]
    row = torch.arange(16, device="cuda")[:, None].expand(16, 8)
    blocks[:, :2048].unflatten(1, (16, 8, 16))[:, row, place] = code.unflatten(2, (8, 16))
    blocks[:, 2048:] = scale.flatten(1)
    return blocks


def _pool(c, n_pages, g):
    n_kv, page = c["n_kv"], c["page"]
    if c.get("kv", "fp4") != "fp4":
        return torch.randn((n_pages, page, n_kv, HEAD), generator=g, device="cuda", dtype=_DT[c["kv"]])
    base = _fp4_blocks(2048, g)
    at = torch.randint(0, 2048, (n_pages, page // 16, n_kv), generator=g, device="cuda")
    return base[at]


def _byte_values():
    """The two values of a byte of codes."""
    table = torch.tensor(_E2M1 + [-x for x in _E2M1], device="cuda")
    return torch.stack([table.repeat(16), table.repeat_interleave(16)], -1)


def _rope_table(n, full):
    r, theta = (FULL_ROPE, FULL_THETA) if full else (HEAD, SLIDE_THETA)
    freq = theta ** (-2.0 * torch.arange(r // 2, dtype=torch.float64, device="cuda") / r)
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.stack([ang.cos(), ang.sin()], -1).float()


def prepare(case, seed):
    c = case
    op = c["op"]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": c}
    if op == "beam":
        n, w = c["groups"] * c["beams"], c["beams"]
        length, ended, live = _beams(c)
        s["logits"] = torch.randn(n, c["vocab"], generator=g, device="cuda").mul_(2.5).to(_DT[c["x"]])
        score = -20.0 - 3.0 * torch.rand(n, generator=g, device="cuda")
        s["score"] = torch.where(_dev(live, torch.bool), score, float("-inf"))
        s["done"], s["length"] = _dev(ended), _dev(length)
        s["history"] = torch.randint(0, c["vocab"], (n, c["max_len"]), generator=g, device="cuda", dtype=torch.int32)
        s["states"] = torch.randn(n, HIDDEN, generator=g, device="cuda")
        s["new_history"], s["new_states"] = torch.zeros_like(s["history"]), torch.zeros_like(s["states"])
        s["new_score"] = torch.zeros(n, device="cuda")
        for name in ("token", "parent", "new_done", "keep_len", "new_len"):
            s[name] = torch.zeros(n, dtype=torch.int32, device="cuda")
    else:
        n_kv, page = c["n_kv"], c["page"]
        ctx, new = _lengths(c)
        pool = int(_pages_of(ctx, page).sum()) + 3
        s["k"], s["v"] = _pool(c, pool, g), _pool(c, pool, g)
        s["table"] = _tables(ctx, page, pool, g)
        s["turn"], s["two"] = _dev(_TURN, torch.int64), _byte_values()
        s["q_start"] = _dev(np.concatenate([[0], np.cumsum(new)]))
        s["seq_len"] = _dev(ctx)
        s["tokens"], s["max_q"], s["max_ctx"] = int(new.sum()), int(new.max()), int(ctx.max())
        if op == "attention":
            s["q"] = torch.randn(s["tokens"], GROUP * n_kv * HEAD, generator=g, device="cuda").to(_DT[c["q"]])
            s["out"] = torch.zeros_like(s["q"])
        elif op == "rope":  # the fused projection's rows: q | k | v
            s["qkv"] = torch.randn(s["tokens"], (GROUP + 2) * n_kv * HEAD, generator=g, device="cuda").to(_DT[c["x"]])
            s["rope"] = _rope_table(s["max_ctx"], c["full"])
            s["q_out"] = torch.zeros(s["tokens"], GROUP * n_kv * HEAD, device="cuda", dtype=_DT[c["x"]])
        if op == "read" or op == "rope" and c["kv"] == "fp4":
            dt = _DT[c["x"]] if op == "read" else torch.bfloat16
            s["k_rows"], s["v_rows"] = (torch.zeros(s["tokens"], n_kv * HEAD, device="cuda", dtype=dt) for _ in "kv")
    if own:
        _keep_handles(s)
    return s


def _keep_handles(s):
    """What a program keeps between calls: geometry, descriptors, workspaces."""
    from decode_attention_block_gb300 import binding as B
    c = s["case"]
    s["B"] = B
    if c["op"] == "beam":
        s["ws"] = B.make_beam_workspace(c["groups"], c["beams"])
        s["moves"] = [B.BeamState(s["history"], s["new_history"], positions=True, push=s["token"]),
                      B.BeamState(s["states"], s["new_states"])]
        return
    geom = s["geom"] = B.spark_geom_default()
    geom.n_kv, geom.n_q = c["n_kv"], GROUP * c["n_kv"]
    s["pool"] = B.PagePool(s["k"], s["v"])
    s["batch"] = B.PagedBatch(s["table"], s["q_start"], s["seq_len"], s["tokens"], s["max_q"])
    s["ws"] = B.make_paged_workspace(geom)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _class(s):
    return s["B"].SPARK_FULL if s["case"]["full"] else s["B"].SPARK_SLIDING


def _own_rope(s):
    B, c = s["B"], s["case"]
    q, kv = GROUP * c["n_kv"] * HEAD, c["n_kv"] * HEAD
    x = s["qkv"]
    B.spark_paged_rope_append(s["geom"], x[:, :q], x[:, q:q + kv], x[:, q + kv:], _class(s), s["rope"], s["pool"],
                              s["batch"], s["q_out"], s["ws"])
    if c["kv"] == "fp4":
        return {"q": s["q_out"], **_own_read(s)}
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _own_attention(s):
    s["B"].spark_paged_attention(s["geom"], s["q"], s["pool"], _class(s), s["batch"], s["out"], s["ws"])
    return s["out"]


def _own_read(s):
    s["B"].spark_paged_read(s["geom"], s["pool"], s["batch"], s["k_rows"], s["v_rows"], s["ws"])
    return {"k": s["k_rows"], "v": s["v_rows"]}


def _own_beam(s):
    B = s["B"]
    B.spark_beam_select(s["logits"], s["score"], s["done"], s["length"], s["case"]["beams"], EOS, s["new_score"],
                        s["token"], s["parent"], s["new_done"], s["keep_len"], s["new_len"], s["ws"])
    B.spark_beam_reorder(s["parent"], s["keep_len"], s["new_len"], s["moves"], s["ws"])
    return {k: s[k] for k in _BEAM}


_BEAM = ("new_score", "token", "parent", "new_done", "keep_len", "new_len", "new_history", "new_states")
_OWN = {"rope": _own_rope, "attention": _own_attention, "read": _own_read, "beam": _own_beam}


def _quantize(x):
    """Codes [.., 128] (two dims a byte, the lower in the low half) and scale bytes [.., 16] of rows [.., 256]."""
    y = x.float().unflatten(-1, (HEAD // 16, 16))
    top = y.abs().amax(-1, keepdim=True) / 6.0
    # five exponent, three mantissa bits: steps of 2^-3 of the power of two below, of 2^-17 at the least
    step = torch.ldexp(torch.ones_like(top), (torch.frexp(top)[1] - 1).clamp(min=-14) - 3)
    scale = ((top / step).round() * step).clamp(max=10240.0)  # 6 of them are an fp16 number
    a = torch.where(scale > 0, (y / scale).abs(), 0.0)
    code = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = (code + 8 * (y < 0)).flatten(-2)
    bits = scale[..., 0].half().view(torch.int16).int() >> 7
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), bits.to(torch.uint8)


def _values(s, code, scale):
    """What codes [.., 128] and scales [.., 16] stand for, in fp32: [.., 256]."""
    v = s["two"].index_select(0, code.flatten().int()).view(*code.shape[:-1], HEAD // 16, 16)
    f = (scale.to(torch.int16) << 7).view(torch.float16).float()
    return v.mul_(f[..., None]).flatten(-2)


def _places(s):
    """Sequence and position of every token."""
    t = torch.arange(s["tokens"], device="cuda")
    ends = s["q_start"][1:].long()
    seq = (ends <= t[:, None]).sum(1)
    return seq, s["seq_len"].long()[seq] - (ends[seq] - t)


def _fp4_at(s, pool):
    """Views of the codes [page, block, head, row, place, 16] and scales [page, block, head, row, 16]."""
    x = s[pool]
    return x[..., :2048].unflatten(3, (16, 8, 16)), x[..., 2048:].unflatten(3, (16, 16))


def _fp4_index(s, seq, pos):
    """Where rows lie: (page, block, head, row, place) of the chunks of codes, (page, block, head, row) of the scales."""
    page, n_kv = s["case"]["page"], s["case"]["n_kv"]
    pg = s["table"][seq, pos // page].long()
    blk, row = pos % page // 16, pos % 16
    head = torch.arange(n_kv, device="cuda")
    place = torch.arange(8, device="cuda") ^ s["turn"][row][:, None]
    scales = pg[:, None], blk[:, None], head, row[:, None]
    return (pg[:, None, None], blk[:, None, None], head[:, None], row[:, None, None], place[:, None]), scales


def _plain_rope(s):
    c, page = s["case"], s["case"]["page"]
    n_kv, n_q = c["n_kv"], GROUP * c["n_kv"]
    seq, pos = _places(s)
    x = s["qkv"].view(s["tokens"], n_q + 2 * n_kv, HEAD)
    turned = x[:, :n_q + n_kv].double()
    cs = s["rope"][pos].double()[:, None]
    half = cs.shape[2]
    a, b = turned[..., :half].clone(), turned[..., half:2 * half].clone()
    turned[..., :half] = a * cs[..., 0] - b * cs[..., 1]
    turned[..., half:2 * half] = b * cs[..., 0] + a * cs[..., 1]
    turned = turned.float()
    q = turned[:, :n_q].to(x.dtype).flatten(1)
    k, v = turned[:, n_q:], x[:, n_q + n_kv:].float()
    if c["kv"] != "fp4":
        at = s["table"][seq, pos // page].long(), pos % page
        s["k"][at] = k.to(s["k"].dtype)
        s["v"][at] = v.to(s["v"].dtype)
        return {"q": q, "k": s["k"], "v": s["v"]}
    for_codes, for_scales = _fp4_index(s, seq, pos)
    _put(s, "k", k, for_codes, for_scales)
    _put(s, "v", v, for_codes, for_scales)
    return {"q": q, **_plain_read(s)}


def _put(s, pool, rows, for_codes, for_scales):
    code, scale = _quantize(rows)
    codes, scales = _fp4_at(s, pool)
    codes[for_codes] = code.unflatten(2, (8, 16))
    scales[for_scales] = scale


def _plain_read(s):
    c, page = s["case"], s["case"]["page"]
    seq, pos = _places(s)
    if c["kv"] != "fp4":
        at = s["table"][seq, pos // page].long(), pos % page
        return {"k": s["k"][at].flatten(1).to(_DT[c["x"]]), "v": s["v"][at].flatten(1).to(_DT[c["x"]])}
    index = _fp4_index(s, seq, pos)
    return {"k": _get(s, "k", *index), "v": _get(s, "v", *index)}


def _get(s, pool, for_codes, for_scales):
    codes, scales = _fp4_at(s, pool)
    return _values(s, codes[for_codes].flatten(2), scales[for_scales]).flatten(1).to(s["k_rows"].dtype)


def _context(s, pool):
    """All rows of the sequences: [n, n_kv, width * page, 256] in fp32."""
    page = s["case"]["page"]
    n, width = s["table"].shape
    x = s[pool][s["table"].clamp(min=0).long()]               # [n, width, blocks, n_kv, 2304]
    x = x.permute(0, 3, 1, 2, 4).flatten(2, 3)                # [n, n_kv, blocks of the row, 2304]
    turn = torch.arange(8, device="cuda") ^ s["turn"][:, None]
    codes = x[..., :2048].unflatten(3, (16, 8, 16))
    codes = codes.gather(4, turn[..., None].expand(codes.shape))
    v = _values(s, codes.flatten(4), x[..., 2048:].unflatten(3, (16, 16)))
    return v.view(n, -1, width * page, HEAD)[:, :, :s["max_ctx"]]


def _plain_attention(s):
    c = s["case"]
    n_kv, n, t = c["n_kv"], s["table"].shape[0], s["tokens"]
    pos = torch.arange(s["max_ctx"], device="cuda")
    q0, length = s["q_start"][:-1].long(), s["seq_len"].long()
    new = s["q_start"][1:].long() - q0
    i = torch.arange(s["max_q"], device="cuda")
    tok = torch.where(i < new[:, None], q0[:, None] + i, t)  # t: a row for those that are not there
    q = s["q"].float().view(t, n_kv, GROUP, HEAD)[tok.clamp(max=t - 1)]
    at = (length - new)[:, None] + i  # position of each token
    seen = pos <= at[:, :, None]
    if not c["full"]:
        seen &= pos > at[:, :, None] - WINDOW
    seen &= pos < length[:, None, None]
    sc = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(n, n_kv, GROUP * s["max_q"], HEAD),
                      _context(s, "k").transpose(2, 3))
    sc = sc.view(n, n_kv, GROUP, s["max_q"], -1).mul_(SCALE)
    sc.masked_fill_(~seen[:, None, None], float("-inf"))
    sc.sub_(sc.amax(-1, keepdim=True)).exp_()
    sc.div_(sc.sum(-1, keepdim=True))
    v = _context(s, "v")
    v.masked_fill_(~seen.any(1)[:, None, :, None], 0.0)  # rows that no token sees may hold anything
    o = torch.matmul(sc.view(n, n_kv, GROUP * s["max_q"], -1), v)
    o = o.view(n, n_kv, GROUP, s["max_q"], HEAD).permute(0, 3, 1, 2, 4).reshape(n * s["max_q"], -1)
    out = torch.zeros(t + 1, n_kv * GROUP * HEAD, device="cuda")
    out[tok.reshape(-1)] = o
    return out[:t].to(s["q"].dtype)


def _plain_beam(s):
    c = s["case"]
    w, vocab = c["beams"], c["vocab"]
    done = s["done"] != 0
    x = s["logits"].double()
    x = x - x.amax(-1, keepdim=True)
    x = s["score"].double()[:, None] + (x - x.exp().sum(-1, keepdim=True).log())
    x[done] = float("-inf")  # an ended beam goes on as it is
    x[:, EOS] = torch.where(done, s["score"].double(), x[:, EOS])
    best, at = torch.sort(x.view(-1, w * vocab), dim=-1, descending=True, stable=True)
    best, at = best[:, :w].flatten(), at[:, :w]
    some = best > float("-inf")
    parent = (at // vocab + w * torch.arange(c["groups"], device="cuda")[:, None]).flatten()
    token = (at % vocab).flatten()
    ended = done[parent] | (token == EOS)
    keep = torch.where(some, s["length"].long()[parent], 0)
    new = torch.where(some, keep + ~done[parent], 0)
    parent, token = torch.where(some, parent, -1), torch.where(some, token, -1)
    old = parent.clamp(min=0)
    col = torch.arange(c["max_len"], device="cuda")
    hist = torch.where(col < keep[:, None], s["history"][old], s["new_history"])
    hist = torch.where((col == keep[:, None]) & (new > keep)[:, None], token.int()[:, None], hist)
    rows = torch.where(some[:, None], s["states"][old], s["new_states"])
    i32 = torch.int32
    return {"new_score": best.float(), "token": token.to(i32), "parent": parent.to(i32),
            "new_done": torch.where(some, ended, True).to(i32), "keep_len": keep.to(i32), "new_len": new.to(i32),
            "new_history": hist, "new_states": rows}


_PLAIN = {"rope": _plain_rope, "attention": _plain_attention, "read": _plain_read, "beam": _plain_beam}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _decode(blocks):
    """Rows [.., 16, 256] in 64 bits of blocks [.., 2304], from the bits."""
    b = blocks.long()
    rows = []
    for r in range(16):
        chunks = [b[..., 128 * r + 16 * (i ^ _TURN[r]): 128 * r + 16 * (i ^ _TURN[r]) + 16] for i in range(8)]
        by = torch.cat(chunks, -1)
        nib = torch.stack([by & 15, by >> 4], -1).flatten(-2)
        e, m = nib >> 1 & 3, nib & 1
        mag = torch.where(e > 0, (2.0 + m) * 2.0 ** (e - 2).double(), 0.5 * m)
        sb = b[..., 2048 + 16 * r: 2064 + 16 * r]
        se, sm = sb >> 3, (sb & 7).double()
        sc = torch.where(se > 0, (8.0 + sm) * 2.0 ** (se - 18).double(), sm * 2.0 ** -17)
        rows.append(torch.where(nib > 7, -mag, mag) * sc.repeat_interleave(16, -1))
    return torch.stack(rows, -2)


def _nearest(x):
    """4-bit values nearest to rows [.., 256] in 64 bits, the even ones of two."""
    f64 = dict(device="cuda", dtype=torch.float64)
    y = x.unflatten(-1, (16, 16))
    top = y.abs().amax(-1, keepdim=True) / 6
    grid = torch.tensor([m * 2.0 ** -17 for m in range(8)] +
                        [(8 + m) * 2.0 ** (e - 18) for e in range(1, 31) for m in range(8)], **f64)
    i = torch.searchsorted(grid, top).clamp(1, len(grid) - 1)
    down, up = top - grid[i - 1], grid[i] - top
    s = torch.where((down < up) | (down == up) & (i % 2 == 1), grid[i - 1], grid[i]).clamp(max=10240.0)
    levels, odd = torch.tensor(_E2M1, **f64), torch.arange(8, device="cuda") % 2
    far = ((y.abs() / s.clamp(min=1e-30))[..., None] - levels).abs()
    near = torch.where(far == far.amin(-1, keepdim=True), odd, 2).argmin(-1)
    return (levels[near] * s * torch.sign(y)).flatten(-2)


def exact(case, seed):
    c = case
    if c["op"] == "attention" and work(c)["flops"] > 6e11:
        return None
    s = prepare(c, seed)
    if c["op"] == "beam":
        score = []
        for i in range(c["groups"]):
            every = []
            for b in range(i * c["beams"], (i + 1) * c["beams"]):
                if bool(s["done"][b]):
                    every.append(s["score"][b:b + 1].double())
                elif bool(torch.isfinite(s["score"][b])):
                    z = torch.log_softmax(s["logits"][b].double(), 0)
                    every.append(s["score"][b].double() + torch.topk(z, min(c["beams"], c["vocab"]))[0])
            score.append(torch.topk(torch.cat(every), c["beams"])[0])
        return {**{k: None for k in _BEAM}, "new_score": torch.cat(score)}
    page, n_kv = c["page"], c["n_kv"]
    ctx, new = s["seq_len"].tolist(), np.diff(s["q_start"].cpu().numpy()).tolist()

    def rows(pool, b, n):
        x = s[pool][s["table"][b, : -(-n // page)].long()]
        if c.get("kv", "fp4") == "fp4":
            return _decode(x).transpose(2, 3).reshape(-1, n_kv, HEAD)[:n]
        return x.reshape(-1, n_kv, HEAD)[:n].double()

    if c["op"] == "read":
        return {p: torch.cat([rows(p, b, n)[n - m:] for b, (n, m) in enumerate(zip(ctx, new))]).flatten(1) for p in "kv"}
    if c["op"] == "rope":
        pos = torch.cat([torch.arange(n - m, n, device="cuda") for n, m in zip(ctx, new)])
        x = s["qkv"].double().view(len(pos), -1, HEAD)
        z = torch.view_as_complex(s["rope"].double())[pos][:, None]
        half, n_q = z.shape[2], GROUP * n_kv
        w = torch.complex(x[:, :n_q + n_kv, :half], x[:, :n_q + n_kv, half:2 * half]) * z
        y = torch.cat([w.real, w.imag, x[:, :n_q + n_kv, 2 * half:]], -1)
        out = {"q": y[:, :n_q].flatten(1)}
        for pool, r in (("k", y[:, n_q:]), ("v", x[:, n_q + n_kv:])):
            if c["kv"] == "fp4":
                out[pool] = torch.cat([_nearest(part) for part in r.split(256)]).flatten(1)
            else:
                out[pool] = s[pool].double()
                t = 0
                for b, (n, m) in enumerate(zip(ctx, new)):
                    at = torch.arange(n - m, n, device="cuda")
                    out[pool][s["table"][b, at // page].long(), at % page] = r[t:t + m]
                    t += m
        return out
    out = torch.zeros(s["tokens"], n_kv, GROUP, HEAD, dtype=torch.float64, device="cuda")
    t = 0
    for b, (n, m) in enumerate(zip(ctx, new)):
        if m == 0:
            continue
        k, v = rows("k", b, n), rows("v", b, n)
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
