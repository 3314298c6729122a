"""Host checks of 4-bit pages, the rotating append and beam search (no GPU):
every status is decided before anything touches a device, and the binding
refuses what the library cannot see."""

import ctypes

import pytest
import torch

import fp4_ref
from test_host_paged import BAD_BATCHES, BAD_POOLS, FAKE, B, _append, _attention, _batch, _pages, _pool  # noqa: F401
from test_host_paged_limits import _t


def test_4_bit_pools_are_pools(B):
    fp4 = dict(dtype=B.SPARK_FP4)
    for kw, want in BAD_POOLS:
        if "dtype" not in kw:
            assert _attention(B, pool=_pool(B, **fp4, **kw)) == want and _append(B, pool=_pool(B, **fp4, **kw)) == want
            for compact in (False, True):
                assert _pages(B, compact, pools=[_pool(B, **fp4), _pool(B, **fp4, **kw)]) == want
    # they pass every check but the workspace's
    assert _attention(B, pool=_pool(B, **fp4), ws=0) == -4 and _append(B, pool=_pool(B, **fp4), ws=0) == -4
    assert _pages(B, False, pools=[_pool(B, **fp4)], ws=0) == -4
    assert _pages(B, False, pools=[_pool(B, **fp4), _pool(B)]) == -1
    # 4 bits are no type of queries or rows
    assert _attention(B, dtype=2) == -1 and _append(B, dtype=2) == -1


def _rope(B, q=FAKE, k=FAKE + 16384, v=FAKE + 20480, ld=6144, dtype=0, cls=1, rope=FAKE, n_pos=100, pool=None, batch=None,
          out=FAKE + (1 << 30), old=4096, ws=FAKE, nbytes=None, geom=None):
    g = geom or B.spark_geom_default()
    nbytes = B.spark_paged_workspace_bytes(B.spark_geom_default()) if nbytes is None else nbytes
    return B.load().spark_paged_rope_append(ctypes.byref(g), q, k, v, ld, dtype, cls, rope, n_pos,
                                            ctypes.byref(pool or _pool(B)), ctypes.byref(batch or _batch(B)), out, old, ws,
                                            nbytes, None)


def test_rope_append_arguments_are_validated(B):
    ok = dict(ws=0)                                       # all else in order: the workspace is looked at last
    assert _rope(B, **ok) == -4 and _rope(B, q=0, out=0, old=0, **ok) == -4
    assert _rope(B, out=FAKE, old=6144, **ok) == -4       # in place
    for kw in (dict(k=0), dict(v=FAKE + 8), dict(q=FAKE + 4), dict(out=0), dict(out=FAKE + (1 << 30) + 8), dict(ld=4092),
               dict(ld=6146), dict(ld=6148, dtype=1), dict(dtype=2), dict(cls=2), dict(rope=0), dict(rope=FAKE + 8), dict(n_pos=0),
               dict(n_pos=(1 << 24) + 1), dict(old=4092), dict(old=4098),
               dict(out=FAKE, old=8192),                  # over q, other rows
               dict(out=FAKE + 16, old=6144), dict(out=FAKE + 16384, old=6144), dict(out=FAKE + 8 * 6144 * 4, old=6144),
               dict(q=FAKE, out=FAKE, old=6144, k=FAKE + 8192)):   # k inside q's rows, rotated in place
        assert _rope(B, **{**ok, **kw}) == -1, kw
    # behind the last of 9 rows it is free
    assert _rope(B, out=FAKE + 8 * 6144 * 4 + 24576, old=4096, **ok) == -4
    assert _rope(B, nbytes=100) == -4 and _rope(B, ws=FAKE + 16) == -4
    for kw, want in BAD_POOLS:
        assert _rope(B, pool=_pool(B, **kw)) == want, kw
    for kw, want in BAD_BATCHES:
        assert _rope(B, batch=_batch(B, **kw)) == want, kw
    g = B.spark_geom_default()
    g.full_rotary_dim = 63
    assert _rope(B, geom=g) == -5


def test_read_arguments_are_validated(B):
    g = B.spark_geom_default()
    need = B.spark_paged_workspace_bytes(g)

    def call(pool=None, batch=None, k=FAKE, v=FAKE + (1 << 20), ld=1024, dtype=0, ws=FAKE, nbytes=need):
        return B.load().spark_paged_read(ctypes.byref(g), ctypes.byref(pool or _pool(B)), ctypes.byref(batch or _batch(B)), k, v,
                                         ld, dtype, ws, nbytes, None)
    for kw, want in BAD_POOLS:
        assert call(pool=_pool(B, **kw)) == want, kw
    for kw, want in BAD_BATCHES:
        assert call(batch=_batch(B, **kw)) == want, kw
    for kw in (dict(k=0), dict(v=0), dict(k=FAKE + 8), dict(ld=1020), dict(ld=1026), dict(dtype=2), dict(v=FAKE), dict(v=FAKE + 4080),
               dict(v=FAKE + 4096 * 8)):
        assert call(**kw) == -1, kw
    assert call(ws=0) == -4 and call(nbytes=need - 1) == -4
    assert call(ld=2048, v=FAKE + 4096, ws=0) == -4       # slices of the same rows


def test_rope_table_arguments_are_validated(B):
    g = B.spark_geom_default()
    call = B.load().spark_rope_table
    assert call(ctypes.byref(g), 2, 10, FAKE, None) == -1 and call(ctypes.byref(g), 1, 0, FAKE, None) == -1
    assert call(ctypes.byref(g), 1, (1 << 24) + 1, FAKE, None) == -1 and call(ctypes.byref(g), 1, 10, 0, None) == -1
    assert call(ctypes.byref(g), 1, 10, FAKE + 8, None) == -1
    g.head_dim = 64
    assert call(ctypes.byref(g), 1, 10, FAKE, None) == -5


def test_beam_select_arguments_are_validated(B):
    need = B.spark_beam_workspace_bytes(2, 4)

    def call(x=FAKE, ld=1000, dtype=0, groups=2, W=4, vocab=1000, score=FAKE, done=FAKE, length=FAKE, eos=3, new_score=FAKE,
             token=FAKE, parent=FAKE, new_done=FAKE, keep=FAKE, new=FAKE, ws=FAKE, nbytes=need):
        return B.load().spark_beam_select(x, ld, dtype, groups, W, vocab, score, done, length, eos, new_score, token, parent,
                                          new_done, keep, new, ws, nbytes, None)
    for kw in (dict(x=0), dict(x=FAKE + 2), dict(ld=999), dict(ld=(1 << 40) + 1), dict(dtype=2), dict(groups=0), dict(W=0),
               dict(W=33), dict(groups=257), dict(groups=(1 << 30) + 1), dict(vocab=0), dict(vocab=(1 << 24) + 1, ld=1 << 25),
               dict(score=0), dict(score=FAKE + 2), dict(eos=-2), dict(eos=1000), dict(eos=-1), dict(new_done=0), dict(new_score=0),
               dict(token=0), dict(parent=FAKE + 1), dict(length=0), dict(keep=0), dict(new=0), dict(done=FAKE + 2)):
        assert call(**kw) == -1, kw
    for kw in (dict(), dict(eos=-1, done=0), dict(eos=-1, done=0, new_done=0), dict(length=0, keep=0, new=0), dict(done=0)):
        assert call(**kw, ws=0) == -4, kw
    assert call(ws=FAKE + 64) == -4 and call(nbytes=need - 1) == -4
    for groups, W in ((0, 1), (1, 0), (1, 33), (1025, 1), (33, 32)):
        assert B.spark_beam_workspace_bytes(groups, W) == 0
    assert B.spark_beam_workspace_bytes(32, 32) > 0


def test_beam_reorder_arguments_are_validated(B):
    need = B.spark_beam_workspace_bytes(1, 1)

    def call(parent=FAKE, keep=FAKE, new=FAKE, n=4, states=None, ws=FAKE, nbytes=need, **kw):
        f = dict(src=FAKE, dst=FAKE + (1 << 20), pitch=400, elem=0, push=0)
        f.update(kw)
        states = [B.SparkBeamState(*f.values())] if states is None else states
        return B.load().spark_beam_reorder(parent, keep, new, n, (B.SparkBeamState * max(1, len(states)))(*states), len(states),
                                           ws, nbytes, None)
    for kw in (dict(parent=0), dict(parent=FAKE + 2), dict(n=0), dict(n=1025), dict(states=[]), dict(src=0), dict(dst=0),
               dict(src=FAKE + 2), dict(pitch=0), dict(pitch=402), dict(pitch=1 << 31), dict(elem=-4), dict(elem=6), dict(elem=404),
               dict(push=FAKE), dict(push=FAKE, elem=8), dict(push=FAKE + 2, elem=4), dict(elem=4, keep=0), dict(elem=4, new=0),
               dict(dst=FAKE), dict(dst=FAKE + 1596), dict(dst=FAKE - 1596), dict(keep=FAKE + 2)):
        assert call(**kw) == -1, kw
    one = B.SparkBeamState(FAKE, FAKE + (1 << 20), 400, 0, 0)
    far = [B.SparkBeamState(FAKE, FAKE + (i << 20), 400, 0, 0) for i in range(1, 34)]
    assert call(states=far) == -1 and call(states=far[:32], ws=0) == -4
    # what is written is read or written nowhere else in the call
    at = FAKE + (2 << 20)
    other = lambda **kw: B.SparkBeamState(*dict(dict(src=at, dst=at + (1 << 20), pitch=400, elem=4, push=0), **kw).values())  # noqa: E731
    assert call(states=[one, other()], ws=0) == -4
    for kw in (dict(src=FAKE + (1 << 20) + 1596), dict(dst=FAKE + (1 << 20) - 1596), dict(dst=FAKE + 1596),
               dict(push=FAKE + (1 << 20) + 1596), dict(push=at + (1 << 20) - 12)):
        assert call(states=[one, other(**kw)], ws=0) == -1, kw
    inside = FAKE + (1 << 20) + 1584
    for kw in (dict(parent=inside), dict(keep=inside), dict(new=inside)):
        assert call(**kw, ws=0) == -1 and call(**{k: v + 16 for k, v in kw.items()}, ws=0) == -4
    assert call(dst=FAKE + 1600, ws=0) == -4 and call(keep=0, new=0, ws=0) == -4 and call(nbytes=need - 1) == -4


# -- the binding -----------------------------------------------------------------

def _calls(B):
    g, i32, u8 = B.spark_geom_default(), torch.int32, torch.uint8

    def pages(**kw):
        return dict(pk=_t(2, 1, 4, 2304, dtype=u8), pv=_t(2, 1, 4, 2304, dtype=u8), table=_t(1, 2, dtype=i32),
                    q_start=_t(2, dtype=i32), seq_len=_t(1, dtype=i32), ws=_t(256, dtype=u8), **kw)

    def batch(c):
        return B.PagedBatch(c["table"], c["q_start"], c["seq_len"], 3, 3)

    def rope(c):
        B.spark_paged_rope_append(g, c["q"], c["k"], c["v"], B.SPARK_FULL, c["rope"], B.PagePool(c["pk"], c["pv"]), batch(c),
                                  c["q_out"], c["ws"])

    def read(c):
        B.spark_paged_read(g, B.PagePool(c["pk"], c["pv"]), batch(c), c["k"], c["v"], c["ws"])

    def table(c):
        B.spark_rope_table(g, B.SPARK_FULL, c["rope"])

    def attention(c):
        B.spark_paged_attention(g, c["q"], B.PagePool(c["pk"], c["pv"]), B.SPARK_FULL, batch(c), c["a"], c["ws"])

    def select(c):
        B.spark_beam_select(c["logits"], c["score"], c["done"], c["length"], 2, 1, c["new_score"], c["token"], c["parent"],
                            c["new_done"], c["keep"], c["new"], c["ws"])

    def reorder(c):
        B.spark_beam_reorder(c["parent"], c["keep"], c["new"], [B.BeamState(c["src"], c["dst"], positions=True, push=c["push"])],
                             c["ws"])
    lists = {k: _t(4, dtype=i32) for k in ("done", "length", "token", "parent", "new_done", "keep", "new")}
    return {
        "rope": (rope, pages(q=_t(3, 4096), k=_t(3, 1024), v=_t(3, 1024), q_out=_t(3, 4096), rope=_t(50, 32, 2))),
        "read": (read, pages(k=_t(3, 1024), v=_t(3, 1024))),
        "table": (table, dict(rope=_t(50, 32, 2))),
        "attention": (attention, pages(q=_t(3, 4096), a=_t(3, 4096))),
        "select": (select, dict(lists, logits=_t(4, 50), score=_t(4), new_score=_t(4), ws=_t(256, dtype=u8))),
        "reorder": (reorder, dict(parent=_t(4, dtype=i32), keep=_t(4, dtype=i32), new=_t(4, dtype=i32), src=_t(4, 9, dtype=i32),
                                  dst=_t(4, 9, dtype=i32), push=_t(4, dtype=i32), ws=_t(256, dtype=u8))),
    }


@pytest.mark.parametrize("name", ["rope", "read", "table", "attention", "select", "reorder"])
def test_tensors_of_another_device_are_refused(B, name, monkeypatch):
    from test_host_paged_limits import OnDevice
    call, tensors = _calls(B)[name]
    if name == "rope":  # slices of a fused projection's rows
        x = _t(3, 6144)
        tensors.update(q=x[:, :4096], k=x[:, 4096:5120], v=x[:, 5120:])
    reached = []

    class Lib:
        def __getattr__(self, entry):
            return lambda *args: reached.append(entry) or 0
    monkeypatch.setattr(B, "load", lambda: Lib())
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_stream", lambda stream: 0)
    call(tensors)
    assert len(reached) == 1
    for which in tensors:
        moved = dict(tensors)
        moved[which] = tensors[which].clone().as_subclass(OnDevice)
        moved[which].dev = 1
        with pytest.raises(ValueError, match="device"):
            call(moved)
    monkeypatch.setattr(B, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="device"):
        call(tensors)
    assert len(reached) == 1


def test_shapes_and_types_are_refused(B, monkeypatch):
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_stream", lambda stream: 0)

    def bad(name, match, **kw):
        call, tensors = _calls(B)[name]
        with pytest.raises((ValueError, TypeError), match=match):
            call({**tensors, **kw})
    x = _t(3, 6144)
    same = dict(q=x[:, :4096], k=x[:, 4096:5120], v=x[:, 5120:])
    bad("rope", "row stride")                                             # q, k and v of their own
    bad("rope", "rope must be", **same, rope=_t(50, 128, 2))
    bad("rope", "same dtype", **same, q_out=_t(3, 4096, dtype=torch.bfloat16))
    bad("rope", "n_tokens", **{**same, "q": x[:2, :4096]})
    bad("rope", "2304", **same, pk=_t(2, 1, 4, 2300, dtype=torch.uint8), pv=_t(2, 1, 4, 2300, dtype=torch.uint8))
    bad("rope", "heads", **same, pk=_t(2, 1, 3, 2304, dtype=torch.uint8), pv=_t(2, 1, 3, 2304, dtype=torch.uint8))
    bad("read", "n_tokens", k=_t(3, 1000), v=_t(3, 1000))
    bad("read", "same dtype", v=_t(3, 1024, dtype=torch.bfloat16))
    bad("table", "rope must be", rope=_t(50, 64))
    bad("select", "done must be", done=_t(3, dtype=torch.int32))
    bad("select", "int32", token=_t(4))
    bad("select", "each beam", logits=_t(5, 50))
    bad("reorder", "a row for each slot", parent=_t(5, dtype=torch.int32))
    bad("reorder", "push must be", src=_t(4, 9), dst=_t(4, 9))
    bad("reorder", "src and dst", dst=_t(4, 8, dtype=torch.int32))


def test_the_plain_format_keeps_what_it_can(B):
    """The reference the GPU tests use: every value of the format is its own
    nearest, and a quotient is at most half a step away."""
    code = torch.arange(16).repeat(16)
    code[7::16] = 7                                  # a 6 in every group: its scale is found again
    for b in (1, 7, 8, 0x70, 0x91, 0xE2):
        v = fp4_ref.values(code[None], torch.full((1, 16), b))
        again = fp4_ref.quantize(v)
        assert torch.equal(again[1], torch.full((1, 16), b)) and torch.equal(fp4_ref.values(*again), v)
    g = torch.Generator().manual_seed(0)
    x = torch.randn(200, 256, generator=g, dtype=torch.float64) * 10 ** torch.randn(200, 1, generator=g, dtype=torch.float64)
    x = x.float().double()
    v = fp4_ref.values(*fp4_ref.quantize(x))
    m = x.unflatten(-1, (16, 16)).abs().amax(-1, keepdim=True).expand(200, 16, 16).flatten(1)
    # steps of 2 up to 6 below the scale, which is m / 6 within 2^-4 (2^-18 at the least)
    assert bool(((x - v).abs() <= m / 6 * (1 + 2.0 ** -4) + m * 2.0 ** -4 + 2.0 ** -15).all())
    assert [fp4_ref.turn(r) for r in range(16)] == [0, 1, 0, 1, 2, 3, 2, 3, 4, 5, 4, 5, 6, 7, 6, 7]
