"""Host checks of the paged cache beside ``test_host_paged.py`` (no GPU): the
work list's arithmetic for groups of eight tokens, and tensors of another
device than the current one, which the binding refuses before a call."""

import shutil
import subprocess

import pytest
import torch

from test_host_paged import CSRC, PROGRAM, B  # noqa: F401


def test_index_arithmetic_of_eight_token_groups(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    old = ("for (int step : {1, 4, 32})", "const Shape shapes[] = {{1, 16, 0},")
    new = ("for (int step : {8, 64})", "const Shape shapes[] = {{8, 16, 0}, {8, 16, 7}, {8, 16, 512}, {8, 16, INT32_MAX}, {1, 16, 0},")
    text = PROGRAM
    for a, b in zip(old, new):
        assert text.count(a) == 1
        text = text.replace(a, b)
    src, exe = tmp_path / "paged.cpp", tmp_path / "paged"
    src.write_text(text)
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I", CSRC,
                    str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout[-3000:] + res.stderr[-2000:]


# -- devices -------------------------------------------------------------------

class OnDevice(torch.Tensor):
    """A tensor that says it lies on a GPU."""
    dev = 0
    is_cuda = True

    def get_device(self):
        return self.dev


def _t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


def _calls(B):
    """Name -> (call, its tensors): calls whose tensors all lie on device 0."""
    g = B.spark_geom_default()
    i32 = torch.int32

    def case():
        return dict(pk=_t(2, 16, 4, 256), pv=_t(2, 16, 4, 256), table=_t(1, 2, dtype=i32), q_start=_t(2, dtype=i32),
                    seq_len=_t(1, dtype=i32), ws=_t(256, dtype=torch.uint8))

    def pool(c):
        return B.PagePool(c["pk"], c["pv"])

    def batch(c):
        return B.PagedBatch(c["table"], c["q_start"], c["seq_len"], 3, 3)

    def append(c):
        B.spark_paged_append(g, c["k"], c["v"], pool(c), batch(c), c["ws"])

    def attention(c):
        B.spark_paged_attention(g, c["q"], pool(c), B.SPARK_FULL, batch(c), c["a"], c["ws"])

    def block(c):
        w = B.LayerWeights(c["norm_w"], c["qkv_w"], c["g_w"], c["o_w"])
        B.spark_attn_paged(g, c["h"], w, pool(c), B.SPARK_FULL, batch(c), [0, 1, 2], c["out"], c["ws"], c["pws"])

    def remap(c):
        B.spark_pages_remap(g, [pool(c)], c["table"], c["parent"], c["keep"], c["new"], c["new_table"], c["ws"])

    def compact(c):
        B.spark_pages_compact(g, [pool(c)], c["table"], c["new_table"], c["n_live"], c["ws"])

    def scores(c):
        B.spark_token_logprobs(c["logits"], c["targets"], c["logprob"], c["entropy"], c["ids"], c["top"], c["ws"])

    tables = {k: v for k, v in case().items() if k in ("pk", "pv", "table", "ws")}
    return {
        "append": (append, dict(case(), k=_t(3, 1024), v=_t(3, 1024))),
        "attention": (attention, dict(case(), q=_t(3, 4096), a=_t(3, 4096))),
        "block": (block, dict(case(), h=_t(3, 2560), out=_t(3, 2560), pws=_t(256, dtype=torch.uint8), norm_w=_t(8),
                              qkv_w=_t(8), g_w=_t(8), o_w=_t(8))),
        "remap": (remap, dict(tables, parent=_t(1, dtype=i32), keep=_t(1, dtype=i32), new=_t(1, dtype=i32),
                              new_table=_t(1, 2, dtype=i32))),
        "compact": (compact, dict(tables, new_table=_t(1, 2, dtype=i32), n_live=_t(1, dtype=i32))),
        "scores": (scores, dict(logits=_t(3, 50), targets=_t(3, dtype=i32), logprob=_t(3), entropy=_t(3),
                                ids=_t(3, 2, dtype=i32), top=_t(3, 2), ws=_t(256, dtype=torch.uint8))),
    }


@pytest.mark.parametrize("name", ["append", "attention", "block", "remap", "compact", "scores"])
def test_tensors_of_another_device_are_refused(B, name, monkeypatch):
    call, tensors = _calls(B)[name]
    reached = []

    class Lib:
        def __getattr__(self, entry):
            return lambda *args: reached.append(entry) or 0
    monkeypatch.setattr(B, "load", lambda: Lib())
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_stream", lambda stream: 0)
    call(tensors)
    assert len(reached) == 1                       # all on the current device: the library is called
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
