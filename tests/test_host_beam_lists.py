"""Lists of slots that are no lists (no GPU): refused by the binding, which hands
the library their length."""

import pytest
import torch

from test_host_paged import B  # noqa: F401
from test_host_paged_limits import _t


@pytest.mark.parametrize("shape", [(2, 2), (4, 1), ()])
def test_parents_are_a_list(B, shape, monkeypatch):
    reached = []

    class Lib:
        def __getattr__(self, entry):
            return lambda *args: reached.append(entry) or 0
    monkeypatch.setattr(B, "load", lambda: Lib())
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_stream", lambda stream: 0)
    i32 = torch.int32
    rows = shape[0] if shape else 1
    state = B.BeamState(_t(rows, 9, dtype=i32), _t(rows, 9, dtype=i32))
    lists = [_t(shape, dtype=i32) for _ in range(3)]
    for lengths in (lists[1:], [None, None]):
        with pytest.raises(ValueError, match="parent must be"):
            B.spark_beam_reorder(lists[0], *lengths, [state], _t(256, dtype=torch.uint8))
    with pytest.raises(TypeError, match="parent"):
        B.spark_beam_reorder(None, None, None, [state], _t(256, dtype=torch.uint8))
    assert not reached
