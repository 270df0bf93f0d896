"""Calls of the expert rows that name no rows, without a GPU."""
import pytest
import torch

from moe_grouped_block_gb300 import mxg


def test_rows_are_needed(monkeypatch):
    """Passed on as a buffer of no rows, nothing would be moved, and sums and gradients would be 0."""
    called = []
    monkeypatch.setattr(mxg, "load", lambda: type("Lib", (), {
        "__getattr__": lambda self, name: lambda *args: called.append(name) or 0})())
    monkeypatch.setattr(mxg, "_here", lambda: -1)  # where tensors of the CPU are
    monkeypatch.setattr(mxg, "_stream_on", lambda stream, here: 7)
    x, at = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: mxg.mxg_dispatch(x, at, None), lambda: mxg.mxg_combine(None, at, x),
                 lambda: mxg.mxg_combine_backward(x, at, None, None, dweight=torch.zeros(4, 2))):
        with pytest.raises(ValueError):
            call()
    assert called == []
    none = torch.zeros(0, 16)  # a buffer without rows is one
    mxg.mxg_dispatch(x, at, none)
    mxg.mxg_combine(none, at, x)
    mxg.mxg_combine_backward(x, at, None, None, y_rows=none, dweight=torch.zeros(4, 2))
    assert called == ["mxg_dispatch", "mxg_combine", "mxg_combine_backward"]
