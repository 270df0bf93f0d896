"""Workspaces and status words that the binding of the routing operators refuses, without a GPU:
kernels would write past them or between the elements of a view."""
import pytest
import torch

from moe_grouped_block_gb300 import mxg

I32, U8 = torch.int32, torch.uint8


@pytest.fixture
def calls(monkeypatch):
    """What the library is called with."""
    seen = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *args: seen.append((name, args)) or 0
    monkeypatch.setattr(mxg, "load", lambda: Recorder())
    monkeypatch.setattr(mxg, "_here", lambda: -1)  # where tensors of the CPU are
    monkeypatch.setattr(mxg, "_stream_on", lambda stream, here: 7)
    return seen


def route(**kw):
    mxg.mxg_route(torch.zeros(10, 8), torch.zeros(10, 2, dtype=I32), torch.zeros(10, 2),
                  torch.zeros(8, dtype=I32), **kw)


def route_rows(**kw):
    mxg.mxg_route_rows(torch.zeros(10, 2, dtype=I32), torch.zeros(8, dtype=I32), **kw)


@pytest.mark.parametrize("call", [route, route_rows])
def test_workspaces(calls, call):
    whole = torch.zeros(4096, dtype=U8)
    # nbytes counts a view's elements, not the memory between or behind them
    for bad in (whole[::2], torch.zeros(1, dtype=U8).expand(4096), torch.zeros(64, 64, dtype=U8)[:, :32]):
        with pytest.raises(ValueError):
            call(workspace=bad)
    assert calls == []
    for ok in (whole, whole[16:], whole.view(I32), whole.view(64, 64)):
        call(workspace=ok)
        args = calls.pop()[1]
        assert ok.data_ptr() in args and ok.nbytes in args


@pytest.mark.parametrize("call", [route, route_rows])
def test_status_words(calls, call):
    ws = torch.zeros(4096, dtype=U8)
    for bad in (torch.zeros(1, dtype=U8), torch.zeros(0, dtype=I32), torch.zeros(1, dtype=torch.int64),
                torch.zeros(4, dtype=U8), torch.zeros(1)):
        with pytest.raises(ValueError):
            call(workspace=ws, dev_status=bad)
    assert calls == []
    three = torch.zeros(3, dtype=I32)
    for ok in (three, three[1:2], three[2]):
        call(workspace=ws, dev_status=ok)
        assert ok.data_ptr() in calls.pop()[1]
    call(workspace=ws, dev_status=three.data_ptr())  # an address, as the other calls take it
    assert three.data_ptr() in calls.pop()[1]
    call(workspace=ws)
    assert calls.pop()[1][-2:] == (0, 7)
