"""The norms called from several host threads at once: each call's launch stands
on its own, whatever shapes the other threads' calls have."""
import ctypes
import threading

import pytest
import torch

from gpu_util import DEV, require_gpu
from moe_grouped_block_gb300 import mxg

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
CALLS = 30000


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


class Calls:
    """The library's entry point for one shape, with nothing between two calls: the
    arguments are recorded once from a call through the binding."""

    def __init__(self, way, rows, cols, monkeypatch):
        g = torch.Generator(device=DEV).manual_seed(cols)
        new = lambda: torch.randn(rows, cols, generator=g, device=DEV).to(BF)  # noqa: E731
        w, ws = torch.ones(cols, dtype=BF, device=DEV), mxg.alloc_block_norm_workspace(rows, cols)
        self.stream = torch.cuda.Stream()
        x, y, a, b = new(), new(), new(), new()
        self.out = [torch.empty_like(x), torch.empty_like(x)]
        self.keep = (x, y, a, b, w, ws)
        lib, name = mxg.load(), "mxg_block_norm" + ("" if way == "forward" else "_backward")
        fn = getattr(lib, name)

        class Recorder:
            def __getattr__(_, entry):
                def call(*args):
                    self.args = [getattr(v, "_obj", v) for v in args]
                    return 0
                return call
        with monkeypatch.context() as m:
            m.setattr(mxg, "load", lambda: Recorder())
            if way == "forward":
                mxg.mxg_block_norm(x, y, w, None, 0, 1.0, self.out[0], w, self.out[1], 1e-5,
                                   stream=self.stream)
            else:
                mxg.mxg_block_norm_backward(x, y, w, None, 0, 1.0, w, 1e-5, a, b, *self.out, None,
                                            None, None, ws, stream=self.stream)
        args = [ctypes.byref(v) if isinstance(v, ctypes.Structure) else v for v in self.args]
        self.call = lambda: fn(*args)
        torch.cuda.synchronize()
        assert self.call() == 0
        torch.cuda.synchronize()
        self.want = [t.clone() for t in self.out]
        self.codes = {}

    def work(self, start):
        start.wait()
        for i in range(CALLS):
            code = self.call()
            self.codes[code] = self.codes.get(code, 0) + 1
            if i % 256 == 255:
                self.stream.synchronize()
        self.stream.synchronize()


@pytest.mark.parametrize("way", ["forward", "backward"])
def test_shapes_of_one_kernel_from_several_threads(way, monkeypatch):
    """Single rows of widths that run the same kernel with different amounts of shared
    memory: 64, 42 and 42 KB."""
    calls = [Calls(way, 1, cols, monkeypatch) for cols in (16384, 10496, 10624)]
    start = threading.Barrier(len(calls))
    threads = [threading.Thread(target=c.work, args=(start,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert [c.codes for c in calls] == [{0: CALLS}] * len(calls)
    for c in calls:
        assert all(torch.equal(a, b) for a, b in zip(c.out, c.want))
