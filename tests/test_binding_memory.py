"""Workspaces and status words that the binding of the block-scaled and 16-bit operators refuses,
without a GPU: kernels would write past them or between the elements of a view."""
import pytest
import torch

from moe_grouped_block_gb300 import mxg

BF, I32, I64, U8 = torch.bfloat16, torch.int32, torch.int64, torch.uint8


@pytest.fixture
def calls(monkeypatch):
    """The names of the library's entry points that are called."""
    seen = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *args: seen.append(name) or 0
    monkeypatch.setattr(mxg, "load", lambda: Recorder())
    monkeypatch.setattr(mxg, "_p", lambda t: t if t is None or isinstance(t, int) else t.data_ptr())
    monkeypatch.setattr(mxg, "_s", lambda stream: None)
    return seen


def norm_backward(ws):
    x = torch.zeros(4, 64, dtype=BF)
    mxg.mxg_block_norm_backward(x, dn=x.clone(), dx=x.clone(), w_pre=x[0].contiguous(), workspace=ws)


def grads(ws):
    return mxg.GradList([], []), torch.zeros(1), ws


WORKSPACE = {"norm_backward": norm_backward, "grad_norm": lambda ws: mxg.mxg_grad_norm(*grads(ws)),
             "grad_clip": lambda ws: mxg.mxg_grad_clip(grads(ws)[0], 1.0, *grads(ws)[1:])}


@pytest.mark.parametrize("name", WORKSPACE)
def test_workspaces(calls, name):
    whole = torch.zeros(4096, dtype=U8)
    for bad in (whole[::2], torch.zeros(1, dtype=U8).expand(4096), torch.zeros(64, 64, dtype=U8)[:, :32]):
        with pytest.raises(ValueError):
            WORKSPACE[name](bad)
    assert calls == []
    WORKSPACE[name](whole)
    WORKSPACE[name](whole.view(64, 64))
    assert len(calls) == 2


def status_calls(st):
    u8, ws, x = torch.zeros(1, dtype=U8), torch.zeros(9, dtype=I64), torch.zeros(128, 128, dtype=BF)
    ab, sizes = (u8, u8), torch.zeros(4, dtype=I32)
    for fn in (mxg.mxg_group_offsets, mxg.mxg_group_offsets_unaligned):
        yield lambda fn=fn: fn(sizes, 1, 128, 512, ws, st)
    yield lambda: mxg.mxg_group_quantize(1, 1, x, 128, 128, ws, 4, u8, u8, dev_status=st)
    yield lambda: mxg.mxg_group_quantize_unaligned(1, x, 128, 128, ws, 4, u8, u8, dev_status=st)
    yield lambda: mxg.mxg_grouped_gemm(1, 0, ab, ab, ws, 4, 128, 128, 128, C=x, dev_status=st)
    yield lambda: mxg.mxg_grouped_gemm_debug(1, 0, ab, ab, ws, 4, 128, 128, 128, C=x, dev_status=st)
    yield lambda: mxg.mxg_grouped_gemm_unaligned(0, ab, ab, ws, 4, 128, 128, 128, C=x, dev_status=st)
    yield lambda: mxg.mxg_grouped_gemm_16bit(0, x, x.expand(4, 128, 128).contiguous(), ws, 4, 128, 128, 128,
                                             C=x, dev_status=st)


def test_status_words(calls):
    for bad in (torch.zeros(1, dtype=U8), torch.zeros(4, dtype=U8), torch.zeros(0, dtype=I32)):
        for call in status_calls(bad):
            with pytest.raises(ValueError):
                call()
    assert calls == []
    for ok in (torch.zeros(1, dtype=I32), torch.zeros(3, dtype=I32)[1], torch.zeros(1, dtype=I64), None, 4096):
        for call in status_calls(ok):
            call()
    assert len(calls) == 5 * 8
