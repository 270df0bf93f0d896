"""What the binding of the routing, row and activation operators passes on and what it
refuses, without a GPU: the library is replaced by a recorder of the descriptors."""
import ctypes

import pytest
import torch

from moe_grouped_block_gb300 import mxg

BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
DESC = {"mxg_route": mxg.Route, "mxg_route_backward": mxg.RouteGrad, "mxg_dispatch": mxg.ExpertRows,
        "mxg_combine": mxg.ExpertRows, "mxg_combine_backward": mxg.ExpertRows,
        "mxg_gated_act": mxg.GatedAct, "mxg_gated_act_backward": mxg.GatedAct}


class Recorder:
    """Stands in for the loaded library: keeps each call's descriptor and other arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            if name in DESC:
                d = DESC[name].from_buffer_copy(args[0].ljust(ctypes.sizeof(DESC[name]), b"\0"))
                self.calls.append((d, args[1:]))
            else:
                self.calls.append((None, args))
            return 0
        return entry


@pytest.fixture
def lib(monkeypatch):
    recorder = Recorder()
    monkeypatch.setattr(mxg, "load", lambda: recorder)
    monkeypatch.setattr(mxg, "_here", lambda: -1)  # where tensors of the CPU are
    monkeypatch.setattr(mxg, "_stream_on", lambda stream, here: 7)
    return recorder


def zeros(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def test_descriptors_are_packed_as_c_lays_them_out():
    for kind in (mxg.Route, mxg.RouteGrad, mxg.ExpertRows, mxg.GatedAct):
        values = [i + 1 for i in range(len(kind._fields_))]
        packed = mxg._packer(kind)(*values).ljust(ctypes.sizeof(kind), b"\0")
        d = kind.from_buffer_copy(packed)
        assert [getattr(d, name) for name, _ in kind._fields_] == values


def test_route(lib):
    x = zeros(10, 12)[:, :8]
    e, w, c = zeros(10, 2, dtype=I32), zeros(10, 2), zeros(8, dtype=I32)
    loss, slope = zeros(1), zeros(8)
    row, groups, ws = zeros(10, 2, dtype=I32), zeros(17, dtype=I64), zeros(999, dtype=torch.uint8)
    mask = torch.ones(10, dtype=torch.bool)
    mxg.mxg_route(x, e, w, c, mask=mask, score=mxg.MXG_SCORE_SIGMOID, normalize=False, scale=2.0,
                  balance=0.5, loss=loss, slope=slope, row_of=row, group_ws=groups, align=128, last_dim=3,
                  workspace=ws)
    d, rest = lib.calls[0]
    assert (d.dtype, d.tokens, d.experts, d.k, d.ld) == (mxg.MXG_F32, 10, 8, 2, 12)
    assert (d.score, d.normalize, d.scale, d.balance) == (1, 0, 2.0, 0.5)
    assert (d.logits, d.mask, d.expert) == (x.data_ptr(), mask.data_ptr(), e.data_ptr())
    assert (d.weight, d.counts, d.loss) == (w.data_ptr(), c.data_ptr(), loss.data_ptr())
    assert (d.slope, d.row_of, d.group_ws) == (slope.data_ptr(), row.data_ptr(), groups.data_ptr())
    assert (d.align, d.rows_capacity, d.last_dim) == (128, 20 + 8 * 127, 3)
    assert rest == (ws.data_ptr(), 999, 0, 7)
    ok = dict(logits=x, expert=e, weight=w, counts=c, workspace=ws)
    for kw in (dict(logits=zeros(10, 8).double()), dict(logits=zeros(1, 8).expand(10, 8)),
               dict(logits=zeros(8, 10).t()), dict(logits=zeros(9, 8)), dict(logits=zeros(80)),
               dict(expert=e.long()), dict(expert=zeros(10, 4, dtype=I32)[:, :2]),
               dict(weight=w.to(BF)), dict(counts=c[:7]), dict(mask=zeros(10)), dict(mask=mask[:9]),
               dict(loss=zeros(2)), dict(slope=zeros(16)[::2]), dict(row_of=row), dict(group_ws=groups),
               dict(row_of=row, group_ws=groups[:16]), dict(row_of=e.long(), group_ws=groups)):
        with pytest.raises(ValueError):
            mxg.mxg_route(**dict(ok, **kw))
    assert len(lib.calls) == 1


def test_route_rows_and_backward(lib):
    e, c = zeros(10, 2, dtype=I32), zeros(8, dtype=I32)
    ws = zeros(99, dtype=torch.uint8)
    mxg.mxg_route_rows(e, c, workspace=ws)
    assert lib.calls[0][1] == (e.data_ptr(), 10, 8, 2, 1, 20, 1, c.data_ptr(), 0, 0, ws.data_ptr(), 99, 0, 7)
    x, d, dw, s, one = zeros(10, 8), zeros(10, 9)[:, :8], zeros(10, 2), zeros(8), zeros(1)
    mxg.mxg_route_backward(x, e, d, dweight=dw, slope=s, dloss=one)
    got = lib.calls[1][0]
    assert (got.ld, got.ldd, got.dlogits, got.dweight) == (0, 9, d.data_ptr(), dw.data_ptr())
    assert (got.slope, got.dloss, got.normalize) == (s.data_ptr(), one.data_ptr(), 1)
    for kw in (dict(dlogits=zeros(10, 7)), dict(dlogits=zeros(10, 8).to(BF)), dict(dweight=zeros(20, 2)),
               dict(dlogits=zeros(1, 8).expand(10, 8)), dict(slope=zeros(7)), dict(dloss=zeros(2))):
        with pytest.raises(ValueError):
            mxg.mxg_route_backward(**dict(dict(logits=x, expert=e, dlogits=d), **kw))


def test_rows(lib):
    x, rows, y = zeros(5, 16, dtype=BF), zeros(40, 24, dtype=BF)[:, :16], zeros(40, 16, dtype=BF)
    at, w = zeros(5, 3, dtype=I32), zeros(5, 3)
    c, groups = zeros(4, dtype=I32), zeros(9, dtype=I64)
    mxg.mxg_dispatch(x, at, rows, counts=c, group_ws=groups)
    mxg.mxg_combine(rows, at, x, weight=w)
    mxg.mxg_combine_backward(x, at, w, None, y_rows=y, dweight=w)
    a, b, g = (d for d, _ in lib.calls)
    for d in (a, b, g):
        assert (d.dtype, d.n, d.cols, d.k, d.rows_capacity) == (mxg.MXG_BF16, 5, 16, 3, 40)
        assert (d.tokens, d.row_of) == (x.data_ptr(), at.data_ptr())
    assert (a.rows, a.ldr, a.experts, a.counts, a.weight) == (rows.data_ptr(), 24, 4, c.data_ptr(), None)
    assert (b.rows, b.weight, b.experts, b.group_ws) == (rows.data_ptr(), w.data_ptr(), 0, None)
    assert (g.rows, g.y_rows, g.ldy, g.dweight) == (None, y.data_ptr(), 0, w.data_ptr())
    wide = zeros(1, 16, dtype=BF).expand(40, 16)
    for call in (lambda: mxg.mxg_dispatch(x, at, wide), lambda: mxg.mxg_dispatch(x[:4], at, rows),
                 lambda: mxg.mxg_dispatch(x, at, zeros(40, 16)), lambda: mxg.mxg_combine(wide, at, x),
                 lambda: mxg.mxg_combine(rows, at, x, weight=zeros(3, 5).t()),
                 lambda: mxg.mxg_dispatch(x, at, rows, counts=c), lambda: mxg.mxg_combine(rows, at.view(-1), x),
                 lambda: mxg.mxg_combine_backward(x, at, w, None), lambda: mxg.mxg_dispatch(x.int(), at, rows),
                 lambda: mxg.mxg_combine_backward(x, at, w, rows, y_rows=y[:39], dweight=w)):
        with pytest.raises(ValueError):
            call()
    assert len(lib.calls) == 3


def test_activation(lib):
    wide = zeros(6, 80, dtype=BF)
    gate, up, h = wide[:, :40], wide[:, 40:], zeros(6, 40, dtype=BF)
    q, sf = zeros(6, 80, dtype=torch.uint8), zeros(6, 4, dtype=torch.uint8)
    groups = zeros(7, dtype=I64)
    mxg.mxg_gated_act(gate, h, up=up, q=q, sf=sf, group_ws=groups, G=3)
    mxg.mxg_gated_act(gate, h)
    mxg.mxg_gated_act_backward(q.view(torch.float8_e4m3fn), sf, h, gate, dup=up, h=h)
    a, b, g = (d for d, _ in lib.calls)
    assert (a.rows, a.cols, a.gated, a.G, a.group_ws) == (6, 40, 1, 3, groups.data_ptr())
    assert (a.gate, a.ldg, a.up, a.ldu, a.ldq) == (gate.data_ptr(), 80, up.data_ptr(), 80, 0)
    assert (a.q, a.sf, a.dh) == (q.data_ptr(), sf.data_ptr(), None)
    assert (b.gated, b.up, b.q, b.sf, b.G) == (0, None, None, None, 0)
    assert (g.dgate, g.lddg, g.dup, g.h, g.gate) == (gate.data_ptr(), 80, up.data_ptr(), h.data_ptr(), None)
    for call in (lambda: mxg.mxg_gated_act(gate, h[:5]), lambda: mxg.mxg_gated_act(gate, h, q=q),
                 lambda: mxg.mxg_gated_act(gate, h, q=q, sf=sf), lambda: mxg.mxg_gated_act(gate, h.float()),
                 lambda: mxg.mxg_gated_act(gate, h, up=up, q=q, sf=sf[:, :3]),
                 lambda: mxg.mxg_gated_act(gate, h, up=up, q=q.float(), sf=sf),
                 lambda: mxg.mxg_gated_act(gate, h, group_ws=groups, G=2),
                 lambda: mxg.mxg_gated_act(zeros(1, 40, dtype=BF).expand(6, 40), h),
                 lambda: mxg.mxg_gated_act_backward(q, sf, h, gate),
                 lambda: mxg.mxg_gated_act_backward(None, None, h.view(-1), gate)):
        with pytest.raises(ValueError):
            call()


def test_tensors_elsewhere_are_refused(lib, monkeypatch):
    monkeypatch.setattr(mxg, "_here", lambda: 0)
    with pytest.raises(ValueError):
        mxg.mxg_gated_act(zeros(4, 8, dtype=BF), zeros(4, 8, dtype=BF))
