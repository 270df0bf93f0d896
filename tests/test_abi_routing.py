"""Refusals of the routing, row and activation entry points, without a GPU: every call
below fails its checks before any device work."""
import ctypes

import pytest
import torch

from moe_grouped_block_gb300 import build as mxg_build
from moe_grouped_block_gb300 import mxg

FAKE = 1 << 20  # aligned and non-null; never dereferenced

no_device_only = pytest.mark.skipif(torch.cuda.is_available(),
                                    reason="fake-pointer validation tests run without a GPU")
OK_BUT_NO_DEVICE, INVALID, ALIGNMENT, TOO_SMALL = 3, 1, 2, 5
MOST = 0x7FFFFF80
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    mxg_build.build()
    return mxg.load()


def test_route_workspace():
    mxg_build.build()
    size = mxg.mxg_route_workspace_bytes
    assert 0 < size(1, 1, 1) <= 1024 and size(8, 8, 2) % 16 == 0
    for bad in ((-1, 8, 2), (8, 0, 1), (8, 1025, 2), (8, 8, 0), (8, 8, 9), (8, 64, 33), (MOST, 8, 2),
                (1 << 62, 8, 1), (8, -5, 1)):
        assert size(*bad) == 0, bad
    assert size(0, 8, 2) > 0
    # it stops growing with the tokens
    assert size(1 << 20, 64, 8) == size(1 << 24, 64, 8) > size(1 << 10, 64, 8)


@no_device_only
def test_route(lib):
    need = mxg.mxg_route_workspace_bytes(100, 64, 4)
    assert need > 0
    base = dict(dtype=0, tokens=100, experts=64, k=4, logits=FAKE, score=0, normalize=1, scale=1.0,
                balance=0.1, expert=FAKE, weight=FAKE, counts=FAKE, loss=FAKE, slope=FAKE, row_of=FAKE,
                group_ws=FAKE, align=1, rows_capacity=400, last_dim=64)

    def call(ws=FAKE, size=need, **kw):
        return lib.mxg_route(ctypes.byref(mxg.Route(**dict(base, **kw))), ws, size, None, None)
    assert lib.mxg_route(None, FAKE, need, None, None) == INVALID
    for kw in ({}, dict(mask=FAKE + 1), dict(loss=None, slope=None), dict(row_of=None, group_ws=None),
               dict(ld=64), dict(ld=65), dict(dtype=2, logits=FAKE + 2), dict(rows_capacity=0),
               dict(tokens=0, logits=None, expert=None, weight=None, row_of=None), dict(align=1024)):
        assert call(**kw) == OK_BUT_NO_DEVICE, kw
    for kw in (dict(dtype=3), dict(tokens=-1), dict(experts=0), dict(experts=1025), dict(k=0), dict(k=33),
               dict(experts=3), dict(tokens=MOST // 4 + 1), dict(logits=None), dict(expert=None),
               dict(weight=None), dict(counts=None), dict(score=2), dict(score=-1), dict(scale=NAN),
               dict(balance=INF), dict(ld=63), dict(ld=1 << 37), dict(ld=-64), dict(row_of=None),
               dict(group_ws=None), dict(align=0), dict(align=1025), dict(rows_capacity=-1),
               dict(rows_capacity=MOST + 1), dict(last_dim=0), dict(last_dim=1 << 60), dict(ws=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(logits=FAKE + 2), dict(dtype=1, logits=FAKE + 1), dict(expert=FAKE + 2),
               dict(weight=FAKE + 1), dict(counts=FAKE + 2), dict(loss=FAKE + 2), dict(slope=FAKE + 2),
               dict(row_of=FAKE + 2), dict(group_ws=FAKE + 4), dict(ws=FAKE + 8)):
        assert call(**kw) == ALIGNMENT, kw
    assert call(size=need - 1) == TOO_SMALL


@no_device_only
def test_route_rows(lib):
    need = mxg.mxg_route_workspace_bytes(100, 64, 4)
    base = dict(expert=FAKE, tokens=100, experts=64, k=4, align=128, cap=9000, last=1, counts=FAKE,
                row_of=FAKE, group_ws=FAKE, ws=FAKE, size=need, st=None, s=None)

    def call(**kw):
        return lib.mxg_route_rows(*dict(base, **kw).values())
    for kw in ({}, dict(row_of=None, group_ws=None), dict(tokens=0, expert=None)):
        assert call(**kw) == OK_BUT_NO_DEVICE, kw
    for kw in (dict(expert=None), dict(counts=None), dict(row_of=None), dict(group_ws=None),
               dict(tokens=-1), dict(k=65), dict(align=0), dict(cap=-1), dict(last=0), dict(ws=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(expert=FAKE + 2), dict(counts=FAKE + 1), dict(ws=FAKE + 4)):
        assert call(**kw) == ALIGNMENT, kw
    assert call(size=need - 1) == TOO_SMALL


@no_device_only
def test_route_backward(lib):
    base = dict(dtype=1, tokens=100, experts=64, k=4, logits=FAKE, expert=FAKE, score=1, normalize=0,
                scale=1.0, dweight=FAKE, slope=FAKE, dloss=FAKE, dlogits=FAKE + 4096)

    def call(**kw):
        return lib.mxg_route_backward(ctypes.byref(mxg.RouteGrad(**dict(base, **kw))), None)
    assert lib.mxg_route_backward(None, None) == INVALID
    for kw in ({}, dict(dweight=None), dict(slope=None, dloss=None), dict(dlogits=FAKE),
               dict(tokens=0, logits=None, expert=None, dlogits=None)):
        assert call(**kw) == OK_BUT_NO_DEVICE, kw
    for kw in (dict(slope=None), dict(dloss=None), dict(logits=None), dict(expert=None), dict(dlogits=None),
               dict(ld=63), dict(ldd=63), dict(dlogits=FAKE, ld=72), dict(scale=INF), dict(k=0),
               dict(dtype=-1), dict(score=5)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dlogits=FAKE + 1), dict(dweight=FAKE + 2), dict(dloss=FAKE + 2), dict(expert=FAKE + 1)):
        assert call(**kw) == ALIGNMENT, kw


@no_device_only
def test_expert_rows(lib):
    base = dict(dtype=1, n=10, cols=64, k=2, rows_capacity=20, tokens=FAKE, rows=FAKE + 8192, row_of=FAKE)

    def call(fn, **kw):
        return getattr(lib, fn)(ctypes.byref(mxg.ExpertRows(**dict(base, **kw))), None)
    pad = dict(experts=4, counts=FAKE, group_ws=FAKE)
    for fn in ("mxg_dispatch", "mxg_combine", "mxg_combine_backward"):
        assert getattr(lib, fn)(None, None) == INVALID
        assert call(fn) == OK_BUT_NO_DEVICE
        assert call(fn, rows_capacity=0, rows=None) == OK_BUT_NO_DEVICE
        assert call(fn, n=0, tokens=None, row_of=None) == OK_BUT_NO_DEVICE
        for kw in (dict(dtype=3), dict(n=-1), dict(cols=0), dict(cols=(1 << 20) + 1), dict(k=0), dict(k=33),
                   dict(n=MOST // 2 + 1), dict(rows_capacity=-1), dict(rows_capacity=MOST + 1),
                   dict(tokens=None), dict(rows=None), dict(row_of=None), dict(ldt=63), dict(ldr=63),
                   dict(ldt=-1), dict(counts=FAKE), dict(group_ws=FAKE), dict(experts=4),
                   dict(pad, counts=None), dict(pad, experts=1025), dict(pad, experts=-1)):
            assert call(fn, **kw) == INVALID, (fn, kw)
        for kw in (dict(tokens=FAKE + 1), dict(rows=FAKE + 1), dict(row_of=FAKE + 2)):
            assert call(fn, **kw) == ALIGNMENT, (fn, kw)
    assert call("mxg_dispatch", **pad) == call("mxg_combine_backward", **pad) == OK_BUT_NO_DEVICE
    assert call("mxg_combine", **pad) == INVALID
    assert call("mxg_dispatch", weight=FAKE) == INVALID
    assert call("mxg_combine", weight=FAKE) == OK_BUT_NO_DEVICE
    assert call("mxg_combine", weight=FAKE + 2) == ALIGNMENT
    for kw in (dict(dweight=FAKE), dict(y_rows=FAKE)):
        assert all(call(fn, **kw) == INVALID
                   for fn in ("mxg_dispatch", "mxg_combine", "mxg_combine_backward")), kw
    both = dict(dweight=FAKE, y_rows=FAKE)
    assert call("mxg_combine_backward", **both) == OK_BUT_NO_DEVICE
    assert call("mxg_combine_backward", rows=None, **both) == OK_BUT_NO_DEVICE
    assert call("mxg_combine_backward", dweight=FAKE, y_rows=FAKE + 8192) == OK_BUT_NO_DEVICE
    assert call("mxg_combine_backward", dweight=FAKE, y_rows=FAKE + 8192, ldr=72) == INVALID
    assert call("mxg_combine_backward", rows=None, **pad, **both) == INVALID
    assert call("mxg_combine_backward", dweight=FAKE + 2, y_rows=FAKE) == ALIGNMENT
    assert call("mxg_dispatch", **dict(pad, counts=FAKE + 2)) == ALIGNMENT
    assert call("mxg_dispatch", **dict(pad, group_ws=FAKE + 4)) == ALIGNMENT


@no_device_only
def test_gated_act(lib):
    fwd = dict(dtype=1, act=0, rows=4, cols=64, gated=1, gate=FAKE, up=FAKE, h=FAKE + 4096, q=FAKE, sf=FAKE)
    bwd = dict(dtype=2, act=1, rows=4, cols=64, gated=1, q=FAKE, sf=FAKE, dh=FAKE, dgate=FAKE + 4096,
               dup=FAKE + 8192)

    def call(back, **kw):
        fn = lib.mxg_gated_act_backward if back else lib.mxg_gated_act
        return fn(ctypes.byref(mxg.GatedAct(**dict(bwd if back else fwd, **kw))), None)
    assert lib.mxg_gated_act(None, None) == lib.mxg_gated_act_backward(None, None) == INVALID
    groups = dict(G=3, group_ws=FAKE)
    for back in (False, True):
        for kw in ({}, groups, dict(h=FAKE + 16384), dict(ldq=200), dict(cols=7)):
            assert call(back, **kw) == OK_BUT_NO_DEVICE, kw
        for kw in (dict(dtype=0), dict(dtype=3), dict(act=2), dict(act=-1), dict(rows=-1),
                   dict(rows=MOST + 1), dict(cols=0), dict(cols=(1 << 20) + 1), dict(gated=0), dict(gated=2),
                   dict(G=3), dict(group_ws=FAKE), dict(groups, G=1025), dict(groups, G=-1), dict(ldq=127),
                   dict(ldh=63), dict(q=None), dict(sf=None)):
            assert call(back, **kw) == INVALID, (back, kw)
        assert call(back, **dict(groups, group_ws=FAKE + 4)) == ALIGNMENT
        assert call(back, h=FAKE + 1) == ALIGNMENT
    for kw in (dict(q=None, sf=None), dict(gated=0, up=None), dict(h=FAKE), dict(h=FAKE, ldh=64),
               dict(rows=0, gate=None, up=None, h=None, q=None, sf=None)):
        assert call(False, **kw) == OK_BUT_NO_DEVICE, kw
    for kw in (dict(gate=None), dict(h=None), dict(up=None), dict(dh=FAKE), dict(dgate=FAKE), dict(dup=FAKE),
               dict(ldg=63), dict(ldu=63), dict(h=FAKE, ldh=72)):
        assert call(False, **kw) == INVALID, kw
    for kw in (dict(gate=FAKE + 1), dict(up=FAKE + 1)):
        assert call(False, **kw) == ALIGNMENT, kw
    for kw in (dict(gated=0, dup=None), dict(dh=FAKE + 4096), dict(dh=FAKE + 8192),
               dict(rows=0, q=None, sf=None, dh=None, dgate=None, dup=None)):
        assert call(True, **kw) == OK_BUT_NO_DEVICE, kw
    for kw in (dict(dh=None), dict(dgate=None), dict(dup=None), dict(gate=FAKE), dict(up=FAKE), dict(lddh=63),
               dict(lddg=63), dict(lddu=63), dict(dh=FAKE + 4096, lddh=72), dict(dh=FAKE + 8192, lddu=72)):
        assert call(True, **kw) == INVALID, kw
    for kw in (dict(dh=FAKE + 1), dict(dgate=FAKE + 1), dict(dup=FAKE + 1)):
        assert call(True, **kw) == ALIGNMENT, kw
