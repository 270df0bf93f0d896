"""Refusals of the 16-bit entry points, without a GPU: every call below fails
its checks before any device work."""
import ctypes

import pytest
import torch

from moe_grouped_block_gb300 import build as mxg_build
from moe_grouped_block_gb300 import mxg

FAKE = 1 << 20  # aligned and non-null; never dereferenced

no_device_only = pytest.mark.skipif(torch.cuda.is_available(),
                                    reason="fake-pointer validation tests run without a GPU")
OK_BUT_NO_DEVICE, INVALID, ALIGNMENT, TOO_SMALL = 3, 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    mxg_build.build()
    return mxg.load()


@no_device_only
def test_grouped_gemm_16bit(lib):
    base = dict(t=1, mode=0, A=FAKE, lda=0, B=FAKE, ldb=0, ws=FAKE, G=4, M=512, N=256, K=256, al=None,
                be=None, C=FAKE, ldc=0, out=0, st=None, s=None)

    def call(**kw):
        return lib.mxg_grouped_gemm_16bit(*dict(base, **kw).values())
    assert call() == OK_BUT_NO_DEVICE
    for kw in (dict(A=None), dict(B=None), dict(C=None), dict(ws=None), dict(G=0), dict(G=1025),
               dict(M=-1), dict(N=0), dict(K=0), dict(t=0), dict(t=3), dict(out=2), dict(mode=3),
               dict(out=5), dict(lda=128), dict(ldb=248), dict(ldc=255), dict(M=1 << 31),
               dict(lda=1 << 37), dict(ldb=1 << 36)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(A=FAKE + 2), dict(B=FAKE + 8), dict(C=FAKE + 2), dict(lda=260), dict(ldb=257),
               dict(K=100), dict(out=1, C=FAKE + 1)):
        assert call(**kw) == ALIGNMENT, kw
    # a ragged matrix without rows needs no memory; the others do
    assert call(M=0, A=None, C=None) == OK_BUT_NO_DEVICE
    assert call(M=0, mode=1, A=None, B=None) == OK_BUT_NO_DEVICE
    assert call(M=0, B=None) == call(M=0, mode=1, C=None) == call(M=0, mode=2, B=None) == INVALID
    # odd widths are fine where the strides are multiples of 8
    assert call(K=100, lda=104, ldb=104) == OK_BUT_NO_DEVICE
    assert call(N=7, out=1, C=FAKE + 2) == OK_BUT_NO_DEVICE
    assert call(mode=2, N=7, lda=8) == OK_BUT_NO_DEVICE


@no_device_only
def test_block_norm(lib):
    base = dict(dtype=1, res_dtype=1, rows=4, cols=64, x=FAKE, y=FAKE, gate_mode=0, res_scale=1.0,
                x_out=FAKE + 4096, n_out=FAKE + 8192, eps=1e-6)

    def call(**kw):
        return lib.mxg_block_norm(ctypes.byref(mxg.BlockNorm(**dict(base, **kw))), None)
    assert lib.mxg_block_norm(None, None) == INVALID
    assert call() == OK_BUT_NO_DEVICE
    assert call(y=None, x_out=None) == OK_BUT_NO_DEVICE
    assert call(rows=0, x=None, y=None, x_out=None, n_out=None) == OK_BUT_NO_DEVICE
    nan, inf = float("nan"), float("inf")
    for kw in (dict(x=None), dict(x_out=None), dict(y=None, n_out=None), dict(rows=-1), dict(cols=0),
               dict(cols=16385), dict(eps=0.0), dict(eps=nan), dict(eps=inf), dict(res_scale=nan),
               dict(dtype=3), dict(res_dtype=2), dict(dtype=0, res_dtype=1), dict(gate_mode=2),
               dict(gate_mode=4, gate=FAKE), dict(ldx=63), dict(ldy=1), dict(ldn=10), dict(ldxo=5),
               dict(y=None, gate=FAKE, gate_mode=1), dict(x_out=FAKE, ldx=64, ldxo=72)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(x=FAKE + 1), dict(y=FAKE + 1), dict(x_out=FAKE + 1), dict(n_out=FAKE + 1),
               dict(w_post=FAKE + 1), dict(w_pre=FAKE + 1), dict(gate=FAKE + 2, gate_mode=1)):
        assert call(**kw) == ALIGNMENT, kw


@no_device_only
def test_block_norm_backward(lib):
    base = dict(dtype=1, res_dtype=0, rows=4, cols=64, x=FAKE, y=FAKE, gate_mode=0, res_scale=1.0,
                eps=1e-6, dx_out=FAKE, dn=FAKE, dx=FAKE + 4096, dy=FAKE + 8192)
    need = mxg.mxg_block_norm_workspace_bytes(4, 64)
    assert need > 0 and mxg.mxg_block_norm_workspace_bytes(-1, 64) == 0

    def call(ws=FAKE, size=need, **kw):
        return lib.mxg_block_norm_backward(ctypes.byref(mxg.BlockNormGrad(**dict(base, **kw))), ws,
                                           size, None)
    assert call() == OK_BUT_NO_DEVICE
    for kw in (dict(dx=None), dict(dy=None), dict(dx_out=None, dn=None), dict(x=None), dict(ws=None),
               dict(lddx=8), dict(lddn=8), dict(lddy=8), dict(lddxo=8), dict(cols=20000),
               dict(dx=FAKE, lddx=72), dict(dy=FAKE, lddy=72), dict(gate_mode=3)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(ws=FAKE + 8), dict(dx=FAKE + 2), dict(dw_pre=FAKE + 2), dict(dy=FAKE + 1)):
        assert call(**kw) == ALIGNMENT, kw
    assert call(size=need - 1) == TOO_SMALL
    assert lib.mxg_block_norm_backward(None, FAKE, need, None) == INVALID


@no_device_only
def test_grad_clip(lib):
    need = mxg.mxg_grad_workspace_bytes()

    def call(n=1, norm=FAKE, ws=FAKE, size=need, limit=1.0, array=True, **kw):
        t = mxg.Grad(**dict(dict(src=FAKE, dst=FAKE, numel=8, src_type=1, dst_type=1), **kw))
        return lib.mxg_grad_clip(ctypes.addressof(t) if array else None, n, limit, norm, ws, size, None)
    assert call() == OK_BUT_NO_DEVICE
    assert call(numel=0, src=None, dst=None) == OK_BUT_NO_DEVICE
    assert call(n=0, array=False) == OK_BUT_NO_DEVICE
    for kw in (dict(n=-1), dict(array=False), dict(norm=None), dict(ws=None), dict(limit=-1.0),
               dict(limit=float("nan")), dict(src=None), dict(dst=None), dict(numel=-1),
               dict(numel=(1 << 40) + 1), dict(src_type=3), dict(dst_type=-1), dict(dst_type=2)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(src=FAKE + 1), dict(dst=FAKE + 1), dict(norm=FAKE + 2), dict(ws=FAKE + 4)):
        assert call(**kw) == ALIGNMENT, kw
    assert call(size=need - 1) == TOO_SMALL
    t = mxg.Grad(FAKE, None, 8, 0, 7)  # the norm alone needs no destination
    assert lib.mxg_grad_norm(ctypes.addressof(t), 1, FAKE, FAKE, need, None) == OK_BUT_NO_DEVICE
