"""What the binding of the 16-bit operators passes on and what it refuses, without a
GPU: the library is replaced by a recorder of the arguments that it is given."""
import pytest
import torch

from moe_grouped_block_gb300 import mxg

BF, F32 = torch.bfloat16, torch.float32


class Recorder:
    """Stands in for the loaded library: keeps each call's arguments, returns MXG_OK."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            # the structures are read here: their memory is the caller's
            self.calls.append((name, [getattr(a, "_obj", a) for a in args]))
            return 0
        return entry


@pytest.fixture
def lib(monkeypatch):
    recorder = Recorder()
    monkeypatch.setattr(mxg, "load", lambda: recorder)
    monkeypatch.setattr(mxg, "_p", lambda t: t if t is None or isinstance(t, int) else t.data_ptr())
    monkeypatch.setattr(mxg, "_s", lambda stream: None)
    return recorder


def broadcast(rows, cols, dtype=BF):
    """One row seen `rows` times: a stride of 0 between the rows."""
    return torch.zeros(1, cols, dtype=dtype).expand(rows, cols)


def test_broadcast_rows_are_refused_by_the_norms(lib):
    """Read as dense they would be read past their end."""
    x, w = torch.zeros(5, 64, dtype=BF), torch.zeros(64, dtype=BF)
    wide, ws = broadcast(5, 64), torch.empty(1 << 16, dtype=torch.uint8)
    new = lambda: torch.zeros_like(x)  # noqa: E731
    for kw in (dict(x=wide), dict(y=wide), dict(gate=wide), dict(x_out=wide), dict(n_out=wide)):
        arg = dict(dict(x=x, y=new(), w_post=w, gate=new(), gate_mode=mxg.MXG_GATE_FULL, x_out=new(),
                        w_pre=w, n_out=new()), **kw)
        with pytest.raises(ValueError):
            mxg.mxg_block_norm(**arg)
    for kw in (dict(x=wide), dict(y=wide), dict(gate=wide), dict(dx_out=wide), dict(dn=wide),
               dict(dx=wide), dict(dy=wide), dict(dgate=wide)):
        arg = dict(dict(x=x, y=new(), w_post=w, gate=new(), gate_mode=mxg.MXG_GATE_FULL, w_pre=w,
                        dx_out=new(), dn=new(), dx=new(), dy=new(), dgate=new(), workspace=ws), **kw)
        with pytest.raises(ValueError):
            mxg.mxg_block_norm_backward(**arg)
    assert lib.calls == []
    # a single row may be the view that it is, and rows that only lie apart are passed on
    mxg.mxg_block_norm(broadcast(1, 64), n_out=torch.zeros(1, 64, dtype=BF), w_pre=w)
    mxg.mxg_block_norm(torch.zeros(5, 80, dtype=BF)[:, :64], n_out=x, w_pre=w)
    assert lib.calls[1][1][0].ldx == 80


def test_broadcast_operands_are_refused_by_the_products(lib):
    x, w, c = torch.zeros(16, 64, dtype=BF), torch.zeros(2, 32, 64, dtype=BF), torch.zeros(16, 32)
    ws = torch.zeros(5, dtype=torch.int64)
    call = lambda a=x, b=w, o=c: mxg.mxg_grouped_gemm_16bit(  # noqa: E731
        mxg.MXG_FPROP_TN, a, b, ws, 2, 16, 32, 64, C=o)
    for kw in (dict(a=broadcast(16, 64)), dict(b=w[:1].expand(2, 32, 64)), dict(b=broadcast(64, 64)),
               dict(b=w[:, :1].expand(2, 32, 64)), dict(o=broadcast(16, 32, F32))):
        with pytest.raises(ValueError):
            call(**kw)
    assert lib.calls == []
    call()
    assert len(lib.calls) == 1
