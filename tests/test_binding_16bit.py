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


FPROP, WGRAD, DGRAD = mxg.MXG_FPROP_TN, mxg.MXG_WGRAD_NT, mxg.MXG_DGRAD_NN
M, N, K, G = 24, 32, 64, 3


def operands(mode):
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt)  # noqa: E731
    return {"A": z(M, K if mode == FPROP else N), "B": z(M, K) if mode == WGRAD else z(G, N, K),
            "C": z(*{FPROP: (M, N), DGRAD: (M, K), WGRAD: (G, N, K)}[mode], dt=F32)}


def product(lib, mode, m=M, n=N, k=K, g=G, alpha=None, beta=None, ws=None, **kw):
    """The leading dimensions of A, B and C that the library is given."""
    t = dict(operands(mode), **kw)
    ws = torch.zeros(2 * g + 1, dtype=torch.int64) if ws is None else ws
    mxg.mxg_grouped_gemm_16bit(mode, t["A"], t["B"], ws, g, m, n, k, alpha, beta, t["C"])
    args = lib.calls[-1][1]
    return args[3], args[5], args[14]


@pytest.mark.parametrize("mode", [FPROP, WGRAD, DGRAD])
def test_products_dense_and_larger(lib, mode):
    assert product(lib, mode) == (0, 0, 0)
    t = operands(mode)
    more = {k: torch.zeros(v.shape[0] + 5, *v.shape[1:], dtype=v.dtype) for k, v in t.items()}
    assert product(lib, mode, **more) == (0, 0, 0)  # more rows, or experts
    # a wider matrix gives its first columns: its row stride counts, contiguous or not
    wide = {k: torch.zeros(*v.shape[:-1], 2 * v.shape[-1], dtype=v.dtype) for k, v in t.items()}
    want = tuple(2 * v.shape[-1] for v in t.values())
    assert product(lib, mode, **wide) == want
    assert product(lib, mode, **{k: v[..., :v.shape[-1] // 2] for k, v in wide.items()}) == want


def test_products_reshapes(lib):
    """Contiguous tensors of other shapes that hold the same matrix."""
    w, x = torch.zeros(G * N, K, dtype=BF), torch.zeros(M, 4, K // 4, dtype=BF)
    assert product(lib, FPROP, A=x, B=w, C=torch.zeros(M * N)) == (0, 0, 0)
    assert product(lib, FPROP, A=x.reshape(-1), B=w.reshape(G, N * K)) == (0, 0, 0)
    wide = torch.zeros(G * N, 2 * K, dtype=BF)[:, :K]
    assert product(lib, DGRAD, B=wide) == (0, 2 * K, 0)
    assert product(lib, DGRAD, B=wide.unflatten(0, (G, N))) == (0, 2 * K, 0)


def test_products_single_rows(lib):
    """One row: its stride, of whatever size, does not matter."""
    for buf in (torch.zeros(1, 100, dtype=BF), torch.zeros(4, 104, dtype=BF)[:1, :100],
                torch.zeros(100, dtype=BF), torch.zeros(100, 3, dtype=BF).t()[:1, :100].contiguous()):
        lda, _, ldc = product(lib, FPROP, m=1, k=100, A=buf,
                              B=torch.zeros(G, N, 104, dtype=BF)[..., :100], C=torch.zeros(1, N))
        assert lda >= 100 and lda % 8 == 0 and ldc >= N
    one = torch.zeros(1, 1, 100, dtype=BF)
    assert product(lib, FPROP, n=1, k=100, g=1, A=torch.zeros(M, 104, dtype=BF), B=one,
                   C=torch.zeros(M, 1))[:2] == (104, 104)
    # one row an expert: the stride is that of the experts
    assert product(lib, FPROP, n=1, B=torch.zeros(G, 2, K, dtype=BF)[:, :1], C=torch.zeros(M, 1))[1] == 2 * K


@pytest.mark.parametrize("mode", [FPROP, WGRAD, DGRAD])
def test_products_refuse_other_shapes(lib, mode):
    """Too few rows, columns or experts: the library would read, or write, past the end."""
    for name, t in operands(mode).items():
        bad = [t[:-1], t[..., :-1], t[..., :-1].contiguous(), t.reshape(-1)[:-1], t[..., 0]]
        if t.dim() == 3:
            bad += [t[:, :-1], t[:, :-1].contiguous(), t.reshape(G * N, K)[:-1],
                    torch.zeros(G, 2 * N, K, dtype=t.dtype), torch.zeros(G, 2 * N, K, dtype=t.dtype)[:, ::2][:, :-1]]
        else:
            bad.append(t.t())
            bad.append(torch.zeros(*reversed(t.shape), dtype=t.dtype))
        for b in bad:
            with pytest.raises(ValueError):
                product(lib, mode, **{name: b})
    f = lambda n, dt=F32: torch.zeros(n, dtype=dt)  # noqa: E731
    for kw in (dict(alpha=f(G - 1)), dict(beta=f(G - 1)), dict(alpha=f(G, torch.float64)),
               dict(beta=f(G, BF)), dict(alpha=f(2 * G)[::2]), dict(ws=f(G - 1, torch.int64))):
        with pytest.raises(ValueError):
            product(lib, mode, **kw)
    assert lib.calls == []
    product(lib, mode, alpha=f(G), beta=f(G + 1))


def test_products_without_rows(lib):
    e = lambda *s, dt=BF: torch.empty(*s, dtype=dt)  # noqa: E731
    for cap in (0, 8):
        product(lib, FPROP, m=cap, A=e(cap, K), C=e(8, N, dt=F32))
        product(lib, WGRAD, m=cap, A=e(cap, N), B=e(8, K))
    for kw in (dict(m=-1), dict(n=0), dict(k=0)):  # the library's to refuse
        product(lib, FPROP, **kw)
