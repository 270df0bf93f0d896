"""The norms around a block, forward and backward, against 64 bits.

Bounds.  A row's sums run over D elements, so what is made of them carries a
relative error of at most (D + 16) 2^-24 (one rounding an addition, and the
square root, the reciprocal, the products); each result is a short sum of
products of such factors and its error is at most c (D + 16) 2^-24 of the sum of
the magnitudes of its terms -- c = 2 forward, 8 backward (dy is made of dx) --
plus one rounding u |ref| to its type (u = 2^-24, 2^-8, 2^-11).  A column's sum
over R rows adds R 2^-24 of the sum of magnitudes.
"""
import pytest
import torch

from gpu_util import DEV, require_gpu
from moe_grouped_block_gb300 import mxg

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
GATES = {"none": 0, "row": 1, "col": 2, "full": 3}
EPS = 1e-5


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def strided(t, pad):
    if pad == 0:
        return t
    buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def make(rows, cols, dtype, res, gate, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = {"x": (2 * r(rows, cols) * scale).to(res), "y": (r(rows, cols) * scale).to(dtype),
         "w_post": (1 + 0.2 * r(cols)).to(dtype), "w_pre": (1 + 0.2 * r(cols)).to(dtype),
         "dx_out": r(rows, cols).to(res), "dn": r(rows, cols).to(dtype)}
    t["gate"] = {"none": None, "row": r(rows), "col": r(cols).to(dtype),
                 "full": r(rows, cols).to(dtype)}[gate]
    return t


def spread_gate(t, gate):
    if gate == "none":
        return torch.ones(1, 1, dtype=torch.float64)
    v = t["gate"].double()
    return v.unsqueeze(1) if gate == "row" else v


def forward_ref(t, gate, s, after=True, before=True):
    x, y = t["x"].double(), t["y"].double()
    mag = x.abs()
    if after:
        ry = (y.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
        add = s * spread_gate(t, gate) * y * ry * t["w_post"].double()
        x, mag = x + add, mag + add.abs()
    rx = (x.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
    w = t["w_pre"].double()
    return x, mag, x * rx * w, mag * rx * w.abs()


def close(got, ref, mag, out, c, n):
    tol = c * (n + 16) * 2.0 ** -24 * mag + U[out] * ref.abs() + (2.0 ** -25 if out == HF else 0)
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(got).all() and not (err > tol).any(), \
        "worst excess %g" % float((err - tol).max())


KINDS = [(BF, BF), (BF, F32), (HF, HF), (HF, F32), (F32, F32)]
SIZES = [(1, 1), (1, 4096), (3, 7), (5, 64), (2, 256), (7, 1000), (4, 2056), (3, 8200), (2, 16384),
         (2, 16383), (700, 40)]


@pytest.mark.parametrize("gate", list(GATES))
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "%s_%s" % (str(k[0])[6:], str(k[1])[6:]))
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(rows, cols, kind, gate):
    dtype, res = kind
    t = make(rows, cols, dtype, res, gate, 1)
    d = {k: None if v is None else v.to(DEV) for k, v in t.items()}
    x_out, n = torch.empty_like(d["x"]), torch.empty_like(d["y"])
    mxg.mxg_block_norm(d["x"], d["y"], d["w_post"], d["gate"], GATES[gate], 0.75, x_out, d["w_pre"],
                       n, EPS)
    x, mx, nn, mn = forward_ref(t, gate, 0.75)
    close(x_out, x, mx, res, 2, cols)
    close(n, nn, mn, dtype, 4, cols)


def backward_ref(t, gate, s, after=True, dxo=True, dn=True):
    z = lambda k: t[k].double()  # noqa: E731
    x, D = z("x"), t["x"].shape[1]
    g = {"dw_pre": None}
    tt = z("dx_out") if dxo else torch.zeros_like(x)
    mag = tt.abs()
    if dn:
        rx = (x.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
        xh, a = x * rx, z("dn") * z("w_pre")
        tt = tt + rx * (a - xh * (a * xh).mean(1, keepdim=True))
        mag = mag + rx * (a.abs() + xh.abs() * (a * xh).abs().mean(1, keepdim=True))
        g["dw_pre"] = ((z("dn") * xh).sum(0), (z("dn") * xh).abs().sum(0))
    g["dx"] = (tt, mag)
    if after:
        y, w, v = z("y"), z("w_post"), s * spread_gate(t, gate)
        ry = (y.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
        yh = y * ry
        b, mb = tt * v * w, mag * (v * w).abs()
        g["dy"] = (ry * (b - yh * (b * yh).mean(1, keepdim=True)),
                   ry * (mb + yh.abs() * (mb * yh.abs()).mean(1, keepdim=True)))
        g["dw_post"] = ((tt * v * yh).sum(0), (mag * (v * yh).abs()).sum(0))
        dg, mg = s * tt * yh * w, abs(s) * mag * (yh * w).abs()
        over = {"row": 1, "col": 0}.get(gate)
        if gate != "none":
            g["dgate"] = (dg, mg) if over is None else (dg.sum(over), mg.sum(over))
    return g


def run_backward(d, gate, s, rows, cols, dtype, res, **without):
    out = {"dx": torch.empty(rows, cols, dtype=res, device=DEV),
           "dy": torch.empty(rows, cols, dtype=dtype, device=DEV),
           "dw_post": torch.empty(cols, device=DEV), "dw_pre": torch.empty(cols, device=DEV),
           "dgate": {"none": None, "row": torch.empty(rows, device=DEV),
                     "col": torch.empty(cols, device=DEV),
                     "full": torch.empty(rows, cols, dtype=dtype, device=DEV)}[gate]}
    arg = dict(x=d["x"], y=d["y"], w_post=d["w_post"], gate=d["gate"], gate_mode=GATES[gate],
               res_scale=s, w_pre=d["w_pre"], eps=EPS, dx_out=d["dx_out"], dn=d["dn"],
               workspace=mxg.alloc_block_norm_workspace(rows, cols), **out)
    arg.update(without)
    arg["workspace"].fill_(255)  # NaN: nothing of it may be read before it is written
    mxg.mxg_block_norm_backward(**arg)
    torch.cuda.synchronize()
    return out


def check_backward(out, ref, dtype, res, gate, rows, cols):
    close(out["dx"], *ref["dx"], res, 8, cols)
    if ref["dw_pre"] is not None:
        close(out["dw_pre"], *ref["dw_pre"], F32, 8, cols + rows)
    if "dy" in ref:
        close(out["dy"], *ref["dy"], dtype, 8, cols)
        close(out["dw_post"], *ref["dw_post"], F32, 8, cols + rows)
        if gate != "none":
            close(out["dgate"], *ref["dgate"], dtype if gate == "full" else F32, 8, cols + rows)


@pytest.mark.parametrize("gate", list(GATES))
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "%s_%s" % (str(k[0])[6:], str(k[1])[6:]))
@pytest.mark.parametrize("rows,cols", SIZES)
def test_backward(rows, cols, kind, gate):
    dtype, res = kind
    t = make(rows, cols, dtype, res, gate, 2)
    d = {k: None if v is None else v.to(DEV) for k, v in t.items()}
    out = run_backward(d, gate, 0.75, rows, cols, dtype, res)
    check_backward(out, backward_ref(t, gate, 0.75), dtype, res, gate, rows, cols)


@pytest.mark.parametrize("pad", [0, 3, 8])
def test_parts_alone_and_strides(pad):
    """Each part without the other, weights of ones, rows of any stride."""
    rows, cols = 9, 264
    t = make(rows, cols, BF, BF, "none", 3)
    ones = dict(t, w_post=torch.ones(cols), w_pre=torch.ones(cols))
    d = {k: strided(v.to(DEV), pad) if v is not None and v.dim() == 2 else v for k, v in t.items()}
    new = lambda: strided(torch.zeros(rows, cols, dtype=BF, device=DEV), pad)  # noqa: E731
    n = new()
    mxg.mxg_block_norm(d["x"], n_out=n, eps=EPS)
    _, _, ref, mag = forward_ref(ones, "none", 1.0, after=False)
    close(n, ref, mag, BF, 4, cols)
    xo = new()
    mxg.mxg_block_norm(d["x"], d["y"], x_out=xo, res_scale=-0.5, eps=EPS)
    ref, mag, _, _ = forward_ref(ones, "none", -0.5)
    close(xo, ref, mag, BF, 2, cols)
    for kw in (dict(y=None, dx_out=None), dict(y=None), dict(dn=None, x=d["x"]), dict(dx_out=None)):
        got = {"dx": new(), "dy": new()}
        arg = dict(x=d["x"], y=d["y"], w_post=None, res_scale=0.5, w_pre=None, eps=EPS,
                   dx_out=d["dx_out"], dn=d["dn"], dx=got["dx"], dy=got["dy"],
                   workspace=mxg.alloc_block_norm_workspace(rows, cols))
        arg.update(kw)
        mxg.mxg_block_norm_backward(**arg)
        ref = backward_ref(ones, "none", 0.5, after=arg["y"] is not None,
                           dxo=arg["dx_out"] is not None, dn=arg["dn"] is not None)
        close(got["dx"], *ref["dx"], BF, 8, cols)
        if arg["y"] is not None:
            close(got["dy"], *ref["dy"], BF, 8, cols)


def test_in_place():
    rows, cols = 33, 512
    t = make(rows, cols, BF, BF, "col", 4)
    d = {k: v.to(DEV) for k, v in t.items()}
    n = torch.empty_like(d["y"])
    mxg.mxg_block_norm(d["x"], d["y"], d["w_post"], d["gate"], 2, 0.5, d["x"], d["w_pre"], n, EPS)
    x, mx, nn, mn = forward_ref(t, "col", 0.5)
    close(d["x"], x, mx, BF, 2, cols)
    close(n, nn, mn, BF, 4, cols)
    d = {k: v.to(DEV) for k, v in t.items()}
    run_backward(d, "col", 0.5, rows, cols, BF, BF, dx=d["dx_out"], dy=d["dn"])
    ref = backward_ref(t, "col", 0.5)
    close(d["dx_out"], *ref["dx"], BF, 8, cols)
    close(d["dn"], *ref["dy"], BF, 8, cols)


def test_rows_of_zeros_and_tiny_rows():
    """A row of zeros: its norm is 1 / sqrt(eps), its outputs 0."""
    rows, cols = 4, 128
    t = make(rows, cols, F32, F32, "none", 5)
    t["x"][1] = 0
    t["y"][1] = 0
    t["x"][2] *= 1e-12
    t["y"][2] *= 1e-12
    d = {k: None if v is None else v.to(DEV) for k, v in t.items()}
    xo, n = torch.empty_like(d["x"]), torch.empty_like(d["y"])
    mxg.mxg_block_norm(d["x"], d["y"], d["w_post"], None, 0, 1.0, xo, d["w_pre"], n, EPS)
    x, mx, nn, mn = forward_ref(t, "none", 1.0)
    close(xo, x, mx, F32, 2, cols)
    close(n, nn, mn, F32, 4, cols)
    assert (xo[1] == 0).all() and (n[1] == 0).all()
    out = run_backward(d, "none", 1.0, rows, cols, F32, F32)
    check_backward(out, backward_ref(t, "none", 1.0), F32, F32, "none", rows, cols)


def test_nan_stays_in_its_row():
    rows, cols = 20, 264
    t = make(rows, cols, BF, F32, "row", 6)
    d = {k: v.to(DEV) for k, v in t.items()}
    d["y"][7, 3] = float("nan")
    d["x"][9, 1] = float("inf")
    xo, n = torch.empty_like(d["x"]), torch.empty_like(d["y"])
    mxg.mxg_block_norm(d["x"], d["y"], d["w_post"], d["gate"], 1, 1.0, xo, d["w_pre"], n, EPS)
    keep = [i for i in range(rows) if i not in (7, 9)]
    x, mx, nn, mn = forward_ref(t, "row", 1.0)
    close(xo[keep], x[keep], mx[keep], F32, 2, cols)
    close(n[keep], nn[keep], mn[keep], BF, 4, cols)
    assert torch.isnan(xo[7]).all() and torch.isnan(n[7]).all() and torch.isnan(n[9, 1])
    out = run_backward(d, "row", 1.0, rows, cols, BF, F32)
    ref = backward_ref(t, "row", 1.0)
    for k in ("dx", "dy", "dgate"):
        close(out[k][keep], ref[k][0][keep], ref[k][1][keep], BF if k == "dy" else F32, 8, cols)


def test_no_rows():
    cols = 72
    z = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device=DEV)  # noqa: E731
    mxg.mxg_block_norm(z(0, cols), n_out=z(0, cols))
    w = torch.ones(cols, dtype=BF, device=DEV)
    dw_post, dw_pre, dg = (torch.full((cols,), 7.0, device=DEV) for _ in range(3))
    mxg.mxg_block_norm_backward(z(0, cols), z(0, cols), w, w, 2, 1.0, w, EPS, None, z(0, cols),
                                z(0, cols), z(0, cols), dw_post, dw_pre, dg,
                                mxg.alloc_block_norm_workspace(0, cols))
    for v in (dw_post, dw_pre, dg):
        assert (v == 0).all()


@pytest.mark.parametrize("gate", list(GATES))
def test_gradients_are_differences(gate):
    """Central differences of the fp32 forward pass along random directions.
    With a step of h = 2^-6 the truncation error is h^2 / 6 times a third
    derivative of order one per unit of direction, 4e-5, and the fp32 roundings
    of the outputs add 2^-24 / h = 4e-6 of the outputs' share: 2e-3 of
    |gradient| |direction| + |outputs' weights| covers both."""
    rows, cols, h = 3, 40, 2.0 ** -6
    t = make(rows, cols, F32, F32, gate, 7)
    d = {k: None if v is None else v.to(DEV) for k, v in t.items()}

    def value(p):
        xo, n = torch.empty_like(p["x"]), torch.empty_like(p["y"])
        mxg.mxg_block_norm(p["x"], p["y"], p["w_post"], p["gate"], GATES[gate], 0.75, xo, p["w_pre"],
                           n, EPS)
        return float((xo.double() * d["dx_out"].double()).sum() + (n.double() * d["dn"].double()).sum())
    xo, n = torch.empty_like(d["x"]), torch.empty_like(d["y"])
    mxg.mxg_block_norm(d["x"], d["y"], d["w_post"], d["gate"], GATES[gate], 0.75, xo, d["w_pre"], n, EPS)
    out = run_backward(dict(d, x=xo), gate, 0.75, rows, cols, F32, F32)
    grads = {"x": out["dx"], "y": out["dy"], "w_post": out["dw_post"], "w_pre": out["dw_pre"],
             "gate": out["dgate"]}
    g = torch.Generator().manual_seed(8)
    for k, grad in grads.items():
        if grad is None:
            continue
        u = torch.randn(d[k].shape, generator=g).to(DEV)
        diff = (value(dict(d, **{k: d[k] + h * u})) - value(dict(d, **{k: d[k] - h * u}))) / (2 * h)
        want = float((grad.double() * u.double()).sum())
        room = 2e-3 * float(grad.norm() * u.norm() + d["dx_out"].norm() + d["dn"].norm())
        assert abs(diff - want) <= room, (k, diff, want, room)


def test_long_offsets():
    """Rows whose element offsets pass 32 bits (a wide stride)."""
    rows, cols, ld = 3, 64, 1 << 30
    buf = torch.empty((rows - 1) * ld + cols, dtype=BF, device=DEV)
    x = buf.as_strided((rows, cols), (ld, 1))
    t = make(rows, cols, BF, BF, "none", 9)
    x.copy_(t["x"].to(DEV))
    n = torch.empty(rows, cols, dtype=BF, device=DEV)
    mxg.mxg_block_norm(x, w_pre=t["w_pre"].to(DEV), n_out=n, eps=EPS)
    _, _, ref, mag = forward_ref(t, "none", 1.0, after=False)
    close(n, ref, mag, BF, 4, cols)


def test_stream_graph_and_same_bits():
    rows, cols = 700, 520
    t = make(rows, cols, BF, BF, "col", 10)
    d = {k: v.to(DEV) for k, v in t.items()}
    want = run_backward(d, "col", 0.5, rows, cols, BF, BF)
    again = run_backward(d, "col", 0.5, rows, cols, BF, BF)
    for k in want:
        assert torch.equal(want[k], again[k])
    n, n2 = torch.empty_like(d["y"]), torch.empty_like(d["y"])
    mxg.mxg_block_norm(d["x"], w_pre=d["w_pre"], n_out=n, eps=EPS)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mxg.mxg_block_norm(d["x"], w_pre=d["w_pre"], n_out=n2, eps=EPS)
    s.synchronize()
    assert torch.equal(n, n2)
    graph = torch.cuda.CUDAGraph()
    n2.zero_()
    with torch.cuda.graph(graph):
        mxg.mxg_block_norm(d["x"], w_pre=d["w_pre"], n_out=n2, eps=EPS)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(n, n2)


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=BF, device=DEV)
    w = torch.zeros(64, dtype=BF, device=DEV)
    ok = torch.zeros_like(x)
    with pytest.raises(ValueError):  # types
        mxg.mxg_block_norm(x, n_out=ok.half(), w_pre=w)
    with pytest.raises(ValueError):  # shapes
        mxg.mxg_block_norm(x, n_out=ok[:3], w_pre=w)
    with pytest.raises(ValueError):  # weights
        mxg.mxg_block_norm(x, n_out=ok, w_pre=w[:63])
    with pytest.raises(ValueError):  # the gate's size
        mxg.mxg_block_norm(x, ok, x_out=ok, gate=w, gate_mode=mxg.MXG_GATE_FULL)
    with pytest.raises(ValueError):  # a ROW gate is fp32
        mxg.mxg_block_norm(x, ok, x_out=ok, gate=w[:4], gate_mode=mxg.MXG_GATE_ROW)
    with pytest.raises(ValueError):  # columns must be contiguous
        mxg.mxg_block_norm(x.t().contiguous().t(), n_out=ok)
    with pytest.raises(mxg.MxgError):  # y without x_out
        mxg.mxg_block_norm(x, ok, n_out=ok)
    with pytest.raises(mxg.MxgError) as e:
        mxg.mxg_block_norm_backward(x, dn=ok, dx=ok, workspace=torch.empty(16, device=DEV))
    assert e.value.code == 5
