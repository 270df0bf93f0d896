"""The norms around a block where a team of threads walks many rows, against 64 bits.

Shapes have more rows than a GPU's teams take at once, several times over and with
a remainder, so that rings of inputs go round, reductions are taken a row ahead,
buffers alternate and a CTA's column sums run over several rows.

Bounds: those of test_gpu_k_block_norm.py.  A row's sums carry (D + 16) 2^-24
relative; results c times that of the sum of their terms' magnitudes (c = 2 for x',
4 for n, 8 backward) and one rounding to their type; sums over R rows R 2^-24 more.
"""
import pytest
import torch

from gpu_util import DEV, require_gpu
from moe_grouped_block_gb300 import mxg
from test_gpu_k_block_norm import (BF, EPS, F32, GATES, HF, KINDS, U, backward_ref, forward_ref,
                                   make, run_backward, strided)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def close(got, ref, mag, out, c, n):
    """The same bound as test_gpu_k_block_norm.close, on the GPU."""
    tol = c * (n + 16) * 2.0 ** -24 * mag + U[out] * ref.abs() + (2.0 ** -25 if out == HF else 0)
    excess = (got.double() - ref).abs() - tol
    assert torch.isfinite(got).all() and float(excess.max()) <= 0, "worst excess %g" % float(excess.max())


def on_gpu(rows, cols, dtype, res, gate, seed):
    return {k: None if v is None else v.to(DEV)
            for k, v in make(rows, cols, dtype, res, gate, seed).items()}


def gpu_ref(fn, d, gate, *args, **kw):
    if gate == "none":
        d = dict(d, gate=torch.ones(1, 1, device=DEV))
        gate = "full"  # a gate of ones
    return fn(d, gate, *args, **kw)


def forward(d, gate, s):
    x_out, n = torch.empty_like(d["x"]), torch.empty_like(d["y"])
    mxg.mxg_block_norm(d["x"], d["y"], d["w_post"], d["gate"], GATES[gate], s, x_out, d["w_pre"], n,
                       EPS)
    return x_out, n


def check_forward(got, ref, dtype, res, cols, keep=slice(None)):
    x, mx, n, mn = ref
    close(got[0][keep], x[keep], mx[keep], res, 2, cols)
    close(got[1][keep], n[keep], mn[keep], dtype, 4, cols)


def check_backward(out, ref, dtype, res, gate, rows, cols):
    close(out["dx"], *ref["dx"], res, 8, cols)
    close(out["dy"], *ref["dy"], dtype, 8, cols)
    close(out["dw_pre"], *ref["dw_pre"], F32, 8, cols + rows)
    close(out["dw_post"], *ref["dw_post"], F32, 8, cols + rows)
    if gate != "none":
        close(out["dgate"], *ref["dgate"], dtype if gate == "full" else F32, 8, cols + rows)


# several teams a CTA; 8 and 16 columns a thread; two or three rows a team; rows shared
# by two CTAs; widths and strides that take single elements
SHAPES = [(100003, 40), (40001, 200), (2777, 4096), (303, 4096), (401, 4096), (1531, 7168),
          (700, 8200), (700, 16384), (613, 8201), (2003, 4099), (5003, 1001)]


@pytest.mark.parametrize("gate", list(GATES))
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "%s_%s" % (str(k[0])[6:], str(k[1])[6:]))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_both_ways(rows, cols, kind, gate):
    dtype, res = kind
    d = on_gpu(rows, cols, dtype, res, gate, 31)
    check_forward(forward(d, gate, 0.75), gpu_ref(forward_ref, d, gate, 0.75), dtype, res, cols)
    out = run_backward(d, gate, 0.75, rows, cols, dtype, res)
    ref = gpu_ref(backward_ref, d, gate, 0.75)
    check_backward(out, ref, dtype, res, gate, rows, cols)


@pytest.mark.parametrize("rows,cols,res", [(2777, 4096, BF), (1531, 7168, F32), (700, 16384, F32),
                                           (2003, 4099, BF), (40001, 200, BF)])
def test_parts_alone(rows, cols, res):
    d = on_gpu(rows, cols, BF, res, "row", 32)
    n = torch.empty_like(d["y"])
    mxg.mxg_block_norm(d["x"], w_pre=d["w_pre"], n_out=n, eps=EPS)
    _, _, ref, mag = forward_ref(d, "row", 1.0, after=False)
    close(n, ref, mag, BF, 4, cols)
    xo = torch.empty_like(d["x"])
    mxg.mxg_block_norm(d["x"], d["y"], d["w_post"], d["gate"], GATES["row"], 0.5, xo, eps=EPS)
    ref, mag, _, _ = forward_ref(d, "row", 0.5)
    close(xo, ref, mag, res, 2, cols)
    for without in (("y",), ("dn",), ("dx_out",), ("dn", "y"), ("dx_out", "y")):
        has = lambda k: k not in without  # noqa: E731
        out = {"dx": torch.empty_like(d["x"]), "dy": torch.empty_like(d["y"]) if has("y") else None,
               "dw_post": torch.empty(cols, device=DEV), "dw_pre": torch.empty(cols, device=DEV),
               "dgate": torch.empty(rows, device=DEV) if has("y") else None}
        mxg.mxg_block_norm_backward(
            d["x"], d["y"] if has("y") else None, d["w_post"], d["gate"] if has("y") else None,
            GATES["row" if has("y") else "none"], 0.5, d["w_pre"], EPS,
            d["dx_out"] if has("dx_out") else None, d["dn"] if has("dn") else None,
            workspace=mxg.alloc_block_norm_workspace(rows, cols).fill_(255), **out)
        ref = backward_ref(d, "row", 0.5, after=has("y"), dxo=has("dx_out"), dn=has("dn"))
        close(out["dx"], *ref["dx"], res, 8, cols)
        if has("y"):
            close(out["dy"], *ref["dy"], BF, 8, cols)
            close(out["dw_post"], *ref["dw_post"], F32, 8, cols + rows)
            close(out["dgate"], *ref["dgate"], F32, 8, cols + rows)
        else:
            assert (out["dw_post"] == 0).all()
        if has("dn"):
            close(out["dw_pre"], *ref["dw_pre"], F32, 8, cols + rows)
        else:
            assert (out["dw_pre"] == 0).all()


@pytest.mark.parametrize("gate", ["col", "full"])
@pytest.mark.parametrize("rows,cols,dtype", [(2777, 4096, BF), (1531, 7168, F32), (700, 16384, F32),
                                             (613, 8201, BF), (2003, 4099, BF)])
def test_in_place(rows, cols, dtype, gate):
    d = on_gpu(rows, cols, dtype, dtype, gate, 33)
    want = forward(d, gate, 0.5)
    got = {k: v.clone() for k, v in d.items()}
    n = torch.empty_like(d["y"])
    mxg.mxg_block_norm(got["x"], got["y"], got["w_post"], got["gate"], GATES[gate], 0.5, got["x"],
                       got["w_pre"], n, EPS)
    assert torch.equal(got["x"], want[0]) and torch.equal(n, want[1])
    want = run_backward(d, gate, 0.5, rows, cols, dtype, dtype)
    for at in ("dn", "y"):
        got = {k: v.clone() for k, v in d.items()}
        out = run_backward(got, gate, 0.5, rows, cols, dtype, dtype, dx=got["dx_out"], dy=got[at])
        assert torch.equal(got["dx_out"], want["dx"]) and torch.equal(got[at], want["dy"])
        for k in ("dw_post", "dw_pre", "dgate"):
            assert torch.equal(out[k], want[k]), k


@pytest.mark.parametrize("rows,cols,res", [(2777, 4096, BF), (1531, 7168, F32), (700, 16384, F32),
                                           (40001, 200, BF), (2003, 4099, F32)])
def test_nan_stays_in_its_row(rows, cols, res):
    d = on_gpu(rows, cols, BF, res, "row", 34)
    hit = [5, rows // 2, rows - 1]
    d["y"][hit[0], 3] = float("nan")
    d["y"][hit[1], cols - 1] = float("nan")
    d["x"][hit[2], 1] = float("nan")
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[hit] = False
    got = forward(d, "row", 1.0)
    check_forward(got, forward_ref(d, "row", 1.0), BF, res, cols, keep)
    for r in hit[:2]:
        assert torch.isnan(got[0][r]).all() and torch.isnan(got[1][r]).all()
    out, ref = run_backward(d, "row", 1.0, rows, cols, BF, res), backward_ref(d, "row", 1.0)
    for k in ("dx", "dy", "dgate"):
        close(out[k][keep], ref[k][0][keep], ref[k][1][keep], {"dx": res, "dy": BF}.get(k, F32), 8, cols)
    assert torch.isnan(out["dw_post"]).all() and torch.isnan(out["dw_pre"]).all()


@pytest.mark.parametrize("rows,cols,res", [(2777, 4096, BF), (1531, 7168, F32), (700, 16384, F32),
                                           (100003, 40, BF), (2003, 4099, F32)])
def test_same_bits_every_time(rows, cols, res):
    d = on_gpu(rows, cols, BF, res, "row", 35)
    first, back = forward(d, "row", 1.0), run_backward(d, "row", 1.0, rows, cols, BF, res)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, forward(d, "row", 1.0)))
        again = run_backward(d, "row", 1.0, rows, cols, BF, res)
        assert all(torch.equal(back[k], again[k]) for k in back)


@pytest.mark.parametrize("pad", [8, 5])
def test_strided_rows(pad):
    rows, cols = 2777, 4096
    d = on_gpu(rows, cols, BF, BF, "full", 36)
    wide = {k: strided(v, pad) if v.dim() == 2 else v for k, v in d.items()}
    check_forward(forward(wide, "full", 0.5), forward_ref(d, "full", 0.5), BF, BF, cols)
    out = run_backward(wide, "full", 0.5, rows, cols, BF, BF)
    check_backward(out, backward_ref(d, "full", 0.5), BF, BF, "full", rows, cols)
