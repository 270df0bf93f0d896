"""Gradients of rows that must be numbers, and a layer's operators one behind the other on finite values.

Bounds: as in test_gpu_s_expert_rows.py; a chain is compared bit by bit.
"""
import importlib.util
import os

import pytest
import torch

from gpu_util import DEV, require_gpu
from moe_grouped_block_gb300 import mxg
from test_gpu_s_expert_rows import LAYOUTS, SHAPES, TINY, U, buffers, normal, plan

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "moe_layer_16bit.py")
    spec = importlib.util.spec_from_file_location("moe_layer_16bit", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("n,cols,E,k", SHAPES + [(900, 4096, 8, 2), (9000, 256, 16, 4)])
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("more,offset", LAYOUTS)
@pytest.mark.parametrize("parts", ["both", "rows", "weights", "in place"])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_backward(n, cols, E, k, dtype, more, offset, parts, weighted):
    """Every gradient is a number: rows and weights that take no part are NaN, as are the outputs before."""
    row_of, _, _, cap = plan(n, E, k, n + cols + 1)
    _, dy = buffers((n, cols), dtype, cols + more, offset, NAN)
    dy.copy_(normal((n, cols), dtype, 4))
    named = torch.zeros(cap, dtype=torch.bool, device=DEV)
    named[row_of[row_of >= 0].long()] = True
    y = normal((cap, cols), dtype, 6)
    y[~named] = NAN
    w = normal((n, k), F32, 5)
    w[row_of < 0] = NAN
    _, drows = buffers((cap, cols), dtype, cols + more, offset, NAN)
    if parts == "in place":
        drows.copy_(y)
    dweight = torch.full((n, k), NAN, device=DEV)
    mxg.mxg_combine_backward(dy, row_of, w if weighted else None, None if parts == "weights" else drows,
                             y_rows={"rows": None, "in place": drows}.get(parts, y),
                             dweight=None if parts == "rows" else dweight)
    for j in range(k):
        at = row_of[:, j].long()
        on, r = at >= 0, at[at >= 0]
        if parts != "rows":
            prod = dy[on].double() * y[r].double()
            tol = (cols / 32 + 48) * 2.0 ** -24 * prod.abs().sum(1) + 2.0 ** -140
            assert ((dweight[on, j].double() - prod.sum(1)).abs() <= tol).all()
            assert (dweight[~on, j] == 0).all()
        if parts != "weights":
            ref = dy[on].double() * (w[on, j, None].double() if weighted else 1.0)
            # (the product in fp32, then its type)
            tol = (U[dtype] + 2.0 ** -23) * ref.abs() + TINY[dtype]
            assert ((drows[r].double() - ref).abs() <= tol).all()
    if parts in ("both", "rows"):
        assert torch.isnan(drows[~named]).all()


@pytest.mark.parametrize("tokens,hidden,ffn,experts,k", [(5, 128, 96, 16, 4), (300, 128, 96, 16, 4),
                                                         (4000, 128, 96, 16, 4), (2000, 256, 64, 128, 8)])
def test_a_layer_again_and_again(example, tokens, hidden, ffn, experts, k):
    """Each kernel is set up while the one before it ends: calls that read what the last one wrote,
    into the same buffers over and over, give the bits of calls that are waited for, in every buffer of
    every round, all of them numbers."""
    names = ("mxg_route", "mxg_dispatch", "mxg_gated_act", "mxg_combine", "mxg_combine_backward",
             "mxg_gated_act_backward", "mxg_route_backward", "mxg_grouped_gemm_16bit")
    real = {name: getattr(mxg, name) for name in names}

    def run(wait):
        layer = example.Layer(tokens, hidden, ffn, experts, k, balance=0.3)
        x, dy, mask = example.batch(tokens, hidden)
        live = int(mask.sum()) * k
        seen = []

        def waited(fn):
            def call(*a, **kw):
                fn(*a, **kw)
                if wait:
                    torch.cuda.synchronize()
            return call
        try:
            for name in names:
                setattr(mxg, name, waited(real[name]))
            for _ in range(20):
                y = layer.forward(x, mask)
                dx = layer.backward(x, dy)
                now = dict(x=x, y=y, dx=dx, expert=layer.expert, row_of=layer.row_of, counts=layer.counts,
                           groups=layer.groups, weight=layer.weight, dweight=layer.dweight, loss=layer.loss,
                           slope=layer.slope, logits=layer.logits, dlogits=layer.dlogits,
                           q=layer.q[:live], sf=layer.sf[:live], rows=layer.rows[:live],
                           drows=layer.drows[:live], h=layer.h[:live], dgu=layer.dgu[:live], **layer.grads)
                seen.append({name: t.clone() for name, t in now.items()})
                x = x.float() + 0.1 * y.float() - 0.1 * dx.float()
                x = (x / x.square().mean(1, keepdim=True).sqrt()).to(BF)  # of the same size again
        finally:
            for name in names:
                setattr(mxg, name, real[name])
        torch.cuda.synchronize()
        return seen
    for a, b in zip(run(True), run(False)):
        for name in a:
            assert torch.isfinite(a[name].float()).all(), name
            assert torch.equal(a[name], b[name]), name
    assert a["counts"].sum() > 0 and (a["wr"] != 0).any() and (a["w1"] != 0).any() and (a["w2"] != 0).any()
