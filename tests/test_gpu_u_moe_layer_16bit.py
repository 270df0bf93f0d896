"""The mixture-of-experts layer of examples/moe_layer_16bit.py: forward and gradients against the
same layer in 64 bits (with the experts that the library chose and the activation's inputs that
its checkpoint stands for), its steps, and a step captured in a CUDA graph.

Bounds.  A gradient passes at most seven roundings to bf16 (2^-8 relative) on its way -- gu, h, rows, dy's
share, dh, dgu, dxs or dl -- each independent, so its error in the 2-norm stays within 7 * 2^-8 of its
size.  The checkpoint's error is not among them: both sides start from what it stands for.
"""
import importlib.util
import os

import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
REL = 7 * 2.0 ** -8


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


def kept_values(layer):
    v = layer.q.view(torch.float8_e4m3fn).float().double()
    scale = torch.exp2(layer.sf.double() - 127)
    F, B = layer.F, (layer.F + 31) // 32
    spread = lambda s: s.repeat_interleave(32, 1)[:, :F]  # noqa: E731
    return v[:, :F] * spread(scale[:, :B]), v[:, F:] * spread(scale[:, B:])


def exact(layer, x, dy, kept):
    w = {k: v.double() for k, v in layer.weights.items()}
    x, dy, F = x.double(), dy.double(), layer.F
    expert, row_of = layer.expert.long(), layer.row_of.long()
    live = expert[:, 0] >= 0
    logits = (x @ w["wr"].t()).requires_grad_()
    p = torch.softmax(logits, 1)
    weight = p.gather(1, expert.clamp(min=0))
    weight = weight / weight.sum(1, keepdim=True) * live[:, None]
    counts = torch.bincount(expert[live].reshape(-1), minlength=layer.E).double()
    slope = layer.balance * layer.E * counts / counts.sum() / live.sum()
    loss = (slope * p[live].sum(0)).sum()
    # the experts' rows
    n = int(live.sum()) * layer.k
    token = torch.empty(n, dtype=torch.long, device=x.device)
    who = torch.empty(n, dtype=torch.long, device=x.device)
    t = torch.arange(len(x), device=x.device)[:, None].expand_as(row_of)
    token[row_of[live]], who[row_of[live]] = t[live], expert[live]
    xs = x[token]
    sizes = torch.bincount(who, minlength=layer.E).tolist()
    each = lambda a, b, f: torch.cat([f(r, m) for r, m in zip(a.split(sizes), b)])  # noqa: E731
    gu = each(xs, w["w1"], lambda r, m: r @ m.t())
    rows = each(gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:], w["w2"], lambda r, m: r @ m.t())
    wr = torch.zeros(n, dtype=torch.float64, device=x.device)
    wr[row_of[live]] = weight.detach()[live]
    y = torch.zeros_like(x).index_add(0, token, rows * wr[:, None])
    # and back
    drows = dy[token] * wr[:, None]
    dweight = torch.zeros_like(weight)
    dots = (dy[token] * rows).sum(1)
    dweight[live] = dots[row_of[live]]
    dh = each(drows, w["w2"], lambda r, m: r @ m)
    g, u = (v[:n] for v in kept)
    s = torch.sigmoid(g)
    dgu = torch.cat([dh * u * (s + g * s * (1 - s)), dh * g * s], 1)
    h = g * s * u
    grads = {"w2": torch.stack([a.t() @ b for a, b in zip(drows.split(sizes), h.split(sizes))]),
             "w1": torch.stack([a.t() @ b for a, b in zip(dgu.split(sizes), xs.split(sizes))])}
    dx = torch.zeros_like(x).index_add(0, token, each(dgu, w["w1"], lambda r, m: r @ m))
    (dl,) = torch.autograd.grad((weight * dweight).sum() + loss, logits)
    dl = torch.where(live[:, None], dl, 0.0)
    grads["wr"] = dl.t() @ x
    return y, float(loss.detach()), dx + dl @ w["wr"], grads


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("tokens,hidden,ffn,experts,k",
                         [(300, 256, 328, 16, 4), (65, 136, 72, 8, 2), (3, 64, 64, 8, 3), (2000, 64, 96, 64, 8)])
@pytest.mark.parametrize("masked", [False, True])
def test_gradients(example, tokens, hidden, ffn, experts, k, masked):
    layer = example.Layer(tokens, hidden, ffn, experts, k, balance=0.5)
    x, dy, mask = example.batch(tokens, hidden)
    y = layer.forward(x, mask if masked else None)
    kept = kept_values(layer)
    dx = layer.backward(x, dy)
    want_y, loss, want_dx, grads = exact(layer, x, dy, kept)
    assert off(y, want_y) <= REL and abs(float(layer.loss) - loss) <= 1e-4 * loss
    for name, v in layer.grads.items():
        assert off(v, grads[name]) <= REL, name
    assert off(dx, want_dx) <= REL
    if masked and tokens >= 10:
        assert (y[mask == 0] == 0).all() and (dx[mask == 0] == 0).all()


def test_steps_and_graph(example):
    layer = example.Layer(200, 128, 96, 8, 2, max_norm=0.01)
    x, target, mask = example.batch(200, 128)
    for _ in range(3):
        assert torch.isfinite(layer.step(x, target, 1.0, mask))
    total = sum(float(g.double().pow(2).sum()) for g in layer.grads.values()) ** 0.5
    assert total <= 0.01 * (1 + 1e-4)
    kept = {k: v.clone() for k, v in layer.weights.items()}
    want = [float(layer.step(x, target, 1.0, mask)) for _ in range(3)]
    for k, v in layer.weights.items():
        v.copy_(kept[k])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loss = layer.step(x, target, 1.0, mask)
    got = []
    for _ in range(3):
        graph.replay()
        got.append(float(loss))
    assert got == want  # the same bits, replayed


def test_padded_groups_feed_the_quantized_products():
    """Groups padded to 128 rows: the workspace that mxg_group_offsets would write, rows that the
    block-scaled quantize and product take as they are, and zeros in the padding."""
    from gpu_util import DEV, status_tensor
    from moe_grouped_block_gb300 import mxg
    T, K, N, E, k = 333, 256, 384, 4, 2
    R = (T * k + E * 127 + 127) // 128 * 128
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(T, K, generator=gen, device=DEV).to(torch.bfloat16)
    w = (torch.randn(E * N, K, generator=gen, device=DEV) * 0.1).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=gen, device=DEV)
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    expert, row_of, counts = i32(T, k), i32(T, k), i32(E)
    weight, groups, st = torch.empty(T, k, device=DEV), mxg.alloc_offsets(E), status_tensor()
    mxg.mxg_route(logits, expert, weight, counts, row_of=row_of, group_ws=groups, align=128,
                  rows_capacity=R, last_dim=K, workspace=mxg.alloc_route_workspace(T, E, k), dev_status=st)
    sizes = ((counts + 127) // 128 * 128).to(torch.int32)
    same = mxg.alloc_offsets(E)
    mxg.mxg_group_offsets(sizes, 1, K, R, same, st)
    assert torch.equal(groups, same)
    rows = torch.full((R, K), float("nan"), dtype=torch.bfloat16, device=DEV)
    mxg.mxg_dispatch(x, row_of, rows, counts=counts, group_ws=groups)
    live = int(groups[:E].sum())
    assert torch.isfinite(rows[:live]).all() and int((rows[:live].abs().sum(1) == 0).sum()) == live - T * k
    qx, qw = mxg.alloc_mxfp8(R, K), mxg.alloc_mxfp8(E * N, K)
    mxg.mxg_group_quantize(mxg.MXG_MXFP8_E4M3, mxg.MXG_ROWWISE, rows, R, K, groups, E, qx["q_row"],
                           qx["sf_row"], dev_status=st)
    mxg.mxg_group_quantize(mxg.MXG_MXFP8_E4M3, mxg.MXG_ROWWISE, w, E * N, K, None, E, qw["q_row"],
                           qw["sf_row"], dev_status=st)
    out = torch.empty(R, N, device=DEV)
    mxg.mxg_grouped_gemm(mxg.MXG_MXFP8_E4M3, mxg.MXG_FPROP_TN, (qx["q_row"], qx["sf_row"], None),
                         (qw["q_row"], qw["sf_row"], None), groups, E, R, N, K, C=out, dev_status=st)
    y = torch.empty(T, N, device=DEV)
    mxg.mxg_combine(out, row_of, y, weight=weight)
    assert int(st) == 0
    w64 = w.double().view(E, N, K)
    want = sum(torch.einsum("tk,tnk->tn", x.double(), w64[expert[:, j].long()]) * weight[:, j, None].double()
               for j in range(k))
    # each operand is off by half a step of E4M3 at most, 2^-4 of the value: independent, so well
    # within twice that in the 2-norm
    assert off(y, want) <= 2 * 2.0 ** -4


@pytest.mark.parametrize("tokens", [5, 300, 4000])
def test_calls_one_after_the_other(example, tokens):
    """Each kernel is set up while the one before it ends: calls that read what the last one wrote,
    into the same buffers over and over, give the same bits as calls that are waited for."""
    from gpu_util import DEV
    from moe_grouped_block_gb300 import mxg
    D, F, E, k = 128, 96, 16, 4

    def run(wait):
        layer = example.Layer(tokens, D, F, E, k, balance=0.3)
        x, dy, mask = example.batch(tokens, D)
        seen = []
        names = [n for n in dir(mxg) if n in (
            "mxg_route", "mxg_dispatch", "mxg_gated_act", "mxg_combine", "mxg_combine_backward",
            "mxg_gated_act_backward", "mxg_route_backward", "mxg_grouped_gemm_16bit")]
        kept = {n: getattr(mxg, n) for n in names}

        def waited(fn):
            def call(*a, **kw):
                fn(*a, **kw)
                if wait:
                    torch.cuda.synchronize()
            return call
        try:
            for n in names:
                setattr(mxg, n, waited(kept[n]))
            for _ in range(20):
                y = layer.forward(x, mask)
                dx = layer.backward(x, dy)
                seen += [y.clone(), dx.clone(), layer.expert.clone(), layer.dlogits.clone()]
                x = (x.float() + 0.1 * y.float() - 0.1 * dx.float()).to(torch.bfloat16)
        finally:
            for n in names:
                setattr(mxg, n, kept[n])
        torch.cuda.synchronize()
        return seen + [x, layer.weight, layer.loss] + list(layer.grads.values())
    # (x grows until, after some 14 rounds, it is past bf16's range: NaN is the same as NaN here)
    for a, b in zip(run(True), run(False)):
        assert torch.equal(torch.isnan(a), torch.isnan(b))
        assert torch.equal(a.nan_to_num(), b.nan_to_num())
    # and each operator on what it wrote itself a moment ago
    rows = torch.zeros(tokens, D, device=DEV)
    t = torch.arange(tokens, dtype=torch.int32, device=DEV)[:, None]
    back = tokens - 1 - t
    a = torch.randn(tokens, D, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV)
    want = a.clone()
    for i in range(60):  # an odd number of reversals in each round
        mxg.mxg_dispatch(a, back.contiguous(), rows)
        mxg.mxg_combine(rows, t, a)
    assert torch.equal(a, want)


def test_captured_behind_copies_and_other_streams():
    """In a graph, a call behind a copy, behind a fill, and behind two streams that meet."""
    from gpu_util import DEV
    from moe_grouped_block_gb300 import mxg
    n, D = 3000, 512
    at = torch.randperm(n, generator=torch.Generator().manual_seed(6)).to(torch.int32)[:, None].to(DEV)
    src = torch.randn(n, D, generator=torch.Generator(device=DEV).manual_seed(7), device=DEV)
    x, rows, y = torch.zeros(n, D, device=DEV), torch.zeros(n, D, device=DEV), torch.zeros(n, D, device=DEV)
    other, z = torch.zeros(n, D, device=DEV), torch.zeros(n, D, device=DEV)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        x.copy_(src)
        mxg.mxg_dispatch(x, at, rows)  # behind a copy
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            other.zero_()
            mxg.mxg_dispatch(src, at, other)  # behind a fill
        mxg.mxg_combine(rows, at, y)
        here.wait_stream(side)
        mxg.mxg_combine(other, at, z)  # behind both streams
        x.zero_()
    for i in range(5):
        src.mul_(1.5)
        rows.fill_(7.0), y.fill_(7.0), z.fill_(7.0)
        graph.replay()
        assert torch.equal(y, src) and torch.equal(z, src) and (x == 0).all()
