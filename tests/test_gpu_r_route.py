"""Routing against 64 bits: choices, weights, counts, the balance loss and its slopes, the rows,
and the gradient of the logits.

Bounds.  With R the span of the exponents' arguments (for softmax the row's range of logits, for
sigmoid its largest magnitude), __expf is off by at most 2 + 1.173 R units in the last place
(2^-23 each) and the subtraction before it by R 2^-24: u(R) = 2^-23 (2 + 1.7 R).  A share or a weight is
a quotient of such a value and a sum of such values, at most 1024 of them added in runs of 32 and five
doublings, rounded a few times more: 2 u(R) + 48 * 2^-24.  Where exponentials leave fp32's normal range
2^-126 is added.  The loss adds shares of one sign, no more than 256 in a row: 256 * 2^-24 more.  A
gradient p (a - sum a p) + q (b - sum b q) carries three such factors: 3 times the bound, relative to
the sum of the magnitudes, and the rounding to its type.
"""
import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu, status_tensor
from moe_grouped_block_gb300 import mxg

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = {F32: 2.0 ** -24, BF: 2.0 ** -8, HF: 2.0 ** -11}
SOFT, SIG = mxg.MXG_SCORE_SOFTMAX, mxg.MXG_SCORE_SIGMOID
TINY = 2.0 ** -126
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def route(logits, k, mask=None, plan=True, losses=True, capacity=None, align=1, last_dim=1, status=None,
          ws=None, **kw):
    T, E = logits.shape
    new = lambda shape, dtype, fill: torch.full(shape, fill, dtype=dtype, device=DEV)  # noqa: E731
    out = {"expert": new((T, k), torch.int32, 77), "weight": new((T, k), F32, NAN),
           "counts": new((E,), torch.int32, 77)}
    if losses:
        out.update(loss=new((1,), F32, NAN), slope=new((E,), F32, NAN))
    if plan:
        out.update(row_of=new((T, k), torch.int32, 77), group_ws=new((2 * E + 1,), torch.int64, 77))
    if ws is None:
        ws = mxg.alloc_route_workspace(T, E, k)
        ws.fill_(255)
    mxg.mxg_route(logits, mask=mask, workspace=ws, align=align, rows_capacity=capacity,
                  last_dim=last_dim, dev_status=status, **out, **kw)
    return out


def rows_of(expert, E, align, capacity, last_dim):
    """The rows in plain numpy."""
    flat = np.asarray(expert).reshape(-1)
    ok = (flat >= 0) & (flat < E)
    counts = np.bincount(flat[ok], minlength=E)
    sizes = -(-counts // align) * align
    ends = np.cumsum(sizes)
    cap = capacity // align * align
    row = np.full(flat.shape, -1, np.int64)
    for e in range(E):
        at = np.nonzero(flat == e)[0]
        row[at] = ends[e] - sizes[e] + np.arange(at.size)
    row[row >= cap] = -1
    kept = np.minimum(ends, cap)
    ws = np.concatenate([np.diff(np.concatenate([[0], kept])), [0], kept * last_dim])
    return counts, row.reshape(np.shape(expert)), ws


def exact(logits, k, mask=None, score=SOFT, normalize=True, scale=1.0, balance=0.0):
    """In 64 bits on the CPU; live: the tokens that take part."""
    x = logits.double().cpu()
    T, E = x.shape
    live = (x > -INF).any(1) | torch.isnan(x).any(1)
    if mask is not None:
        live &= mask.cpu().bool()
    order = torch.sort(torch.where(torch.isnan(x), INF, x) + 0.0, dim=1, descending=True, stable=True)
    expert = order.indices[:, :k]
    expert = torch.where((order.values[:, :k] > -INF) & live[:, None], expert, -1)
    at = expert.clamp(min=0)
    s = torch.softmax(x, 1) if score == SOFT else torch.sigmoid(x)
    if score == SOFT:
        p = s
    else:  # (shares of sigmoids that underflow, by their logarithms)
        p = torch.softmax(torch.nn.functional.logsigmoid(x), 1)
    chosen = p if normalize else s
    w = torch.where(expert >= 0, chosen.gather(1, at), 0.0)
    if normalize:
        w = w / w.sum(1, keepdim=True)
    w = torch.where(expert >= 0, scale * w, 0.0)
    counts = torch.bincount(expert[expert >= 0].reshape(-1), minlength=E)
    n = int(live.sum())
    slope = balance * E * counts.double() / max(1, int(counts.sum())) / max(1, n)
    loss = float((slope * p[live].sum(0)).sum())
    span = float((x - x.amax(1, keepdim=True)).where(x > -INF, torch.zeros(())).abs().max()) if T else 0.0
    if score == SIG and T:
        span = float(x.where(x.abs() < INF, torch.zeros(())).abs().max())
    return dict(expert=expert, weight=w, counts=counts, slope=slope, loss=loss, live=live, p=p, s=s,
                rel=2 * 2.0 ** -23 * (2 + 1.7 * span) + 48 * 2.0 ** -24)


def check(logits, k, mask=None, align=1, capacity=None, last_dim=1, **kw):
    T, E = logits.shape
    st = status_tensor()
    got = route(logits, k, mask, align=align, capacity=capacity, last_dim=last_dim, status=st, **kw)
    want = exact(logits, k, mask, **kw)
    cap = T * k + E * (align - 1) if capacity is None else capacity
    counts, row, ws = rows_of(want["expert"].numpy(), E, align, cap, last_dim)
    assert torch.equal(got["expert"].cpu().long(), want["expert"])
    assert torch.equal(got["counts"].cpu().long(), want["counts"])
    assert np.array_equal(got["row_of"].cpu().numpy(), row)
    assert np.array_equal(got["group_ws"].cpu().numpy(), ws)
    assert int(st) == (mxg.MXG_DEV_SUM_OVER_CAPACITY if (-(-counts // align) * align).sum()
                       > cap // align * align else 0)
    w = got["weight"].cpu().double()
    off = (w - want["weight"]).abs()
    tiny = TINY * abs(kw.get("scale", 1.0))
    assert not (off > want["rel"] * want["weight"].abs() + tiny).any()
    slope = got["slope"].cpu().double()
    assert not ((slope - want["slope"]).abs() > 6 * 2.0 ** -24 * want["slope"].abs()).any()
    bound = (want["rel"] + 256 * 2.0 ** -24) * abs(want["loss"])
    assert abs(float(got["loss"]) - want["loss"]) <= bound + TINY * T * E
    return got, want


def draw(T, E, dtype, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g) * spread + torch.randn(E, generator=g) * 0.5
    return x.to(dtype).to(DEV)


SHAPES = [(1, 1, 1), (1, 8, 2), (7, 2, 2), (64, 8, 2), (300, 13, 5), (2000, 8, 8), (65, 64, 8),
          (5000, 64, 6), (129, 100, 3), (1000, 256, 8), (33, 257, 32), (70, 512, 9), (500, 1000, 10),
          (40, 1024, 32), (3000, 16, 1), (1500, 64, 20), (9000, 32, 4)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("score,normalize", [(SOFT, True), (SOFT, False), (SIG, True), (SIG, False)])
def test_route(T, E, k, dtype, score, normalize):
    g = torch.Generator().manual_seed(T)
    mask = (torch.rand(T, generator=g) < 0.9).to(torch.uint8).to(DEV) if T % 2 == 0 else None
    check(draw(T, E, dtype, T + E), k, mask, align=128 if E % 8 == 0 else 1, last_dim=3, score=score,
          normalize=normalize, scale=2.5, balance=0.3)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("E,k", [(8, 3), (64, 8), (1024, 32)])
def test_equal_logits_go_to_the_lower_expert(dtype, E, k):
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-1, 2, (700, E), generator=g).float()
    x[::3] *= -0.0  # zeros of both signs
    x[1] = 5.0
    check(x.to(dtype).to(DEV), k, balance=1.0)


def test_logits_of_minus_infinity_are_not_chosen():
    x = draw(400, 20, F32, 4)
    x[::2, 3:] = -INF      # three left
    x[5] = -INF            # none left: as a masked token
    x[7] = torch.finfo(F32).min
    x[9, 1:] = torch.finfo(F32).min
    for score in (SOFT, SIG):
        for normalize in (True, False):
            got, want = check(x, 6, score=score, normalize=normalize, balance=0.5, align=4)
            assert (got["expert"][5] == -1).all() and not want["live"][5]
    mask = torch.zeros(400, dtype=torch.bool, device=DEV)
    got, _ = check(x, 6, mask, balance=0.5)  # nothing takes part
    assert float(got["loss"]) == 0 and (got["slope"] == 0).all() and (got["counts"] == 0).all()


@pytest.mark.parametrize("level", [-30.0, -95.0, -200.0, 60.0])
def test_sigmoids_that_underflow(level):
    """Shares and normalised weights of tokens whose scores vanish or are all 1."""
    x = draw(200, 24, F32, 5) + level
    got, want = check(x, 4, score=SIG, normalize=True, balance=0.5)
    assert torch.allclose(got["weight"].sum(1).cpu(), torch.ones(200))
    check(x, 4, score=SIG, normalize=False, balance=0.5)


def test_nan_and_infinity():
    x = draw(300, 40, F32, 6)
    x[10, 7], x[11, 8], x[12, 3] = NAN, INF, -NAN
    got = route(x, 4, balance=0.1)
    assert int(got["expert"][10, 0]) == 7 and int(got["expert"][11, 0]) == 8
    assert int(got["expert"][12, 0]) == 3
    bad = torch.isnan(got["weight"]).all(1).nonzero()[:, 0].tolist()
    assert bad == [10, 11, 12] and torch.isnan(got["loss"]).all()
    assert not torch.isnan(got["slope"]).any()
    clean = x.clone()
    clean[10:13] = 0
    others = torch.ones(300, dtype=torch.bool)
    others[10:13] = False
    assert torch.equal(route(clean, 4)["weight"].cpu()[others], got["weight"].cpu()[others])


@pytest.mark.parametrize("align", [1, 16, 128, 1000])
@pytest.mark.parametrize("T", [40, 6000])
def test_rows_past_the_capacity_are_dropped(T, align):
    x = draw(T, 12, F32, 7)
    for capacity in (0, 1, 100, T, 3 * T + 5):
        check(x, 3, align=align, capacity=capacity, last_dim=7, balance=0.2)


def test_only_what_is_asked_for():
    x = draw(5000, 64, F32, 8)
    full = route(x, 4, balance=0.2)
    for plan in (True, False):
        for losses in (True, False):
            got = route(x, 4, plan=plan, losses=losses, balance=0.2)
            assert all(torch.equal(got[name], full[name]) for name in got)


@pytest.mark.parametrize("offset,ld", [(0, 72), (0, 67), (1, 64), (3, 65)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_strided_logits(offset, ld, dtype):
    x = draw(600, 64, dtype, 9)
    flat = torch.full((600 * ld + 8,), NAN, dtype=dtype, device=DEV)
    view = flat[offset:offset + 600 * ld].view(600, ld)[:, :64]
    view.copy_(x)
    a, b = route(x, 8, balance=0.1), route(view, 8, balance=0.1)
    assert all(torch.equal(a[name], b[name]) for name in a)


def test_no_tokens():
    x = torch.empty(0, 16, device=DEV)
    got = route(x, 2, balance=1.0)
    assert (got["counts"] == 0).all() and (got["slope"] == 0).all() and float(got["loss"]) == 0
    assert (got["group_ws"] == 0).all()


# ------------------------------------------------------------------ rows of given choices
@pytest.mark.parametrize("T,E,k", [(0, 4, 2), (1, 1, 1), (50, 8, 2), (3000, 64, 8), (20000, 10, 3),
                                   (4000, 1024, 5), (100000, 256, 1)])
@pytest.mark.parametrize("align", [1, 128])
def test_rows_of_given_choices(T, E, k, align):
    """Values outside the experts are none; the same expert twice is two rows."""
    g = torch.Generator().manual_seed(T + E)
    expert = torch.randint(-2, E + 2, (T, k), generator=g, dtype=torch.int32)
    if T > 2 and k > 1:
        expert[1] = 0
        expert[2] = torch.iinfo(torch.int32).min
    counts = torch.full((E,), 7, dtype=torch.int32, device=DEV)
    row = torch.full((T, k), 7, dtype=torch.int32, device=DEV)
    ws = torch.full((2 * E + 1,), 7, dtype=torch.int64, device=DEV)
    work = mxg.alloc_route_workspace(T, E, k)
    work.fill_(255)
    mxg.mxg_route_rows(expert.to(DEV), counts, row, ws, align=align, last_dim=5, workspace=work)
    c, r, w = rows_of(expert.numpy(), E, align, T * k + E * (align - 1), 5)
    assert np.array_equal(counts.cpu().numpy(), c) and np.array_equal(row.cpu().numpy(), r)
    assert np.array_equal(ws.cpu().numpy(), w)
    counts.fill_(9)
    mxg.mxg_route_rows(expert.to(DEV), counts, workspace=work)
    assert np.array_equal(counts.cpu().numpy(), c)


def test_rows_agree_with_the_routing():
    x = draw(7000, 64, BF, 10)
    a = route(x, 6, align=128, last_dim=64)
    counts, row = torch.empty_like(a["counts"]), torch.empty_like(a["row_of"])
    ws = torch.empty_like(a["group_ws"])
    mxg.mxg_route_rows(a["expert"], counts, row, ws, align=128, last_dim=64,
                       workspace=mxg.alloc_route_workspace(7000, 64, 6))
    assert torch.equal(counts, a["counts"]) and torch.equal(row, a["row_of"])
    assert torch.equal(ws, a["group_ws"])


# ------------------------------------------------------------------ the gradient
def exact_gradient(logits, want, dweight, dloss, score, normalize, scale, with_loss):
    """By automatic differentiation in 64 bits; and the sum of the magnitudes that the formula adds."""
    x = logits.double().cpu().requires_grad_()
    expert, live = want["expert"], want["live"]
    s = torch.softmax(x, 1) if score == SOFT else torch.sigmoid(x)
    p = s if score == SOFT else torch.softmax(torch.nn.functional.logsigmoid(x), 1)
    chosen = torch.where(expert >= 0, (p if normalize else s).gather(1, expert.clamp(min=0)), 0.0)
    w = chosen
    if normalize:
        w = chosen / torch.where(live, chosen.sum(1), 1.0)[:, None]
    total = x.sum() * 0
    db = torch.zeros(expert.shape, dtype=torch.float64)
    if dweight is not None:
        db = torch.where(expert >= 0, dweight.double().cpu(), 0.0) * scale
        total = total + (w * db)[live].sum()
    a = torch.zeros(x.shape[1], dtype=torch.float64)
    if with_loss:
        a = want["slope"] * dloss
        total = total + (p[live] * a).sum()
    (grad,) = torch.autograd.grad(total, x)
    with torch.no_grad():
        size = p * (a.abs() + (a.abs() * p).sum(1, keepdim=True))
        each = w.abs() * (db.abs() + (db.abs() * w.abs()).sum(1, keepdim=True))
        if score == SOFT and not normalize:
            size = size + p * (db.abs() * w).sum(1, keepdim=True)
        # An expert that is not chosen has no part in normalised weights, its gradient through them is
        # exactly 0.  Automatic differentiation forms it as p (x - x), with x a sum of at most 34 terms
        # each |db| w / (sum of the chosen p) at most: off by 2^-53 * 40 of it.
        if normalize:
            chosen_p = torch.where(live, chosen.sum(1), 1.0)[:, None]
            noise = 2.0 ** -47 * p * (db.abs().sum(1, keepdim=True)) / chosen_p
            size = size + noise / (3 * want["rel"])
        size = size.scatter_add(1, expert.clamp(min=0), torch.where(expert >= 0, each, 0.0))
    return torch.where(live[:, None], grad, 0.0), torch.where(live[:, None], size, 0.0)


def check_gradient(logits, k, mask=None, use=("weight", "loss"), score=SOFT, normalize=True, scale=1.0,
                   balance=0.0, seed=1):
    T, E = logits.shape
    got = route(logits, k, mask, score=score, normalize=normalize, scale=scale, balance=balance)
    want = exact(logits, k, mask, score, normalize, scale, balance)
    assert torch.equal(got["expert"].cpu().long(), want["expert"])
    g = torch.Generator().manual_seed(seed)
    dw = torch.randn(T, k, generator=g).to(DEV) if "weight" in use else None
    if dw is not None:
        dw[got["expert"] < 0] = NAN  # beside no expert: any value
    dloss = torch.full((1,), 1.7, device=DEV) if "loss" in use else None
    d = torch.full_like(logits, NAN)
    mxg.mxg_route_backward(logits, got["expert"], d, dweight=dw, score=score, normalize=normalize,
                           scale=scale, slope=got["slope"] if "loss" in use else None, dloss=dloss)
    saved = dict(want, slope=got["slope"].double().cpu())
    ref, size = exact_gradient(logits, saved, dw, 1.7, score, normalize, scale, "loss" in use)
    tol = 3 * want["rel"] * size + U[logits.dtype] * ref.abs() + TINY * 8
    if logits.dtype is HF:
        tol = tol + 2.0 ** -25
    d = d.double().cpu()
    assert torch.isfinite(d).all() and not ((d - ref).abs() > tol).any()
    assert (d[~want["live"]] == 0).all()


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("score,normalize", [(SOFT, True), (SOFT, False), (SIG, True), (SIG, False)])
def test_gradient(T, E, k, dtype, score, normalize):
    g = torch.Generator().manual_seed(T)
    mask = (torch.rand(T, generator=g) < 0.9).to(torch.uint8).to(DEV) if T % 2 == 0 else None
    check_gradient(draw(T, E, dtype, T + E), k, mask, score=score, normalize=normalize, scale=2.5,
                   balance=30.0)


@pytest.mark.parametrize("use", [("weight",), ("loss",), ()])
@pytest.mark.parametrize("score,normalize", [(SOFT, True), (SOFT, False), (SIG, True), (SIG, False)])
def test_either_gradient_alone(use, score, normalize):
    check_gradient(draw(500, 48, F32, 11), 4, use=use, score=score, normalize=normalize, balance=9.0)


def test_gradient_with_logits_of_minus_infinity():
    x = draw(300, 20, F32, 12)
    x[::2, 3:] = -INF
    x[5] = -INF
    for normalize in (True, False):
        check_gradient(x, 6, normalize=normalize, balance=5.0)


def test_gradient_by_differences():
    """d(sum of weights . c + loss) / d(logit) by central differences of the 64-bit forward pass,
    without a change of the chosen experts."""
    x = draw(6, 12, F32, 13)
    for score, normalize in [(SOFT, True), (SOFT, False), (SIG, True), (SIG, False)]:
        kw = dict(score=score, normalize=normalize, scale=1.5, balance=4.0)
        got = route(x, 3, **kw)
        c = torch.randn(6, 3, generator=torch.Generator().manual_seed(2)).to(DEV)
        d = torch.empty_like(x)
        mxg.mxg_route_backward(x, got["expert"], d, dweight=c, score=score, normalize=normalize,
                               scale=1.5, slope=got["slope"], dloss=torch.ones(1, device=DEV))

        def value(logits):
            r = exact(logits, 3, **kw)
            assert torch.equal(r["expert"], got["expert"].cpu().long())
            return float((r["weight"] * c.double().cpu()).sum()) + r["loss"]
        x64, h = x.double(), 1e-5
        # (the magnitudes in a gradient add up to less than 10 here)
        tol = 3 * exact(x, 3, **kw)["rel"] * 10 + 1e-8
        for t in range(6):
            for e in range(12):
                up, down = x64.clone(), x64.clone()
                up[t, e] += h
                down[t, e] -= h
                slope = (value(up) - value(down)) / (2 * h)
                # the difference's own error: h^2 of a third derivative of order 10, and 1e-15 / h
                assert abs(float(d[t, e]) - slope) <= tol


@pytest.mark.parametrize("dtype", [F32, BF])
def test_gradient_in_place_and_strided(dtype):
    x = draw(700, 64, dtype, 14)
    got = route(x, 5, balance=1.0)
    dw, dloss = torch.randn(700, 5, device=DEV), torch.ones(1, device=DEV)
    plain = torch.empty_like(x)
    kw = dict(dweight=dw, slope=got["slope"], dloss=dloss)
    mxg.mxg_route_backward(x, got["expert"], plain, **kw)
    for ld, offset in [(72, 0), (65, 0), (64, 1)]:
        flat = torch.full((700 * ld + 8,), 3.0, dtype=dtype, device=DEV)
        view = flat[offset:offset + 700 * ld].view(700, ld)
        mxg.mxg_route_backward(x, got["expert"], view[:, :64], **kw)
        assert torch.equal(view[:, :64], plain) and (view[:, 64:] == 3.0).all()
    y = x.clone()
    mxg.mxg_route_backward(y, got["expert"], y, **kw)
    assert torch.equal(y, plain)


# ------------------------------------------------------------------ how it is called
def test_same_bits_streams_and_graphs():
    x = draw(20000, 64, F32, 15)
    first = route(x, 8, balance=0.1, align=128)
    for _ in range(3):
        again = route(x, 8, balance=0.1, align=128)
        assert all(torch.equal(first[name], again[name]) for name in first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = route(x, 8, balance=0.1, align=128)
    side.synchronize()
    assert all(torch.equal(first[name], there[name]) for name in first)
    # two captured calls that share a workspace, replayed one after the other
    ws = mxg.alloc_route_workspace(20000, 64, 8)
    y = draw(300, 64, F32, 16)
    want = route(y, 8, balance=0.1)
    graphs = []
    for logits, align in ((x, 128), (y, 1)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = route(logits, 8, balance=0.1, align=align, ws=ws)
        graphs.append((graph, out))
    for _ in range(2):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first[name], graphs[0][1][name]) for name in first)
    assert all(torch.equal(want[name], graphs[1][1][name]) for name in want)


def test_large_batch():
    """More choices than a chunk's 16 bits, and many chunks."""
    T, E, k = 300000, 8, 2
    x = draw(T, E, BF, 17)
    got, _ = check(x, k, balance=0.1, align=128)
    check_gradient(x[:100000], k, balance=0.1)


def test_past_32_bits_of_logits():
    T, E, k = (1 << 21) + 77, 1024, 2
    x = torch.empty(T, E, dtype=BF, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(19)
    for part in x.split(1 << 19):
        part.normal_(generator=gen)
    got = route(x, k, balance=0.1)
    order = got["row_of"].view(-1).long().argsort()
    assert torch.equal(got["row_of"].view(-1).long().sort().values, torch.arange(T * k, device=DEV))
    flat = got["expert"].view(-1)[order]
    assert (flat[1:] >= flat[:-1]).all()  # sorted by expert, and within one by token
    same = flat[1:] == flat[:-1]
    assert (order[1:][same] > order[:-1][same]).all()
    d = torch.empty_like(x)
    dw = torch.randn(T, k, generator=gen, device=DEV)
    mxg.mxg_route_backward(x, got["expert"], d, dweight=dw, normalize=False)
    for rows in (slice(0, 50), slice(T // 2, T // 2 + 50), slice(T - 50, T)):
        want = exact(x[rows], k)
        assert torch.equal(got["expert"][rows].cpu().long(), want["expert"])
        p = torch.softmax(x[rows].double(), 1)
        at, g = got["expert"][rows].long(), dw[rows].double()
        chosen = p.gather(1, at)
        ref = -p * (g * chosen).sum(1, keepdim=True)
        ref = ref.scatter_add(1, at, g * chosen)
        size = p * (g.abs() * chosen).sum(1, keepdim=True)
        size = size.scatter_add(1, at, g.abs() * chosen)
        tol = 3 * want["rel"] * size + U[BF] * ref.abs() + TINY * 8
        assert not ((d[rows].double() - ref).abs() > tol).any()


def test_refusals():
    x = draw(10, 8, F32, 18)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    e, w, c = i32(10, 2), torch.zeros(10, 2, device=DEV), i32(8)
    ws = mxg.alloc_route_workspace(10, 8, 2)
    ok = dict(logits=x, expert=e, weight=w, counts=c, workspace=ws)
    mxg.mxg_route(**ok)
    for kw in (dict(expert=e.long()), dict(weight=w.double()), dict(counts=i32(7)), dict(logits=x.int()),
               dict(logits=x[:9]), dict(mask=torch.ones(9, dtype=torch.uint8, device=DEV)),
               dict(row_of=i32(10, 2)), dict(slope=torch.zeros(9, device=DEV)),
               dict(loss=torch.zeros(2, device=DEV)), dict(expert=i32(20)),
               dict(weight=torch.zeros(2, 10, device=DEV).t()), dict(logits=x.cpu()),
               dict(logits=x[:1].expand(10, 8))):
        with pytest.raises(ValueError):
            mxg.mxg_route(**dict(ok, **kw))
    for kw, code in ((dict(scale=NAN), 1), (dict(balance=INF), 1), (dict(workspace=None), 1),
                     (dict(workspace=ws[:8]), 5), (dict(score=2), 1), (dict(align=0), 1),
                     (dict(expert=i32(10, 9), weight=torch.zeros(10, 9, device=DEV)), 1)):
        with pytest.raises(mxg.MxgError) as err:
            mxg.mxg_route(**dict(ok, **kw))
        assert err.value.code == code, kw
    with pytest.raises(mxg.MxgError):  # a slope without the loss's gradient
        mxg.mxg_route_backward(x, e, torch.empty_like(x), slope=torch.zeros(8, device=DEV))
    with pytest.raises(ValueError):
        mxg.mxg_route_backward(x, e, torch.empty(10, 8, dtype=BF, device=DEV))
