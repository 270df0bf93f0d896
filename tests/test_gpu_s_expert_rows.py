"""Rows between the tokens' order and the experts', against 64 bits.

Bounds.  A copy is exact.  A sum of k products is rounded k times in fp32 and once to its type:
k 2^-24 of the sum of the magnitudes, and u of the result.  A product rounded to its type: u.  A dot
product over c columns is added in runs (a lane's columns: at most c / 32 + 32 of them) and ten
doublings: (c / 32 + 48) 2^-24 of the sum of the magnitudes.
"""
import pytest
import torch

from gpu_util import DEV, require_gpu
from moe_grouped_block_gb300 import mxg

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = {F32: 2.0 ** -24, BF: 2.0 ** -8, HF: 2.0 ** -11}
TINY = {F32: 2.0 ** -149, BF: 2.0 ** -134, HF: 2.0 ** -25}
NAN = float("nan")

# tokens, columns, experts, k
SHAPES = [(1, 8, 4, 1), (1, 4096, 8, 2), (5, 1, 3, 3), (37, 100, 8, 4), (300, 512, 16, 8),
          (64, 1000, 8, 5), (2000, 136, 64, 6), (130, 4100, 4, 2), (513, 257, 40, 32), (16, 7168, 64, 8),
          (50, 264, 40, 32), (70, 128, 32, 11), (3, 521, 9, 3), (1, 1033, 16, 9)]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def plan(n, E, k, seed, none=0.1, align=1, spare=0):
    """Distinct experts per token, some choices none; (row_of, counts, group_ws, capacity)."""
    g = torch.Generator().manual_seed(seed)
    expert = torch.rand(n, E, generator=g).argsort(1)[:, :k].to(torch.int32)
    expert[torch.rand(n, k, generator=g) < none] = -1
    if n > 3:
        expert[2] = -1
    counts = torch.empty(E, dtype=torch.int32, device=DEV)
    row_of = torch.empty(n, k, dtype=torch.int32, device=DEV)
    ws = torch.empty(2 * E + 1, dtype=torch.int64, device=DEV)
    mxg.mxg_route_rows(expert.to(DEV), counts, row_of, ws, align=align,
                       workspace=mxg.alloc_route_workspace(n, E, k))
    return row_of, counts, ws, n * k + E * (align - 1) + spare


def buffers(shape, dtype, ld, offset, fill):
    """(whole, view): rows ld apart, from `offset` elements into their buffer on."""
    rows, cols = shape
    whole = torch.full((rows * ld + offset + 8,), fill, dtype=dtype, device=DEV)
    return whole, whole[offset:offset + rows * ld].view(rows, ld)[:, :cols]


# elements more in a row, elements before the first; (7, 0) brings rows of 8 n + 1 columns, whose
# last element is no whole piece, to 16 bytes and more
LAYOUTS = [(0, 0), (8, 0), (7, 0), (3, 1)]


@pytest.mark.parametrize("n,cols,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("more,offset", LAYOUTS)
@pytest.mark.parametrize("align", [0, 16])
def test_dispatch(n, cols, E, k, dtype, more, offset, align):
    row_of, counts, ws, cap = plan(n, E, k, n + cols, align=max(align, 1), spare=3)
    _, x = buffers((n, cols), dtype, cols + more, offset, NAN)
    x.copy_(normal((n, cols), dtype, 1))
    whole, rows = buffers((cap, cols), dtype, cols + more, offset, 7.0)
    pad = dict(counts=counts, group_ws=ws) if align else {}
    mxg.mxg_dispatch(x, row_of, rows, **pad)
    want = torch.full((cap, cols), 7.0, dtype=dtype, device=DEV)
    if align:
        want[:int(ws[:E].sum())] = 0
    at = row_of.reshape(-1).long()
    who = torch.arange(n * k, device=DEV) // k
    want[at[at >= 0]] = x[who[at >= 0]]
    assert torch.equal(rows, want)
    whole.view(-1)[offset:offset + cap * (cols + more)].view(cap, -1)[:, :cols] = 7.0
    assert (whole == 7.0).all()  # nothing between the rows or around them


@pytest.mark.parametrize("n,cols,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("more,offset", LAYOUTS)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(n, cols, E, k, dtype, more, offset, weighted):
    row_of, _, _, cap = plan(n, E, k, n + cols)
    _, rows = buffers((cap, cols), dtype, cols + more, offset, NAN)
    rows.copy_(normal((cap, cols), dtype, 2))
    named = torch.zeros(cap, dtype=torch.bool, device=DEV)
    named[row_of[row_of >= 0].long()] = True
    rows[~named] = NAN  # rows that no token names are not read
    w = normal((n, k), F32, 3) if weighted else None
    if weighted:
        w[row_of < 0] = NAN  # nor is a weight beside no row
    whole, y = buffers((n, cols), dtype, cols + more, offset, 7.0)
    mxg.mxg_combine(rows, row_of, y, weight=w)
    want, size = torch.zeros(n, cols, dtype=torch.float64, device=DEV), 0
    for j in range(k):
        at = row_of[:, j].long()
        each = torch.where((at >= 0)[:, None], rows[at.clamp(min=0)].double(), 0.0)
        if weighted:
            each = each * torch.where(at >= 0, w[:, j].double(), 0.0)[:, None]
        want, size = want + each, size + each.abs()
    tol = k * 2.0 ** -24 * size + U[dtype] * (want.abs() + k * 2.0 ** -24 * size) + TINY[dtype]
    assert not ((y.double() - want).abs() > tol).any() and torch.isfinite(y).all()
    y.fill_(7.0)
    assert (whole == 7.0).all()


@pytest.mark.parametrize("n,cols,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("more,offset", LAYOUTS)
@pytest.mark.parametrize("align", [0, 16])
@pytest.mark.parametrize("parts", ["both", "rows", "weights", "in place"])
def test_combine_backward(n, cols, E, k, dtype, more, offset, align, parts):
    row_of, counts, ws, cap = plan(n, E, k, n + cols, align=max(align, 1), spare=2)
    _, dy = buffers((n, cols), dtype, cols + more, offset, NAN)
    dy.copy_(normal((n, cols), dtype, 4))
    w = normal((n, k), F32, 5)
    w[row_of < 0] = NAN
    y = normal((cap, cols), dtype, 6)
    named = torch.zeros(cap, dtype=torch.bool, device=DEV)
    named[row_of[row_of >= 0].long()] = True
    y[~named] = NAN
    whole, drows = buffers((cap, cols), dtype, cols + more, offset, 7.0)
    if parts == "in place":
        drows.copy_(y)
    dweight = torch.full((n, k), NAN, device=DEV)
    pad = dict(counts=counts, group_ws=ws) if align and parts != "weights" else {}
    mxg.mxg_combine_backward(dy, row_of, w, None if parts == "weights" else drows,
                             y_rows={"rows": None, "in place": drows}.get(parts, y),
                             dweight=None if parts == "rows" else dweight, **pad)
    for j in range(k):
        at = row_of[:, j].long()
        on, r = at >= 0, at[at >= 0]
        if parts != "rows":
            prod = dy[on].double() * y[r].double()
            tol = (cols / 32 + 48) * 2.0 ** -24 * prod.abs().sum(1) + 2.0 ** -140
            assert not ((dweight[on, j].double() - prod.sum(1)).abs() > tol).any()
            assert torch.isfinite(dweight[on, j]).all() and (dweight[~on, j] == 0).all()
        if parts != "weights":
            ref = dy[on].double() * w[on, j, None].double()
            # (the product in fp32, then its type)
            tol = (U[dtype] + 2.0 ** -23) * ref.abs() + TINY[dtype]
            assert not ((drows[r].double() - ref).abs() > tol).any()
    if parts in ("both", "rows"):
        padding = ~named
        padding[int(ws[:E].sum()) if align else 0:] = False
        assert (drows[padding] == 0).all()
        assert (drows[~named & ~padding] == 7.0).all()
        drows.fill_(7.0)
        assert (whole == 7.0).all()


def test_a_gradient_of_dispatch_is_a_combination_without_weights():
    """<dispatch(x), r> = <x, combine(r)> in whole numbers."""
    row_of, _, _, cap = plan(200, 16, 4, 7)
    g = torch.Generator().manual_seed(8)
    x = torch.randint(-4, 5, (200, 96), generator=g).float().to(DEV)
    r = torch.randint(-4, 5, (cap, 96), generator=g).float().to(DEV)
    rows, y = torch.zeros(cap, 96, device=DEV), torch.empty(200, 96, device=DEV)
    mxg.mxg_dispatch(x, row_of, rows)
    mxg.mxg_combine(r, row_of, y)
    assert float((rows.double() * r.double()).sum()) == float((x.double() * y.double()).sum())


def test_rows_outside_the_buffer_are_none():
    row_of = torch.tensor([[0, 9], [10, -1], [1 << 30, -(1 << 31)]], dtype=torch.int32, device=DEV)
    x, rows = normal((3, 40), BF, 9), torch.full((10, 40), 7.0, dtype=BF, device=DEV)
    mxg.mxg_dispatch(x, row_of, rows)
    assert torch.equal(rows[0], x[0]) and torch.equal(rows[9], x[0]) and (rows[1:9] == 7.0).all()
    y = torch.full((3, 40), 7.0, dtype=BF, device=DEV)
    mxg.mxg_combine(rows, row_of, y)
    assert torch.equal(y[0], (2 * x[0].float()).to(BF)) and (y[1:] == 0).all()
    dw = torch.full((3, 2), 7.0, device=DEV)
    mxg.mxg_combine_backward(x, row_of, None, None, y_rows=rows, dweight=dw)
    assert (dw[1:] == 0).all() and (dw[0] != 0).all()


def test_nothing_to_do():
    none = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    x, rows = torch.empty(0, 16, device=DEV), torch.full((4, 16), 7.0, device=DEV)
    mxg.mxg_dispatch(x, none, rows)
    mxg.mxg_combine(rows, none, x)
    mxg.mxg_combine_backward(x, none, None, rows)
    assert (rows == 7.0).all()
    # groups of padding alone
    counts = torch.tensor([0, 0], dtype=torch.int32, device=DEV)
    ws = torch.tensor([0, 3, 0, 0, 3], dtype=torch.int64, device=DEV)
    mxg.mxg_dispatch(x, none, rows, counts=counts, group_ws=ws)
    assert (rows[:3] == 0).all() and (rows[3] == 7.0).all()
    # no rows at all
    some = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    y, dw = torch.full((3, 16), 7.0, device=DEV), torch.full((3, 2), 7.0, device=DEV)
    empty = torch.empty(0, 16, device=DEV)
    mxg.mxg_dispatch(y, some, empty)
    mxg.mxg_combine(empty, some, y)
    assert (y == 0).all()
    mxg.mxg_combine_backward(y, some, None, empty, y_rows=empty, dweight=dw)
    assert (dw == 0).all()


def test_past_32_bits_of_elements():
    """Rows whose elements lie past 2^32 bytes and 2^31 elements."""
    cols, cap = 1 << 16, (1 << 15) + 70
    rows = torch.zeros(cap, cols, dtype=BF, device=DEV)
    at = torch.tensor([[cap - 1, 3], [cap - 2, 1 << 15]], dtype=torch.int32, device=DEV)
    x = normal((2, cols), BF, 10)
    mxg.mxg_dispatch(x, at, rows)
    assert torch.equal(rows[cap - 1], x[0]) and torch.equal(rows[1 << 15], x[1])
    y, dw = torch.empty_like(x), torch.empty(2, 2, device=DEV)
    mxg.mxg_combine(rows, at, y)
    assert torch.equal(y, (2 * x.float()).to(BF))
    mxg.mxg_combine_backward(x, at, None, rows, y_rows=rows, dweight=dw)
    want = x.double().square().sum(1, keepdim=True).expand(2, 2)
    assert not ((dw.double() - want).abs() > (cols / 32 + 48) * 2.0 ** -24 * want).any()


def test_same_bits_streams_and_graphs():
    row_of, counts, ws, cap = plan(900, 16, 4, 11, align=128)
    x, y_rows = normal((900, 768), BF, 12), normal((cap, 768), BF, 13)
    w = normal((900, 4), F32, 14)

    def all_three():
        rows = torch.zeros(cap, 768, dtype=BF, device=DEV)
        y, drows = torch.empty_like(x), torch.zeros_like(rows)
        dw = torch.empty(900, 4, device=DEV)
        mxg.mxg_dispatch(x, row_of, rows, counts=counts, group_ws=ws)
        mxg.mxg_combine(y_rows, row_of, y, weight=w)
        mxg.mxg_combine_backward(x, row_of, w, drows, y_rows=y_rows, dweight=dw, counts=counts,
                                 group_ws=ws)
        return rows, y, drows, dw
    first = all_three()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = all_three()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = all_three()
    graph.replay()
    torch.cuda.synchronize()
    for got in (all_three(), there, captured):
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_refusals():
    x, rows = normal((4, 16), BF, 15), normal((9, 16), BF, 16)
    at = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    w = torch.ones(4, 2, device=DEV)
    counts = torch.zeros(3, dtype=torch.int32, device=DEV)
    ws = torch.zeros(7, dtype=torch.int64, device=DEV)
    for call in (lambda: mxg.mxg_dispatch(x, at.long(), rows), lambda: mxg.mxg_dispatch(x, at[:3], rows),
                 lambda: mxg.mxg_dispatch(x, at, rows.float()), lambda: mxg.mxg_dispatch(x, at, rows[:, :8]),
                 lambda: mxg.mxg_dispatch(x, at, rows, counts=counts),
                 lambda: mxg.mxg_dispatch(x, at, rows, counts=counts, group_ws=ws[:6]),
                 lambda: mxg.mxg_dispatch(x, at, rows.cpu()), lambda: mxg.mxg_dispatch(x, at.view(-1), rows),
                 lambda: mxg.mxg_dispatch(x, at, rows[:1].expand(9, 16)),
                 lambda: mxg.mxg_combine(rows, at, x, weight=w.half()),
                 lambda: mxg.mxg_combine(rows, at, x.t()),
                 lambda: mxg.mxg_combine_backward(x, at, w, None),
                 lambda: mxg.mxg_combine_backward(x, at, w, rows, y_rows=rows[:8], dweight=w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mxg.mxg_combine_backward(x, at, w, rows, dweight=w.clone()),
                 lambda: mxg.mxg_combine_backward(x, at, w, rows, y_rows=rows),
                 lambda: mxg.mxg_dispatch(x, torch.zeros(4, 33, dtype=torch.int32, device=DEV), rows)):
        with pytest.raises(mxg.MxgError) as err:
            call()
        assert err.value.code == 1


def test_calls_from_several_threads():
    """Each thread on a stream of its own, with its own k and so its own kernel and shared memory."""
    import threading
    want, wrong = {}, []

    def call(k):
        row_of, _, _, cap = plan(64, 16, k, 20 + k)
        rows, x = normal((cap, 256), BF, k), normal((64, 256), BF, 30 + k)
        w = normal((64, k), F32, 50 + k)

        def once():
            y, d, dw = torch.empty_like(x), torch.zeros_like(rows), torch.empty(64, k, device=DEV)
            mxg.mxg_combine(rows, row_of, y, weight=w)
            mxg.mxg_combine_backward(x, row_of, w, d, y_rows=rows, dweight=dw)
            return y, d, dw
        return once
    calls = {k: call(k) for k in (1, 2, 3, 8)}
    for k, once in calls.items():
        want[k] = once()
    torch.cuda.synchronize()

    def work(k):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(100):
                got = calls[k]()
                side.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                    wrong.append(k)
    threads = [threading.Thread(target=work, args=(k,)) for k in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []
