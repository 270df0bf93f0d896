"""The norm of a list of gradients and their clipping against 64 bits.

Bounds.  Squares are summed in fp32 over at most 64 + 8 terms (relative error
at most 72 2^-24 with the squares' own rounding) and in fp64 from there; the
square root halves it: 2^-18 of the norm covers that and the rounding to fp32.
The factor carries the same, and a clipped value one more product and one
rounding to its type: 2^-18 + u, u = 2^-24, 2^-8, 2^-11 (plus half of the
smallest subnormal where the result is one).
"""
import math

import pytest
import torch

from gpu_util import DEV, require_gpu
from moe_grouped_block_gb300 import mxg

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = {F32: 2.0 ** -24, BF: 2.0 ** -8, HF: 2.0 ** -11}
TINY = {F32: 2.0 ** -150, BF: 2.0 ** -134, HF: 2.0 ** -25}
REL = 2.0 ** -18


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def exact_norm(grads):
    return math.sqrt(math.fsum(float(g.double().pow(2).sum()) for g in grads))


def norm_of(grads):
    norm = torch.full((1,), 7.0, device=DEV)
    ws = mxg.alloc_grad_workspace()
    ws.fill_(255)
    mxg.mxg_grad_norm(mxg.grad_list(grads), norm, ws)
    return float(norm)


def clip(grads, max_norm, dst=None):
    norm = torch.full((1,), 7.0, device=DEV)
    ws = mxg.alloc_grad_workspace()
    ws.fill_(255)
    mxg.mxg_grad_clip(mxg.grad_list(grads, dst), max_norm, norm, ws)
    torch.cuda.synchronize()
    return float(norm)


def check(grads, dst, max_norm, norm):
    want = exact_norm(grads)
    assert abs(norm - want) <= REL * want
    factor = min(1.0, max_norm / (want + 1e-6))
    for g, d in zip(grads, dst):
        ref = g.double() * factor
        tol = (REL + U[d.dtype]) * ref.abs() + TINY[d.dtype]
        assert torch.isfinite(d).all() and not ((d.double() - ref).abs() > tol).any()


def draw(sizes, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(dtype).to(DEV) for n in sizes]


SIZES = [[1], [7], [8, 9, 1], [16384], [16385, 1], [100000, 3, 0, 65536], [1] * 65, [5] * 700, [0, 0],
         [3 << 20, 77]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%dx%d" % (len(s), max(s)))
@pytest.mark.parametrize("src,dst", [(BF, BF), (BF, F32), (HF, F32), (HF, HF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("ratio", [0.1, 3.0])
def test_clip(sizes, src, dst, ratio):
    grads = draw(sizes, src, 1, 0.5)
    out = [torch.full((n,), float("nan"), dtype=dst, device=DEV) for n in sizes]
    max_norm = ratio * exact_norm(grads)
    check(grads, out, max_norm, clip(grads, max_norm, out))
    assert abs(norm_of(grads) - exact_norm(grads)) <= REL * exact_norm(grads)


def test_mixed_list_in_place():
    grads = draw([1000, 3], BF, 2) + draw([33, 70000], F32, 3, 1e-3) + draw([511], HF, 4)
    kept = [g.clone() for g in grads]
    check(kept, grads, 0.25, clip(grads, 0.25))


@pytest.mark.parametrize("a,b", [(0, 1), (1, 0), (3, 3), (1, 2)])
@pytest.mark.parametrize("src,dst", [(BF, BF), (BF, F32), (F32, HF)])
def test_tensors_that_start_anywhere(a, b, src, dst):
    """Views that begin a few elements into a buffer; the neighbours stay."""
    n = 40003
    g = draw([n + 8], src, 5)[0]
    o = torch.full((n + 8,), 7.0, dtype=dst, device=DEV)
    grads, out = [g[a:a + n]], [o[b:b + n]]
    check(grads, out, 1.0, clip(grads, 1.0, out))
    assert (o[:b] == 7.0).all() and (o[b + n:] == 7.0).all()


@pytest.mark.parametrize("scale", [1e-36, 1e-30, 1e-22, 1e-15, 1e15, 1e18, 1e25, 1e33])
def test_neither_overflow_nor_underflow(scale):
    """Squares outside fp32's range."""
    grads = [(g.double() * scale).to(F32) for g in draw([5000, 3], F32, 6)]
    want = exact_norm(grads)
    assert abs(norm_of(grads) - want) <= REL * want
    grads.append(draw([999], F32, 7)[0])  # beside gradients of order one
    want = exact_norm(grads)
    assert abs(norm_of(grads) - want) <= REL * want


def test_large_and_small_in_one_vector():
    g = torch.ones(64, device=DEV)
    g[3], g[11] = 1e30, 1e-30
    want = exact_norm([g])
    assert abs(norm_of([g]) - want) <= REL * want


def test_zeros_and_nothing():
    assert norm_of([]) == 0.0
    assert norm_of([torch.empty(0, device=DEV)]) == 0.0
    z = torch.zeros(300, dtype=BF, device=DEV)
    assert clip([z], 1.0) == 0.0 and (z == 0).all()
    assert clip([], 1.0) == 0.0
    g = draw([300], F32, 8)
    clip(g, 0.0)
    assert (g[0] == 0).all()


def test_infinite_limit_copies():
    g = draw([5000], BF, 9)[0]
    o = torch.zeros(5000, dtype=BF, device=DEV)
    clip([g], float("inf"), [o])
    assert torch.equal(g, o)


def test_nan_and_infinity():
    """NaN anywhere makes the norm and every output NaN; an infinity gives the
    factor 0: finite values become 0 and the infinity itself NaN."""
    a, b = draw([9000, 50], F32, 10)
    b[7] = float("nan")
    assert math.isnan(norm_of([a, b]))
    x, y = a.clone(), b.clone()
    assert math.isnan(clip([x, y], 1.0)) and torch.isnan(x).all() and torch.isnan(y).all()
    b[7] = float("-inf")
    x, y = a.clone(), b.clone()
    assert clip([x, y], 1.0) == float("inf")
    assert (x == 0).all() and torch.isnan(y[7]) and (torch.cat([y[:7], y[8:]]) == 0).all()


def test_more_than_32_bits_of_elements():
    n = (1 << 31) + 5
    g = torch.zeros(n, dtype=BF, device=DEV)
    g[0], g[1 << 30], g[n - 1] = 3.0, 4.0, 12.0
    assert norm_of([g]) == 13.0
    clip([g], 6.5)
    assert float(g[0]) == 1.5 and float(g[1 << 30]) == 2.0 and float(g[n - 1]) == 6.0
    assert int((g != 0).sum()) == 3


def test_same_bits_streams_and_graphs():
    grads = draw([70000, 1000, 13] * 30, BF, 11)
    first = norm_of(grads)
    assert all(norm_of(grads) == first for _ in range(3))
    l, ws = mxg.grad_list(grads), mxg.alloc_grad_workspace()
    norm = torch.zeros(1, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mxg.mxg_grad_norm(l, norm, ws)
    s.synchronize()
    assert float(norm) == first
    out = [torch.zeros_like(g) for g in grads]
    lo = mxg.grad_list(grads, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxg.mxg_grad_clip(lo, 1.0, norm, ws)
    grads[0].mul_(0.5)  # the values are read when the graph runs
    graph.replay()
    torch.cuda.synchronize()
    check(grads, out, 1.0, float(norm))


def test_refusals():
    g = torch.zeros(8, device=DEV)
    norm, ws = torch.zeros(1, device=DEV), mxg.alloc_grad_workspace()
    with pytest.raises(ValueError):
        mxg.grad_list([torch.zeros(4, 4, device=DEV).t()[:2]])
    with pytest.raises(ValueError):
        mxg.grad_list([g], [g[:7]])
    with pytest.raises(ValueError):
        mxg.grad_list([g.int()])
    with pytest.raises(ValueError):
        mxg.grad_list([g.cpu()])
    l = mxg.grad_list([g])
    for bad in (-1.0, float("nan")):
        with pytest.raises(mxg.MxgError):
            mxg.mxg_grad_clip(l, bad, norm, ws)
    with pytest.raises(mxg.MxgError) as e:
        mxg.mxg_grad_norm(l, norm, ws[:16])
    assert e.value.code == 5
