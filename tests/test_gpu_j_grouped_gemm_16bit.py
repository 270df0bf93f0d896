"""Grouped products on bf16 / fp16 operands against plain products in 64 bits.

Bounds.  Products of two 16-bit values are exact in fp32, so an output differs
from the exact value by at most the fp32 accumulation's error -- kdim + 8 steps
(the products, alpha, beta), each at most 2^-23 (truncation) of the sum of
magnitudes S = |alpha| sum |a||b| + |beta c| -- and by one rounding to the
output type, u |ref| with u = 2^-24, 2^-8, 2^-11 for fp32, bf16, fp16 (and half
of fp16's smallest subnormal, 2^-25).
Small integers are exact everywhere: those tests ask for equality.
"""
import itertools

import pytest
import torch

from gpu_util import DEV, require_gpu
from moe_grouped_block_gb300 import mxg

pytestmark = pytest.mark.gpu

FPROP, WGRAD, DGRAD = mxg.MXG_FPROP_TN, mxg.MXG_WGRAD_NT, mxg.MXG_DGRAD_NN
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
MODES = {"fprop": FPROP, "wgrad": WGRAD, "dgrad": DGRAD}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rows_ld(t, ld):
    """A copy of t whose rows lie ld elements apart (NaN between them)."""
    flat = t.reshape(-1, t.shape[-1])
    buf = torch.full((flat.shape[0], ld), float("nan"), dtype=t.dtype, device=t.device)
    buf[:, :t.shape[-1]] = flat
    if t.dim() == 3:
        return buf.as_strided(t.shape, (t.shape[1] * ld, ld, 1))
    return buf[:, :t.shape[-1]]


def up8(n):
    return (n + 7) // 8 * 8


def group_ws(sizes, cap):
    ws = mxg.alloc_offsets(len(sizes), DEV)
    mxg.mxg_group_offsets_unaligned(torch.tensor(sizes, dtype=torch.int64, device=DEV), 1, 1, cap, ws)
    return ws


def inputs(mode, sizes, N, K, dtype, seed, cap=None, integers=False, lda=None, ldb=None):
    g = torch.Generator().manual_seed(seed)
    G, M = len(sizes), cap if cap is not None else sum(sizes)

    def draw(*shape):
        if integers:
            return torch.randint(-3, 4, shape, generator=g).to(dtype)
        return torch.randn(*shape, generator=g).to(dtype)
    a = draw(M, K if mode == FPROP else N)
    b = draw(M, K) if mode == WGRAD else draw(G, N, K)
    live = sum(sizes)
    a[live:] = float("nan")  # rows past the groups take no part
    if mode == WGRAD:
        b[live:] = float("nan")
    return (a, b, rows_ld(a.to(DEV), lda or up8(a.shape[-1])), rows_ld(b.to(DEV), ldb or up8(K)))


def reference(mode, a, b, sizes, alpha=None, beta=None, c=None):
    """(exact, sum of magnitudes, contraction length per output) in fp64."""
    A, B, off = a.double(), b.double(), 0
    ref, mag, kd = [], [], []
    for g, m in enumerate(sizes):
        r = slice(off, off + m)
        off += m
        if mode == FPROP:
            p, q = A[r], B[g].t()
        elif mode == DGRAD:
            p, q = A[r], B[g]
        else:
            p, q = A[r].t(), B[r]
        al = 1.0 if alpha is None else alpha[g]
        be = 0.0 if beta is None else beta[g]
        old = 0.0
        if be != 0.0:
            old = be * (c[g].double() if mode == WGRAD else c[r].double())
        ref.append(al * (p @ q) + old)
        mag.append(abs(al) * (p.abs() @ q.abs()) + (old.abs() if be != 0.0 else 0.0))
        kd.append(p.shape[1])
    if mode == WGRAD:
        return torch.stack(ref), torch.stack(mag), max(kd)
    return torch.cat(ref), torch.cat(mag), max(kd)


def check(got, ref, mag, kdim, out):
    assert torch.isfinite(got).all()
    tol = (kdim + 8) * 2.0 ** -23 * mag + U[out] * ref.abs() + (2.0 ** -25 if out == torch.float16 else 0)
    bad = (got.double() - ref).abs() > tol + 1e-300
    assert not bad.any(), "%d of %d outputs out of bounds, worst %g" % (
        int(bad.sum()), bad.numel(), float(((got.double() - ref).abs() - tol).max()))


def run(mode, A, B, sizes, N, K, out, cap=None, alpha=None, beta=None, c=None, ldc=None, status=None):
    G, M = len(sizes), cap if cap is not None else sum(sizes)
    shape = {FPROP: (M, N), DGRAD: (M, K), WGRAD: (G, N, K)}[mode]
    C = torch.full(shape, 7.0, dtype=out, device=DEV) if c is None else c.to(DEV)
    if ldc:
        C = rows_ld(C, ldc)
    f = lambda v: None if v is None else torch.tensor(v, dtype=torch.float32, device=DEV)  # noqa: E731
    mxg.mxg_grouped_gemm_16bit(mode, A, B, group_ws(sizes, M), G, M, N, K, f(alpha), f(beta), C,
                               dev_status=status)
    torch.cuda.synchronize()
    return C


SHAPES = [  # sizes, N, K
    ([1], 8, 8),
    ([1, 0, 1], 128, 64),
    ([5, 0, 3, 17], 136, 72),
    ([128, 256, 64], 256, 256),
    ([63, 64, 65], 264, 200),
    ([0, 0, 130, 0], 24, 520),
    ([257, 1, 255, 31], 392, 320),
    ([300, 513], 520, 136),
    ([2] * 40, 72, 264),
]


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%s_%d_%d" % (len(s[0]), s[1], s[2]))
def test_products(mode, dtype, shape):
    mode, (sizes, N, K) = MODES[mode], shape
    a, b, A, B = inputs(mode, sizes, N, K, dtype, 1)
    ref, mag, kd = reference(mode, a, b, sizes)
    for out in (torch.float32, dtype):
        check(run(mode, A, B, sizes, N, K, out).cpu(), ref, mag, kd, out)


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("N,K", [(1, 1), (7, 3), (129, 65), (255, 131), (1, 300), (300, 1), (61, 257)])
def test_odd_widths_and_strides(mode, N, K):
    """N and K of any value with rows that are multiples of 8 apart; C of any
    row stride and alignment.  NaN fills the gaps between rows."""
    mode, sizes = MODES[mode], [3, 0, 70, 129]
    a, b, A, B = inputs(mode, sizes, N, K, torch.bfloat16, 2, lda=up8(max(N, K)) + 8,
                        ldb=up8(K) + 16)
    ref, mag, kd = reference(mode, a, b, sizes)
    cols = N if mode == FPROP else K
    for out, ldc in itertools.product((torch.float32, torch.bfloat16), (None, cols + 1, up8(cols) + 24)):
        C = run(mode, A, B, sizes, N, K, out, ldc=ldc)
        check(C.cpu(), ref, mag, kd, out)
        if ldc:  # what lies between the rows stays
            gap = C.as_strided((C.numel() // cols, ldc - cols), (ldc, 1), C.storage_offset() + cols)
            assert torch.isnan(gap[:-1]).all()


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_integers_are_exact(mode, dtype):
    mode, sizes, N, K = MODES[mode], [130, 0, 1, 257, 64], 328, 264
    a, b, A, B = inputs(mode, sizes, N, K, dtype, 3, integers=True)
    ref, _, _ = reference(mode, a, b, sizes)
    assert torch.equal(run(mode, A, B, sizes, N, K, torch.float32).cpu().double(), ref)


def test_gradients_are_the_differences_of_fprop():
    """The product is linear, and small integers are exact in every step: the
    differences of <dY, fprop> are the gradients to the last bit."""
    sizes, N, K, dt = [40, 0, 129, 7], 136, 72, torch.bfloat16
    x, w, X, W = inputs(FPROP, sizes, N, K, dt, 4, integers=True)
    g = torch.Generator().manual_seed(5)
    dy = torch.randint(-2, 3, (sum(sizes), N), generator=g).to(dt)
    dx = torch.randint(-1, 2, x.shape, generator=g).to(dt)
    dw = torch.randint(-1, 2, w.shape, generator=g).to(dt)
    f = lambda xx, ww: (run(FPROP, xx.to(DEV), ww.to(DEV), sizes, N, K, torch.float32)  # noqa: E731
                        .cpu().double() * dy.double()).sum()
    gx = run(DGRAD, dy.to(DEV), W, sizes, N, K, torch.float32).cpu().double()
    gw = run(WGRAD, dy.to(DEV), X, sizes, N, K, torch.float32).cpu().double()
    assert f(x + dx, w) - f(x, w) == (gx * dx.double()).sum()
    assert f(x, w + dw) - f(x, w) == (gw * dw.double()).sum()


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_alpha_beta(mode, out):
    mode, sizes, N, K = MODES[mode], [129, 0, 64, 3], 136, 264
    a, b, A, B = inputs(mode, sizes, N, K, torch.bfloat16, 6)
    g = torch.Generator().manual_seed(7)
    shape = {FPROP: (196, N), DGRAD: (196, K), WGRAD: (4, N, K)}[mode]
    c = torch.randn(*shape, generator=g).to(out)
    alpha, beta = [0.5, 2.0, -1.25, 0.0], [1.0, -0.5, 0.0, 2.0]
    if mode == WGRAD:
        c[2] = float("nan")  # not read where beta is 0
    else:
        c[129:193] = float("nan")
    ref, mag, kd = reference(mode, a, b, sizes, alpha, beta, c)
    check(run(mode, A, B, sizes, N, K, out, alpha=alpha, beta=beta, c=c).cpu(), ref, mag, kd, out)


@pytest.mark.parametrize("mode", ["fprop", "dgrad"])
def test_rows_past_the_groups_are_not_written(mode):
    mode, sizes, N, K, cap = MODES[mode], [5, 130], 264, 136, 512
    a, b, A, B = inputs(mode, sizes, N, K, torch.bfloat16, 8, cap=cap)
    ref, mag, kd = reference(mode, a, b, sizes)
    C = run(mode, A, B, sizes, N, K, torch.float32, cap=cap).cpu()
    check(C[:135], ref, mag, kd, torch.float32)
    assert (C[135:] == 7.0).all()


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nan_and_infinity_stay_in_their_group(mode, value):
    mode, sizes, N, K = MODES[mode], [70, 1, 33, 200, 0, 15], 136, 136
    a, b, A, B = inputs(mode, sizes, N, K, torch.bfloat16, 9)
    ref, mag, kd = reference(mode, a, b, sizes)
    lo, hi = 71, 104  # group 2, next to groups 1 and 3
    A[lo:hi] = value
    if mode == WGRAD:
        B[lo:hi] = value
    else:
        B[2] = value
    C = run(mode, A, B, sizes, N, K, torch.float32).cpu()
    if mode == WGRAD:
        keep = [0, 1, 3, 4, 5]
        check(C[keep], ref[keep], mag[keep], kd, torch.float32)
        assert not torch.isfinite(C[2]).any()
    else:
        keep = torch.cat([torch.arange(lo), torch.arange(hi, sum(sizes))])
        check(C[keep], ref[keep], mag[keep], kd, torch.float32)
        assert not torch.isfinite(C[lo:hi]).any()


@pytest.mark.parametrize("mode", list(MODES))
def test_no_rows_at_all(mode):
    mode, N, K = MODES[mode], 136, 72
    one = torch.ones(8, up8(max(N, K)), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(3, N, K, dtype=torch.bfloat16, device=DEV)
    for cap in (0, 8):
        A, B = one[:, :K if mode == FPROP else N], one[:, :K] if mode == WGRAD else w
        shape = {FPROP: (8, N), DGRAD: (8, K), WGRAD: (3, N, K)}[mode]
        for beta, want in ((None, 0.0), ([1.0, 0.5, 0.0], None)):
            C = torch.full(shape, 7.0, dtype=torch.float32, device=DEV)
            bt = None if beta is None else torch.tensor(beta, device=DEV)
            mxg.mxg_grouped_gemm_16bit(mode, A, B, group_ws([0, 0, 0], cap), 3, cap, N, K, None, bt, C)
            C = C.cpu()
            if mode != WGRAD:
                assert (C == 7.0).all()
            elif beta is None:
                assert (C == want).all()
            else:
                assert (C == torch.tensor(beta).view(3, 1, 1) * 7.0).all()


def test_sizes_that_do_not_fit_are_recorded():
    """A negative size counts as 0 and rows past M_cap are dropped."""
    N, K, cap = 72, 64, 100
    a, b, A, B = inputs(FPROP, [60, 0, 40], N, K, torch.bfloat16, 10)
    ws = torch.tensor([60, -5, 90, 0, 0, 0, 0], dtype=torch.int64, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    C = torch.empty(cap, N, device=DEV)
    mxg.mxg_grouped_gemm_16bit(FPROP, A, B, ws, 3, cap, N, K, C=C, dev_status=st)
    assert int(st) == mxg.MXG_DEV_NEG_SIZE | mxg.MXG_DEV_SUM_OVER_CAPACITY
    ref, mag, kd = reference(FPROP, a, b, [60, 0, 40])
    check(C.cpu(), ref, mag, kd, torch.float32)


@pytest.mark.parametrize("mode", list(MODES))
def test_many_groups(mode):
    mode, N, K = MODES[mode], 24, 40
    g = torch.Generator().manual_seed(11)
    sizes = torch.randint(0, 4, (1024,), generator=g).tolist()
    a, b, A, B = inputs(mode, sizes, N, K, torch.float16, 12)
    ref, mag, kd = reference(mode, a, b, sizes)
    check(run(mode, A, B, sizes, N, K, torch.float32).cpu(), ref, mag, kd, torch.float32)


@pytest.mark.parametrize("mode", list(MODES))
def test_long_contraction(mode):
    """4096 and more products an output."""
    mode, sizes, N, K = MODES[mode], [4100, 30], 144, 4104
    if mode == DGRAD:
        N, K = 4104, 144
    elif mode == FPROP:
        sizes = [30, 100]
    a, b, A, B = inputs(mode, sizes, N if mode != WGRAD else 72, K if mode != WGRAD else 72,
                        torch.bfloat16, 13)
    N, K = (72, 72) if mode == WGRAD else (N, K)
    ref, mag, kd = reference(mode, a, b, sizes)
    check(run(mode, A, B, sizes, N, K, torch.float32).cpu(), ref, mag, kd, torch.float32)


def test_fp32_outputs_of_very_long_sums():
    """Sums of 32768 products.  512 of them are added at a time by truncation --
    32 additions, each losing less than 2^-23 of the sum so far -- and the 64 such
    sums by rounding to nearest: 32 2^-23 + 64 2^-24 = 8e-6 of the result at most,
    and half of that for sums that grow (added by truncation alone, the 2048 steps
    lost 4e-5)."""
    g = torch.Generator(device=DEV).manual_seed(20)
    dy = torch.randn(32768, 264, generator=g, device=DEV).to(torch.bfloat16)
    x = torch.randn(32768, 136, generator=g, device=DEV).to(torch.bfloat16)
    C = run(WGRAD, dy, x, [32768], 264, 136, torch.float32)
    ref = dy.double().t() @ x.double()
    assert float((C[0].double() - ref).norm() / ref.norm()) <= 4e-6


def test_outputs_past_32_bits():
    """C of more than 2^31 elements, an odd last group."""
    N, K, sizes = 32776, 64, [40000, 25537]
    M = sum(sizes)
    g = torch.Generator(device=DEV).manual_seed(14)
    X = torch.randint(-3, 4, (M, K), generator=g, device=DEV).to(torch.bfloat16)
    W = torch.randint(-3, 4, (2, N, K), generator=g, device=DEV).to(torch.bfloat16)
    C = run(FPROP, X, W, sizes, N, K, torch.float32)
    for r in (0, 39999, 40000, M - 1):
        want = W[0 if r < 40000 else 1].double() @ X[r].double()
        assert torch.equal(C[r].double(), want)


def test_another_stream_and_a_graph():
    sizes, N, K = [100, 30], 136, 264
    a, b, A, B = inputs(FPROP, sizes, N, K, torch.bfloat16, 15)
    ref, mag, kd = reference(FPROP, a, b, sizes)
    ws = group_ws(sizes, 130)
    C = torch.zeros(130, N, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mxg.mxg_grouped_gemm_16bit(FPROP, A, B, ws, 2, 130, N, K, C=C)
    s.synchronize()
    check(C.cpu(), ref, mag, kd, torch.float32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxg.mxg_grouped_gemm_16bit(FPROP, A, B, ws, 2, 130, N, K, C=C)
    # the sizes are read when the graph runs
    ws.copy_(group_ws([20, 110], 130))
    C.zero_()
    graph.replay()
    torch.cuda.synchronize()
    ref, mag, kd = reference(FPROP, a, b, [20, 110])
    check(C.cpu(), ref, mag, kd, torch.float32)


def test_same_bits_every_time():
    for mode in (FPROP, DGRAD, WGRAD):
        sizes, N, K = [3, 200, 12], 520, 1032
        a, b, A, B = inputs(mode, sizes, N, K, torch.bfloat16, 16)
        first = run(mode, A, B, sizes, N, K, torch.float32)
        for _ in range(3):
            assert torch.equal(first, run(mode, A, B, sizes, N, K, torch.float32))


SHARED = [  # mode, sizes, N, K: few outputs, long contractions
    ("fprop", [1], 1000, 4104), ("fprop", [33], 520, 4100), ("fprop", [100], 520, 4100),
    ("fprop", [300], 300, 4096), ("fprop", [5, 0, 3], 256, 2100), ("fprop", [40], 4088, 1030),
    ("dgrad", [1], 4104, 1000), ("dgrad", [257], 4097, 264), ("dgrad", [0, 20, 70], 1100, 700),
    ("wgrad", [5000], 300, 200), ("wgrad", [2048], 512, 512), ("wgrad", [1, 0, 40, 7, 9000], 129, 70),
    ("wgrad", [4500, 4400, 4200], 50, 1032),
]


@pytest.mark.parametrize("case", SHARED, ids=lambda c: "%s_%s_%d_%d" % (c[0], len(c[1]), c[2], c[3]))
def test_shared_contractions(case):
    mode, sizes, N, K = case
    mode, G, M = MODES[mode], len(sizes), sum(sizes)
    cap = M + 5
    a, b, A, B = inputs(mode, sizes, N, K, torch.bfloat16, 21, cap=cap)
    alpha, beta = [0.5 + g for g in range(G)], [(-1.0) ** g * (g % 3) for g in range(G)]
    g = torch.Generator().manual_seed(22)
    c = torch.randn(*{FPROP: (cap, N), DGRAD: (cap, K), WGRAD: (G, N, K)}[mode], generator=g)
    for out in (torch.float32, torch.bfloat16):
        ref, mag, kd = reference(mode, a, b, sizes)
        C = run(mode, A, B, sizes, N, K, out, cap=cap)
        live = C if mode == WGRAD else C[:M]
        check(live.cpu(), ref, mag, kd, out)
        if mode != WGRAD:
            assert (C[M:] == 7.0).all()
        assert torch.equal(C, run(mode, A, B, sizes, N, K, out, cap=cap))
        old = c.to(out)
        ref, mag, kd = reference(mode, a, b, sizes, alpha, beta, old)
        C = run(mode, A, B, sizes, N, K, out, cap=cap, alpha=alpha, beta=beta, c=old)
        check((C if mode == WGRAD else C[:M]).cpu(), ref, mag, kd, out)
    a, b, A, B = inputs(mode, sizes, N, K, torch.float16, 23, integers=True)
    ref, _, _ = reference(mode, a, b, sizes)
    assert torch.equal(run(mode, A, B, sizes, N, K, torch.float32).cpu().double(), ref)


def test_shared_contractions_with_sizes_that_do_not_fit():
    """Clusters without a unit, and sizes past the capacity or below zero."""
    N, K = 256, 4096
    a, b, A, B = inputs(FPROP, [2, 3, 1], N, K, torch.bfloat16, 24)
    for sizes, taken in (([2, 3, 1], [2, 3, 1]), ([0, 0, 0], [0, 0, 0]), ([-4, 2, 0], [0, 2, 0]),
                         ([3, 900, 1], [3, 3, 0])):
        ws = torch.tensor(sizes + [0, 0, 0, 0], dtype=torch.int64, device=DEV)
        C = torch.full((6, N), 7.0, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        mxg.mxg_grouped_gemm_16bit(FPROP, A, B, ws, 3, 6, N, K, None, None, C, dev_status=status)
        torch.cuda.synchronize()
        m = sum(taken)
        if m:
            ref, mag, kd = reference(FPROP, a, b, taken)
            check(C[:m].cpu(), ref, mag, kd, torch.float32)
        assert (C[m:] == 7.0).all()
        assert bool(status.item()) == (sizes != taken)


def test_binding_refusals():
    x = torch.zeros(16, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(2, 32, 64, dtype=torch.bfloat16, device=DEV)
    c = torch.zeros(16, 32, device=DEV)
    ws = group_ws([8, 8], 16)
    call = lambda a=x, b=w, o=c: mxg.mxg_grouped_gemm_16bit(  # noqa: E731
        FPROP, a, b, ws, 2, 16, 32, 64, C=o)
    with pytest.raises(ValueError):
        call(a=x.half())
    with pytest.raises(ValueError):
        call(a=x.float(), b=w.float())
    with pytest.raises(ValueError):
        call(a=x.t().contiguous().t())
    with pytest.raises(ValueError):
        call(b=torch.zeros(2, 40, 64, dtype=torch.bfloat16, device=DEV)[:, :32])
    with pytest.raises(mxg.MxgError):
        call(o=c.half())
    with pytest.raises(ValueError):
        call(a=x.cpu())
