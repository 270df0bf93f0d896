"""The gated activation, its 8-bit checkpoint and its backward pass, against 64 bits.

Bounds.  h = x sigmoid(z) u: __expf(-z) is off by 2 + 1.173 |z| units (2^-23 each) and z itself, where it
is a polynomial, by three roundings (3 |z| 2^-24); the exponential's share e / (1 + e) of the sigmoid's error
is at most 1, and it is at most |z| = 20 before that share is below 1e-8 on one side, or the result below
fp16's subnormals and 2^-126 relative to one on the other.  With the quotient (2 units) and two products:
2^-23 (6 + 1.173 |z| + 2 |z|) <= 2^-23 (6 + 3.2 |z|) relative, and one rounding to the type.  Beyond |z| of
87 __fdividef may return 0 for a value below x 2^-126.  The gradient's slope s + x s (1 - s) z' adds
terms: the same relative bound of the sum of their magnitudes, doubled, and the rounding of 1 - s, 2^-24 of
x s z'.  The checkpoint is exact: largest magnitude, power of two and one rounding to nearest even.
"""
import math

import pytest
import torch

from gpu_util import DEV, require_gpu
from moe_grouped_block_gb300 import mxg

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, HF: 2.0 ** -11}
TINY = {BF: 2.0 ** -134, HF: 2.0 ** -25}
SILU, GELU = mxg.MXG_ACT_SILU, mxg.MXG_ACT_GELU_TANH
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def normal(shape, dtype, seed, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def z_of(x, act):
    return x if act == SILU else 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)


def dz_of(x, act):
    return torch.ones_like(x) if act == SILU else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x ** 2)


def close(got, want, tol, dtype):
    tol = tol + U[dtype] * (want.abs() + tol) + TINY[dtype]
    return torch.isfinite(got).all() and not ((got.double() - want).abs() > tol).any()


def check_h(h, gate, up, act, dtype):
    x = gate.double()
    z = z_of(x, act)
    a = x * torch.sigmoid(z)
    u = 1.0 if up is None else up.double()
    eps = 2.0 ** -23 * (6 + 3.2 * z.abs().clamp(max=90))
    assert close(h, a * u, eps * (a * u).abs() + (x * u).abs() * 2.0 ** -126, dtype)


def kept(x):
    """Bytes of E4M3 (signs of zeros and NaN aside, their values) and scale bytes, by definition."""
    rows, cols = x.shape
    qs, sfs = [], []
    for part in x.double().split(32, 1):
        fine = torch.isfinite(part)
        top = torch.where(fine, part.abs(), 0.0).amax(1, keepdim=True)
        m, e = torch.frexp(top)  # [0.5, 1): 448 = 0.875 2^9
        e = torch.where(top > 0, e - 9 + (m > 0.875).to(e.dtype), -127).clamp(-127, 127)
        # fp32's subnormals take the least scale
        e = torch.where(top < 2.0 ** -126, -127, e)
        v = part * torch.exp2(-e.double())
        _, b = torch.frexp(v)
        step = torch.exp2((b - 1).clamp(min=-6).double() - 3)
        v = torch.where(fine, torch.round(v / step) * step, NAN)
        qs.append(v)
        sfs.append((e + 127).to(torch.uint8))
    return torch.cat(qs, 1), torch.cat(sfs, 1)


def values(q, sf, cols):
    """What a checkpoint of one matrix stands for, in 64 bits."""
    v = q.view(torch.float8_e4m3fn).float().double()
    return v * torch.exp2(sf.double() - 127).repeat_interleave(32, 1)[:, :cols]


def check_kept(q, sf, parts):
    cols, blocks = parts[0].shape[1], (parts[0].shape[1] + 31) // 32
    for i, x in enumerate(parts):
        want, scale = kept(x)
        got = q[:, i * cols:(i + 1) * cols].contiguous().view(torch.float8_e4m3fn).float().double()
        assert torch.equal(sf[:, i * blocks:(i + 1) * blocks], scale)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(), want.nan_to_num())


def check_backward(q, sf, dh, dgate, dup, h, act, dtype):
    cols, blocks = dh.shape[1], (dh.shape[1] + 31) // 32
    x = values(q[:, :cols].contiguous(), sf[:, :blocks], cols)
    gated = dup is not None
    u = values(q[:, cols:2 * cols].contiguous(), sf[:, blocks:], cols) if gated else torch.ones_like(x)
    z, dz, d = z_of(x, act), dz_of(x, act), dh.double()
    s, rest = torch.sigmoid(z), torch.sigmoid(-z)
    a = x * s
    eps = 2.0 ** -23 * (6 + 3.2 * z.abs().clamp(max=90))
    floor = (x.abs() + 1) * 2.0 ** -126
    slope, size = s + a * rest * dz, s + (a * rest * dz).abs()
    err = 2 * eps * size + 2.0 ** -24 * (a * dz).abs() + floor * (1 + dz)
    # (three products after the slope)
    assert close(dgate, d * u * slope, (d * u).abs() * (err + 3 * 2.0 ** -24 * size), dtype)
    if gated:
        assert close(dup, d * a, d.abs() * (eps * a.abs() + floor), dtype)
    if h is not None:
        assert close(h, a * u, u.abs() * (eps * a.abs() + floor), dtype)


def wide(rows, cols, dtype, more, offset, fill, parts=2):
    """(buffer, views): `parts` matrices side by side in rows that are `more` elements longer."""
    ld = parts * cols + more
    buf = torch.full((rows * ld + offset + 16,), fill, dtype=dtype, device=DEV)
    m = buf[offset:offset + rows * ld].view(rows, ld)
    return buf, [m[:, i * cols:(i + 1) * cols] for i in range(parts)]


SHAPES = [(1, 1), (1, 32), (3, 7), (5, 48), (4, 64), (17, 100), (130, 1408), (33, 4099), (2, 14336),
          (700, 16), (257, 272)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("act", [SILU, GELU])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("more,offset", [(0, 0), (16, 0), (5, 1)])
def test_both_directions(rows, cols, dtype, act, gated, more, offset):
    parts = 2 if gated else 1
    blocks = (cols + 31) // 32
    _, ins = wide(rows, cols, dtype, more, offset, NAN, parts)
    for i, m in enumerate(ins):
        m.copy_(normal((rows, cols), dtype, 1 + i))
    gate, up = ins[0], ins[1] if gated else None
    hbuf, (h,) = wide(rows, cols, dtype, more, offset, 7.0, 1)
    qbuf = torch.full((rows, parts * cols + more), 0x55, dtype=torch.uint8, device=DEV)
    q = qbuf[:, :parts * cols]
    sf = torch.full((rows, parts * blocks), 0x55, dtype=torch.uint8, device=DEV)
    alone = torch.empty(rows, cols, dtype=dtype, device=DEV)
    mxg.mxg_gated_act(gate, h, up=up, act=act, q=q, sf=sf)
    mxg.mxg_gated_act(gate, alone, up=up, act=act)
    check_h(h, gate, up, act, dtype)
    assert torch.equal(h, alone)
    check_kept(q, sf, ins)
    assert (qbuf[:, parts * cols:] == 0x55).all()

    dh = normal((rows, cols), dtype, 5, 0.1)
    dbuf, outs = wide(rows, cols, dtype, more, offset, 7.0, parts)
    again = torch.full((rows, cols), NAN, dtype=dtype, device=DEV)
    dup = outs[1] if gated else None
    mxg.mxg_gated_act_backward(q, sf, dh, outs[0], dup=dup, act=act, h=again)
    check_backward(q, sf, dh, outs[0], dup, again, act, dtype)
    kept_outs = [o.clone() for o in outs]
    mxg.mxg_gated_act_backward(q, sf, dh, outs[0], dup=dup, act=act)
    assert all(torch.equal(a, b) for a, b in zip(kept_outs, outs))
    for m in outs + [h]:
        m.fill_(7.0)
    assert (dbuf == 7.0).all() and (hbuf == 7.0).all()


@pytest.mark.parametrize("act", [SILU, GELU])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_every_value_of_a_type(act, dtype):
    """All 16-bit numbers up to half the largest as the gate (above, a kept value may round
    past the type's range)."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    x = bits.view(dtype)
    x = x[x.float().abs() <= torch.finfo(dtype).max / 2].to(DEV)
    x = x[:x.numel() // 32 * 32].view(-1, 32).contiguous()
    one = torch.ones_like(x)
    h, (q, sf) = torch.empty_like(x), mxg.alloc_act_checkpoint(x.shape[0], 32, True)
    mxg.mxg_gated_act(x, h, up=one, act=act, q=q, sf=sf)
    check_h(h, x, one, act, dtype)
    check_kept(q, sf, [x, one])
    dg, du, again = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    mxg.mxg_gated_act_backward(q, sf, one, dg, dup=du, act=act, h=again)
    check_backward(q, sf, one, dg, du, again, act, dtype)


@pytest.mark.parametrize("scale", [0.0, 1e-39, 1e-36, 1e-20, 1e20, 1e37])
def test_blocks_of_any_magnitude(scale):
    x = normal((40, 96), torch.float64, 6, 1.0)
    x = (x * scale).to(BF)
    x[3, 32:64] = 0
    x[4] = 448.0 * 2 ** -3
    x[5] = torch.tensor(448.0 * 2 ** 4) * (1 + 2.0 ** -7)  # just over: the next scale
    h, (q, sf) = torch.empty_like(x), mxg.alloc_act_checkpoint(40, 96, False)
    mxg.mxg_gated_act(x, h, q=q, sf=sf)
    check_kept(q, sf, [x])
    # a kept value is off by at most half a step: 2^-4 of it, or 2^-10 of the scale
    off = (values(q, sf, 96) - x.double()).abs()
    least = torch.exp2(sf.double() - 127 - 10).repeat_interleave(32, 1)
    assert not (off > 2.0 ** -4 * x.double().abs() + least).any()


def test_nan_and_infinity_stay_where_they_are():
    x, u = normal((6, 128), BF, 7), normal((6, 128), BF, 8)
    clean = [t.clone() for t in (x, u)]
    x[1, 5], x[2, 40], x[3, 70], u[4, 100], u[5, 31] = NAN, INF, -INF, INF, NAN
    (q0, s0), (q, sf) = mxg.alloc_act_checkpoint(6, 128), mxg.alloc_act_checkpoint(6, 128)
    h0, h = torch.empty_like(x), torch.empty_like(x)
    for m in ((1, 5), (2, 40), (3, 70)):
        clean[0][m] = 0
    for m in ((4, 100), (5, 31)):
        clean[1][m] = 0
    mxg.mxg_gated_act(clean[0], h0, up=clean[1], q=q0, sf=s0)
    mxg.mxg_gated_act(x, h, up=u, q=q, sf=sf)
    spots = torch.zeros(6, 128, dtype=torch.bool, device=DEV)
    for m in ((1, 5), (2, 40), (3, 70), (4, 100), (5, 31)):
        spots[m] = True
    assert torch.equal(h[~spots], h0[~spots]) and not torch.isfinite(h[spots]).any()
    check_kept(q, sf, [x, u])
    assert torch.equal(sf, s0)
    dh, d = normal((6, 128), BF, 9), torch.empty(6, 256, dtype=BF, device=DEV)
    d0 = torch.empty_like(d)
    mxg.mxg_gated_act_backward(q0, s0, dh, d0[:, :128], dup=d0[:, 128:])
    mxg.mxg_gated_act_backward(q, sf, dh, d[:, :128], dup=d[:, 128:])
    twice = torch.cat([spots, spots], 1)
    assert torch.equal(d[~twice], d0[~twice])
    assert torch.isnan(d[:, :128][spots]).all()


def test_gradient_by_differences():
    """The slope at the kept values against central differences of the 64-bit activation."""
    for act in (SILU, GELU):
        x, u = normal((8, 64), HF, 10), normal((8, 64), HF, 11)
        h, (q, sf) = torch.empty_like(x), mxg.alloc_act_checkpoint(8, 64)
        mxg.mxg_gated_act(x, h, up=u, act=act, q=q, sf=sf)
        dh = torch.ones_like(x)
        dg, du = torch.empty_like(x), torch.empty_like(x)
        mxg.mxg_gated_act_backward(q, sf, dh, dg, dup=du, act=act)
        g, w = values(q[:, :64].contiguous(), sf[:, :2], 64), values(q[:, 64:].contiguous(), sf[:, 2:], 64)
        f = lambda t: t * torch.sigmoid(z_of(t, act))  # noqa: E731
        step = 1e-5
        slope = (f(g + step) - f(g - step)) / (2 * step) * w
        # 2^-11 of the value and its fp32 part, with room for the difference's own 1e-9
        assert not ((dg.double() - slope).abs() > 2.0 ** -11 * slope.abs() + 2.0 ** -18 * w.abs()
                    * (1 + g.abs()) + 1e-8).any()
        assert not ((du.double() - f(g)).abs() > 2.0 ** -11 * f(g).abs() + 2.0 ** -18 * g.abs() + 1e-8).any()


@pytest.mark.parametrize("sizes", [[0, 0], [5, 0, 9], [64, -3, 10], [200, 200], [129, 1 << 40]])
@pytest.mark.parametrize("cols", [64, 52])
def test_rows_behind_the_groups_stay(sizes, cols):
    rows = 200
    G = len(sizes)
    ws = torch.tensor(sizes + [0] * (G + 1), dtype=torch.int64, device=DEV)
    live = min(rows, sum(max(0, min(s, rows)) for s in sizes))
    x, u = normal((rows, cols), BF, 12), normal((rows, cols), BF, 13)
    x[live:], u[live:] = NAN, NAN
    h = torch.full_like(x, 7.0)
    q, sf = mxg.alloc_act_checkpoint(rows, cols)
    q.fill_(0x55), sf.fill_(0x55)
    mxg.mxg_gated_act(x, h, up=u, q=q, sf=sf, group_ws=ws, G=G)
    check_h(h[:live], x[:live], u[:live], SILU, BF)
    check_kept(q[:live], sf[:live], [x[:live], u[:live]])
    assert (h[live:] == 7.0).all() and (q[live:] == 0x55).all() and (sf[live:] == 0x55).all()
    dh, d = normal((rows, cols), BF, 14), torch.full((rows, 2 * cols), 7.0, dtype=BF, device=DEV)
    mxg.mxg_gated_act_backward(q, sf, dh, d[:, :cols], dup=d[:, cols:], h=h, group_ws=ws, G=G)
    check_backward(q[:live], sf[:live], dh[:live], d[:live, :cols], d[:live, cols:], h[:live], SILU, BF)
    assert (d[live:] == 7.0).all() and (h[live:] == 7.0).all()


@pytest.mark.parametrize("cols", [64, 37])
def test_in_place(cols):
    x, u = normal((50, cols), BF, 15), normal((50, cols), BF, 16)
    h, (q, sf) = torch.empty_like(x), mxg.alloc_act_checkpoint(50, cols)
    mxg.mxg_gated_act(x, h, up=u, q=q, sf=sf)
    for which in (0, 1):
        a, b = x.clone(), u.clone()
        q2, s2 = mxg.alloc_act_checkpoint(50, cols)
        mxg.mxg_gated_act(a, (a, b)[which], up=b, q=q2, sf=s2)
        assert torch.equal((a, b)[which], h) and torch.equal(q, q2) and torch.equal(sf, s2)
    dh, dg, du = normal((50, cols), BF, 17), torch.empty_like(x), torch.empty_like(x)
    mxg.mxg_gated_act_backward(q, sf, dh, dg, dup=du)
    for which in (0, 1):
        a, other = dh.clone(), torch.empty_like(x)
        mxg.mxg_gated_act_backward(q, sf, a, (a, other)[which], dup=(other, a)[which])
        assert torch.equal((a, other)[which], dg) and torch.equal((other, a)[which], du)


def test_past_32_bits_of_elements():
    rows, cols = (1 << 12) + 3, 1 << 18  # 2^30 values a matrix, 2^31 side by side
    w = torch.zeros(rows, 2 * cols, dtype=BF, device=DEV)
    w[-1], w[5, :64], w[1 << 11, cols:] = normal(2 * cols, BF, 18), 1.5, -2.0
    h = torch.full((rows, cols), NAN, dtype=BF, device=DEV)
    q, sf = mxg.alloc_act_checkpoint(rows, cols)
    mxg.mxg_gated_act(w[:, :cols], h, up=w[:, cols:], q=q, sf=sf)
    for r in (0, 5, 1 << 11, rows - 1):
        check_h(h[r:r + 1], w[r:r + 1, :cols], w[r:r + 1, cols:], SILU, BF)
        check_kept(q[r:r + 1], sf[r:r + 1], [w[r:r + 1, :cols], w[r:r + 1, cols:]])
    h.fill_(1.0)
    mxg.mxg_gated_act_backward(q, sf, h, w[:, :cols], dup=w[:, cols:])
    one = torch.ones(1, cols, dtype=BF, device=DEV)
    for r in (0, 5, 1 << 11, rows - 1):
        check_backward(q[r:r + 1], sf[r:r + 1], one, w[r:r + 1, :cols], w[r:r + 1, cols:], None, SILU, BF)


def test_same_bits_streams_and_graphs():
    x, u, dh = (normal((3000, 704), BF, 19 + i) for i in range(3))

    def both():
        h, (q, sf) = torch.empty_like(x), mxg.alloc_act_checkpoint(3000, 704)
        dg, du = torch.empty_like(x), torch.empty_like(x)
        mxg.mxg_gated_act(x, h, up=u, q=q, sf=sf)
        mxg.mxg_gated_act_backward(q, sf, dh, dg, dup=du)
        return h, q, sf, dg, du
    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both()
    graph.replay()
    torch.cuda.synchronize()
    for got in (both(), there, captured):
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_refusals():
    x, h = normal((4, 64), BF, 22), torch.empty(4, 64, dtype=BF, device=DEV)
    q, sf = mxg.alloc_act_checkpoint(4, 64)
    ws = torch.zeros(5, dtype=torch.int64, device=DEV)
    for call in (lambda: mxg.mxg_gated_act(x, h[:3]), lambda: mxg.mxg_gated_act(x, h.half()),
                 lambda: mxg.mxg_gated_act(x, h, up=x[:, :32]), lambda: mxg.mxg_gated_act(x, h, q=q),
                 lambda: mxg.mxg_gated_act(x, h, q=q, sf=sf), lambda: mxg.mxg_gated_act(x, h, up=x, q=q, sf=sf[:3]),
                 lambda: mxg.mxg_gated_act(x, h, group_ws=ws, G=3), lambda: mxg.mxg_gated_act(x.cpu(), h),
                 lambda: mxg.mxg_gated_act(x[:1].expand(4, 64), h),
                 lambda: mxg.mxg_gated_act_backward(q, sf, x, h),
                 lambda: mxg.mxg_gated_act_backward(q[:, :64], sf[:, :2], x, h)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mxg.mxg_gated_act(x, h, act=2), lambda: mxg.mxg_gated_act(x.float(), h.float()),
                 lambda: mxg.mxg_gated_act(x, h, group_ws=ws[:1])):
        with pytest.raises(mxg.MxgError) as err:
            call()
        assert err.value.code == 1
