"""Routing in every layout of a token over lanes, both ways of choosing and all types, against 64 bits;
logits that are no numbers, infinite or extreme; sums over millions of tokens.

Bounds, of a token on its own.  With R its span (softmax: the range of its logits above -infinity, sigmoid:
their largest magnitude; 90 at most, beyond which the exponential is below 2^-126 and counts as 0), an
exponential is off by 2 + 1.2 R units of 2^-23 (ex2.approx: 2; the product with log2 e: 1.2 R) and the
subtraction before it by R 2^-24: 2^-23 (2 + 1.7 R).  A weight or share is a quotient of such a value and a
sum of such values: twice that; 37 roundings of the sum (32 columns a lane, five doublings) and 19 of
1 + e (twice), its reciprocal at 2^-23 (four times), its second exponential, the quotient and the scale:
56 * 2^-24.  What is flushed is at most 2^-126 of a sum that is 1/2 or more: 2 * 2^-126 times the scale,
4 with its own rounding.  The loss adds shares of one sign: those of a team's tokens one after the other --
1216 teams at least where there are many CTAs -- and fewer than 256 more: (tokens / 1216 + 256) 2^-24.  A
slope has six roundings.
"""
import random

import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu, status_tensor
from moe_grouped_block_gb300 import mxg
from test_gpu_r_route import check_gradient, draw, route, rows_of
from test_route_layouts import SHAPES, SIZES_BY_RANK, forward, with_candidates

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
SOFT, SIG = mxg.MXG_SCORE_SOFTMAX, mxg.MXG_SCORE_SIGMOID
INF, NAN = float("inf"), float("nan")
TINY = 2.0 ** -126
KINDS = [(SOFT, True), (SOFT, False), (SIG, True), (SIG, False)]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def best(x, k):
    """The k best of each row and their values: NaN above infinity, the lower column first."""
    nan = torch.isnan(x)
    v, at = torch.sort(torch.where(nan, INF, x) + 0.0, dim=1, descending=True, stable=True)
    _, again = torch.sort(nan.gather(1, at).to(torch.int8), dim=1, descending=True, stable=True)
    return at.gather(1, again)[:, :k], v.gather(1, again)[:, :k]


def strict(logits, k, mask=None, align=1, score=SOFT, normalize=True, scale=1.0, balance=0.0):
    """Every output of mxg_route against 64 bits; NaN only where the formula has it."""
    T, E = logits.shape
    st = status_tensor()
    got = route(logits, k, mask, align=align, last_dim=3, status=st, score=score, normalize=normalize,
                scale=scale, balance=balance)
    x = logits.double().cpu()
    live = ((x > -INF) | torch.isnan(x)).any(1)
    if mask is not None:
        live &= mask.cpu().bool()
    at, value = best(x, k)
    expert = torch.where((value > -INF) & live[:, None], at, -1)
    assert torch.equal(got["expert"].cpu().long(), expert)
    counts, row, ws = rows_of(expert.numpy(), E, align, T * k + E * (align - 1), 3)
    assert np.array_equal(got["counts"].cpu().numpy(), counts) and int(st) == 0
    assert np.array_equal(got["row_of"].cpu().numpy(), row)
    assert np.array_equal(got["group_ws"].cpu().numpy(), ws)

    s = torch.softmax(x, 1) if score == SOFT else torch.sigmoid(x)
    p = s if score == SOFT else torch.softmax(torch.nn.functional.logsigmoid(x), 1)
    fine = x.abs() < INF
    if score == SOFT:
        span = x.where(fine, torch.tensor(-INF)).amax(1) - x.where(fine, torch.tensor(INF)).amin(1)
    else:
        span = x.where(fine, torch.zeros(())).abs().amax(1)
    span = span.clamp(0.0, 90.0)
    rel = 2 * 2.0 ** -23 * (2 + 1.7 * span) + 56 * 2.0 ** -24

    w = (p if normalize else s).gather(1, expert.clamp(min=0))
    none = expert < 0
    w[none] = 0
    if normalize:
        w = w / w.sum(1, keepdim=True)
    w = scale * w
    w[none] = 0
    mine = got["weight"].cpu().double()
    assert (mine[none] == 0).all()
    assert torch.equal(torch.isnan(mine), torch.isnan(w))
    ok = ~torch.isnan(w)
    assert ((mine - w).abs() <= rel[:, None] * w.abs() + 4 * TINY * abs(scale))[ok].all()

    n, total = int(live.sum()), int(counts.sum())
    slope = balance * E * torch.from_numpy(counts).double() / max(1, total) / max(1, n)
    mine = got["slope"].cpu().double()
    assert ((mine - slope).abs() <= 6 * 2.0 ** -24 * slope.abs()).all()
    each = (p * slope).sum(1)[live]
    want = float(each.sum())
    loss = float(got["loss"])
    if torch.isnan(each).any():
        assert loss != loss
    else:
        bound = float((each.abs() * rel[live]).sum()) + (T / 1216 + 256 + 8) * 2.0 ** -24 * abs(want)
        assert abs(loss - want) <= bound + TINY * T * E
    return got, expert


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("score,normalize", KINDS)
def test_every_layout(T, E, k, dtype, score, normalize):
    g = torch.Generator().manual_seed(T)
    mask = (torch.rand(T, generator=g) < 0.9).to(torch.uint8).to(DEV) if T % 2 == 0 else None
    strict(draw(T, E, dtype, T + E), k, mask, 16 if E % 8 == 0 else 1, score, normalize, 2.5, 0.3)


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("score,normalize", KINDS)
def test_every_layout_of_the_gradient(T, E, k, dtype, score, normalize):
    g = torch.Generator().manual_seed(T)
    mask = (torch.rand(T, generator=g) < 0.9).to(torch.uint8).to(DEV) if T % 2 == 0 else None
    check_gradient(draw(T, E, dtype, T + E), k, mask, score=score, normalize=normalize, scale=2.5,
                   balance=30.0)


# ------------------------------------------------------------------ the choice
@pytest.mark.parametrize("E,k", SIZES_BY_RANK)
@pytest.mark.parametrize("dtype", [F32, BF, HF])
def test_as_many_candidates_as_are_ranked_and_more(E, k, dtype):
    """Rows of 26 to 36 candidates (31 are ranked), alone in a warp and beside others."""
    T = 3000
    assert forward(T, E, k) == forward(1 << 20, E, k)
    rng = random.Random(E)
    most = 36 if E > 64 else 28
    rows = torch.tensor([with_candidates(E, k, n, rng) for n in range(most - 10, most + 1) for _ in range(4)])
    x = draw(T, E, F32, 21).cpu()
    x[:1000] = rows[torch.randint(len(rows), (1000,), generator=torch.Generator().manual_seed(1))]
    x[1000:2000:7] = rows[torch.randint(len(rows), (143,), generator=torch.Generator().manual_seed(2))]
    strict(x.to(dtype).to(DEV), k, balance=0.1)


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF, HF])
def test_rising_and_falling_rows(T, E, k, dtype):
    """The best side by side, so that few parts hold them; of 16-bit types many are alike."""
    x = torch.arange(E).float().div(8).sub(2)[None].repeat(T, 1)
    x[1::3] = x[1::3].flip(1)
    x[2::3, ::2] *= -1
    strict(x.to(dtype).to(DEV), k, balance=0.5)


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("score,normalize", KINDS)
def test_minus_infinity(T, E, k, dtype, score, normalize):
    """Less than k logits to choose from, and none."""
    g = torch.Generator().manual_seed(E)
    x = draw(T, E, dtype, 22).cpu()
    x[torch.rand(T, E, generator=g) < 0.5] = -INF
    few = torch.rand(T, generator=g) < 0.3
    x[few] = torch.where(torch.rand(T, E, generator=g) < 1.5 / E, x, -INF)[few]
    low = torch.finfo(dtype).min
    if T > 3:
        x[1], x[2, 1:], x[3, ::2] = low, low, low
    x[T // 2] = -INF
    _, expert = strict(x.to(DEV), k, None, 4, score, normalize, 1.5, 0.5)
    assert (expert[T // 2] == -1).all()


@pytest.mark.parametrize("T,E,k", [s for s in SHAPES if s[0] > 4])
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("score,normalize", KINDS)
def test_nan_and_infinity(T, E, k, dtype, score, normalize):
    """Several of them in a row, of either sign; then in masked tokens alone."""
    g = torch.Generator().manual_seed(E + 1)
    x = draw(T, E, dtype, 23).cpu()
    hit = torch.rand(T, generator=g) < 0.2
    hit[0] = True
    for v in (NAN, -NAN, INF, -INF, -0.0, torch.finfo(dtype).max, torch.finfo(dtype).min):
        put = hit[:, None] & (torch.rand(T, E, generator=g) < 0.1)
        x[put] = v
    x[0, E - 1] = NAN
    if dtype is not F32:  # every bit pattern of NaN is one
        bits = x.view(torch.int16)
        bits[0, 0] = -1
        bits[4, E // 2] = torch.tensor(NAN, dtype=dtype).view(torch.int16).item() | 1
    strict(x.to(DEV), k, None, 1, score, normalize, 1.0, 0.5)
    got, _ = strict(x.to(DEV), k, (~hit).to(DEV), 1, score, normalize, 1.0, 0.5)
    if dtype is F32:  # (the patterns above lie in rows 0 and 4)
        assert torch.isfinite(got["loss"]).all() and torch.isfinite(got["weight"]).all()


# ------------------------------------------------------------------ many tokens
def test_many_choices_a_chunk():
    """More than 65536 of them, and 67 tokens' shares one after the other."""
    T, E, k = 5_200_000, 8, 2
    assert T * k > 152 * 65536
    x = torch.randn(T, E, generator=torch.Generator(device=DEV).manual_seed(24), device=DEV).to(BF)
    got = route(x, k, balance=0.1, align=128)
    x64 = x.double()
    at = torch.sort(x64, dim=1, descending=True, stable=True).indices[:, :k].contiguous()
    assert torch.equal(got["expert"].long(), at)
    counts = torch.bincount(at.view(-1), minlength=E)
    assert torch.equal(got["counts"].long(), counts)
    sizes = (counts + 127) // 128 * 128
    start = sizes.cumsum(0) - sizes
    for e in range(E):
        mine = got["row_of"].view(-1)[at.view(-1) == e].long()
        assert torch.equal(mine, start[e] + torch.arange(len(mine), device=DEV))
    p = torch.softmax(x64, 1)
    w = p.gather(1, at)
    w = w / w.sum(1, keepdim=True)
    span = x64.amax(1) - x64.amin(1)
    rel = 2 * 2.0 ** -23 * (2 + 1.7 * span) + 56 * 2.0 ** -24
    assert ((got["weight"].double() - w).abs() <= rel[:, None] * w).all()
    slope = 0.1 * E * counts.double() / (counts.sum() * T)
    each = (p * slope).sum(1)
    bound = (each * rel).sum() + (T / 1216 + 264) * 2.0 ** -24 * each.sum()
    assert float((got["loss"].double() - each.sum()).abs()) <= float(bound)


def test_loss_and_weights_past_32_bits_of_logits():
    T, E, k = (1 << 21) + 77, 1024, 3
    x = torch.empty(T, E, dtype=BF, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(25)
    for part in x.split(1 << 19):
        part.normal_(generator=gen)
    got = route(x, k, balance=0.1, plan=False)
    counts, sums = torch.zeros(E, dtype=torch.long, device=DEV), 0.0
    top = 0.0
    for at in range(0, T, 1 << 16):
        rows = slice(at, min(T, at + (1 << 16)))
        x64 = x[rows].double()
        v, e = torch.sort(x64, dim=1, descending=True, stable=True)
        assert torch.equal(got["expert"][rows].long(), e[:, :k])
        counts += torch.bincount(e[:, :k].reshape(-1), minlength=E)
        p = torch.softmax(x64, 1)
        w = p.gather(1, e[:, :k])
        w = w / w.sum(1, keepdim=True)
        rel = 2 * 2.0 ** -23 * (2 + 1.7 * (v[:, 0] - v[:, -1])) + 56 * 2.0 ** -24
        assert ((got["weight"][rows].double() - w).abs() <= rel[:, None] * w).all()
        sums, top = sums + p.sum(0), max(top, float(rel.max()))
    assert torch.equal(got["counts"].long(), counts)
    want = float((0.1 * E * counts.double() / (counts.sum() * T) * sums).sum())
    assert abs(float(got["loss"]) - want) <= (top + (T / 1216 + 264) * 2.0 ** -24) * want
