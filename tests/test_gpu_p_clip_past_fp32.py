"""Clipping where the norm passes fp32's range, against 64 bits.

Bounds.  The norm of a sum of squares in fp64 carries 2^-18 (test_gpu_l_grad_clip.py),
the factor the same, and a clipped value one rounding to its type: 2^-18 + u, plus
four times half of the smallest subnormal where the result or a factor is one.
"""
import math

import pytest
import torch

from gpu_util import DEV, require_gpu
from test_gpu_l_grad_clip import BF, F32, HF, TINY, U, clip, draw, exact_norm

pytestmark = pytest.mark.gpu
REL = 2.0 ** -18
INF = float("inf")


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def check(grads, out, limit):
    """float64 holds every norm and factor here."""
    factor = min(1.0, limit / (exact_norm(grads) + 1e-6))
    for g, o in zip(grads, out):
        ref = g.double() * factor
        tol = (REL + U[o.dtype]) * ref.abs() + 4 * TINY[o.dtype]
        assert torch.isfinite(o).all() and not ((o.double() - ref).abs() > tol).any()


def huge(dtype, seed=1, n=5000):
    g = draw([n, 77], F32, seed)
    return [(v.double().clamp(-3, 3) * 1e38).to(dtype) for v in g]


@pytest.mark.parametrize("src,dst", [(F32, F32), (BF, BF), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("limit", [1.0, 1e30, 3e38, 1e-3, 1e-20, 1e-37, 1e-44, 0.0])
def test_norm_past_fp32(src, dst, limit):
    """Finite gradients whose norm is not an fp32 number."""
    grads = huge(src)
    assert exact_norm(grads) > 2.0 ** 128
    out = [torch.full((len(g),), 7.0, dtype=dst, device=DEV) for g in grads]
    assert clip(grads, limit, out) == INF  # the norm itself is returned in fp32
    check(grads, out, limit)


@pytest.mark.parametrize("src,dst", [(F32, F32), (BF, BF), (F32, HF), (HF, F32)])
@pytest.mark.parametrize("norm,limit", [(1e38, 1e-1), (3e38, 1e-6), (1e30, 1e-20), (1e20, 1e-30),
                                        (1.0, 1e-40), (1e4, 1e-36)])
def test_factors_below_the_normal_range(norm, limit, src, dst):
    """A factor that is an fp32 subnormal, with results that are not."""
    if src == HF and norm > 1e4:
        pytest.skip("past fp16")
    g = draw([3000, 5], F32, 2)
    each = norm / math.sqrt(3005)
    grads = [(v.double().clamp(-3, 3) * each).to(src) for v in g]
    out = [torch.full((len(v),), 7.0, dtype=dst, device=DEV) for v in grads]
    clip(grads, limit, out)
    check(grads, out, limit)


@pytest.mark.parametrize("types", [(F32, F32), (BF, BF), (BF, F32)])
def test_infinite_limit_clips_nothing(types):
    src, dst = types
    for grads in (huge(src, 3), draw([5000, 3], src, 4)):
        want = [g.to(dst) for g in grads]
        out = [torch.full((len(g),), 7.0, dtype=dst, device=DEV) for g in grads]
        clip(grads, INF, out)
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_infinite_limit_and_infinite_gradient():
    """With nothing to clip the factor is 1: an infinity stays what it is.  A NaN still
    makes every output NaN."""
    a, b = draw([9000, 50], F32, 5)
    b[7] = -INF
    x, y = a.clone(), b.clone()
    assert clip([x, y], INF) == INF
    assert torch.equal(x, a) and torch.equal(y, b)
    b[7] = float("nan")
    x, y = a.clone(), b.clone()
    assert math.isnan(clip([x, y], INF))
    assert torch.isnan(x).all() and torch.isnan(y).all()


def test_mixed_types_past_fp32():
    grads = huge(F32, 6) + draw([1000], HF, 7) + huge(BF, 8, 300)
    kept = [g.clone() for g in grads]
    clip(grads, 2.0)
    check(kept, grads, 2.0)
