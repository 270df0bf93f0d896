"""Grouped products on 16-bit operands: long contractions and large groups.

Small integers are exact in every step -- products, fp32 sums below 2^24 -- so an
fp32 output equals the exact sum, and a 16-bit one the exact sum rounded once.
"""
import pytest
import torch

from gpu_util import DEV, require_gpu
from moe_grouped_block_gb300 import mxg
from test_gpu_j_grouped_gemm_16bit import DGRAD, FPROP, MODES, WGRAD, group_ws

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def draw(mode, sizes, N, K, dtype, most, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    new = lambda *s: torch.randint(-most, most + 1, s, generator=g, device=DEV).to(dtype)  # noqa: E731
    M = sum(sizes)
    return new(M, K if mode == FPROP else N), new(M, K) if mode == WGRAD else new(len(sizes), N, K)


def exact(mode, a, b, sizes):
    parts, at = [], 0
    for g, m in enumerate(sizes):
        r = slice(at, at + m)
        at += m
        if mode == WGRAD:
            parts.append(a[r].double().t() @ b[r].double())
        else:
            parts.append(a[r].double() @ (b[g].double().t() if mode == FPROP else b[g].double()))
    return torch.stack(parts) if mode == WGRAD else torch.cat(parts)


def run(mode, a, b, sizes, N, K, out):
    G, M = len(sizes), sum(sizes)
    C = torch.full({FPROP: (M, N), DGRAD: (M, K), WGRAD: (G, N, K)}[mode], 7.0, dtype=out, device=DEV)
    mxg.mxg_grouped_gemm_16bit(mode, a, b, group_ws(sizes, M), G, M, N, K, C=C)
    return C


LONG = [  # mode, sizes, N, K: more units than clusters, or too many to share a contraction
    ("fprop", [300, 0, 129], 8200, 4104), ("fprop", [1, 31], 16392, 8200),
    ("dgrad", [300, 0, 129], 4104, 8200), ("dgrad", [16], 14336, 20480),
    ("wgrad", [4100, 0, 3999, 5001], 1104, 1208), ("wgrad", [8209], 2056, 2568),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("case", LONG, ids=lambda c: "%s_%d_%d_%d" % (c[0], len(c[1]), c[2], c[3]))
def test_integers_in_long_contractions(case, dtype):
    mode, sizes, N, K = case
    mode = MODES[mode]
    a, b = draw(mode, sizes, N, K, dtype, 3, 41)  # sums below 9 * 14336
    ref = exact(mode, a, b, sizes)
    for out in (F32, dtype):
        C = run(mode, a, b, sizes, N, K, out)
        assert torch.equal(C, ref.to(out)), out
        assert torch.equal(C, run(mode, a, b, sizes, N, K, out))


@pytest.mark.parametrize("mode,sizes,N,K", [
    # a group's rows times the contraction pass 32 MB: its units are walked in blocks of columns
    ("fprop", [4500, 70], 8200, 4096), ("fprop", [2300], 9000, 8192), ("dgrad", [4500, 9], 4096, 8456),
    # a contraction so long that a block is one or two units wide
    ("fprop", [300], 1400, 60000), ("dgrad", [200, 400], 50008, 1544)])
def test_groups_beyond_the_l2_budget(mode, sizes, N, K):
    mode = MODES[mode]
    a, b = draw(mode, sizes, N, K, BF, 3, 42)
    ref = exact(mode, a, b, sizes)
    for out in (F32, BF):
        assert torch.equal(run(mode, a, b, sizes, N, K, out), ref.to(out))


@pytest.mark.parametrize("mode", list(MODES))
def test_16bit_outputs_are_rounded_once(mode):
    """Against the exact sum: one rounding to bf16, 2^-8 |ref| at most, and what the fp32
    sum lost by truncation, 2^-23 of the sum of magnitudes in each step of 16 products."""
    mode, sizes, N, K = MODES[mode], [700, 0, 900], 1032, 2056
    g = torch.Generator(device=DEV).manual_seed(43)
    new = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)  # noqa: E731
    a, b = new(1600, K if mode == FPROP else N), new(1600, K) if mode == WGRAD else new(3, N, K)
    ref, mag = exact(mode, a, b, sizes), exact(mode, a.abs(), b.abs(), sizes)
    steps = {FPROP: K, DGRAD: N, WGRAD: 900}[mode] / 16 + 2
    C = run(mode, a, b, sizes, N, K, BF)
    assert not ((C.double() - ref).abs() > 2.0 ** -8 * ref.abs() + steps * 2.0 ** -23 * mag).any()
    assert torch.equal(C, run(mode, a, b, sizes, N, K, BF))
