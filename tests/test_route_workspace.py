"""The workspace of the routing calls, without a GPU: what serves a batch serves the smaller ones, so
that a program can allocate for the largest."""
import random

import pytest

from moe_grouped_block_gb300 import build as mxg_build
from moe_grouped_block_gb300 import mxg


@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (16, 4), (32, 8), (64, 8), (100, 12), (128, 8), (256, 8),
                                 (256, 32), (384, 8), (512, 8), (1000, 8), (1024, 32)])
def test_it_grows_with_the_tokens(E, k):
    mxg_build.build()
    size, rng = mxg.load().mxg_route_workspace_bytes, random.Random(E)
    tokens = list(range(4000)) + sorted(rng.randint(4000, 400000) for _ in range(4000))
    sizes = [size(T, E, k) for T in tokens]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert sizes[-1] <= size((1 << 31) // k - 128, E, k) <= 152 * (2 * (E + 3) + 1) * 4 + 16
