"""The status word of the routing entry points, without a GPU: it is written by an atomic, which
takes a word on 4 bytes."""
import ctypes

import pytest
import torch

from moe_grouped_block_gb300 import build as mxg_build
from moe_grouped_block_gb300 import mxg

FAKE = 1 << 20  # aligned and non-null; never dereferenced
OK_BUT_NO_DEVICE, ALIGNMENT = 3, 2

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake-pointer validation tests run without a GPU")


@pytest.fixture(scope="module")
def lib():
    mxg_build.build()
    return mxg.load()


@pytest.mark.parametrize("off,code", [(0, OK_BUT_NO_DEVICE), (4, OK_BUT_NO_DEVICE), (1, ALIGNMENT),
                                      (2, ALIGNMENT), (3, ALIGNMENT)])
def test_status_word(lib, off, code):
    need = mxg.mxg_route_workspace_bytes(100, 64, 4)
    d = mxg.Route(dtype=0, tokens=100, experts=64, k=4, logits=FAKE, scale=1.0, expert=FAKE, weight=FAKE,
                  counts=FAKE, align=1, last_dim=1)
    assert lib.mxg_route(ctypes.byref(d), FAKE, need, FAKE + off, None) == code
    assert lib.mxg_route_rows(FAKE, 100, 64, 4, 1, 400, 1, FAKE, None, None, FAKE, need, FAKE + off,
                              None) == code
