"""Size queries of the 16-bit operators over their whole range and past it, in a
process of their own: a query takes any argument."""
import subprocess
import sys

import pytest

from moe_grouped_block_gb300 import build as mxg_build
from moe_grouped_block_gb300 import mxg

MOST = 16384  # columns of a norm's row


@pytest.fixture(scope="module", autouse=True)
def lib():
    mxg_build.build()
    return mxg.load()


def query(*sizes):
    code = ("import ctypes, sys\n"
            "f = ctypes.CDLL(%r).mxg_block_norm_workspace_bytes\n"
            "f.restype, f.argtypes = ctypes.c_size_t, [ctypes.c_int64] * 2\n"
            "print(*[f(*map(int, line.split())) for line in sys.stdin])" % mxg.LIB_PATH)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       input="".join("%d %d\n" % s for s in sizes))
    assert r.returncode == 0, "the process ended with %d" % r.returncode
    return [int(v) for v in r.stdout.split()]


@pytest.mark.parametrize("rows", [0, 1, 4096, 1 << 40])
@pytest.mark.parametrize("cols", [MOST + 1, MOST + 16, 20000, 1 << 20, (1 << 31) - 1, 1 << 40, (1 << 63) - 1])
def test_norm_workspace_of_rows_too_wide(rows, cols):
    assert query((rows, cols)) == [0]


def test_norm_workspace_of_no_size():
    assert query((-1, 64), (4, 0), (4, -5), (0, 64)) == [0, 0, 0, 0]


def test_norm_workspace_of_every_width():
    """One partial row of two fp32 sums a column for each row, up to some number of them
    that does not depend on the rows."""
    widths = range(1, MOST + 1)
    got = query(*[(1, c) for c in widths], *[(1 << 20, c) for c in widths])
    assert got[:MOST] == [8 * c for c in widths]
    assert all(b % (8 * c) == 0 and 8 * c <= b <= 8 * c * 160 * 8 for c, b in zip(widths, got[MOST:]))
