"""A header that changed rebuilds every object: the build is run with a compiler
that only records what it is asked to do."""
import glob
import os
import types

import pytest

from moe_grouped_block_gb300 import build as mxg_build

HEADERS = sorted(p for p in glob.glob(os.path.join(mxg_build.CSRC, "*"))
                 if os.path.isfile(p) and not p.endswith(".cu")) + [mxg_build.HEADER]


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """Builds with fake times, `newer` being newer than all objects; the sources compiled."""
    def run(newer):
        commands = []
        monkeypatch.setattr(mxg_build, "BUILD_DIR", str(tmp_path))
        monkeypatch.setattr(mxg_build, "_nvcc", lambda: "/bin/nvcc")
        monkeypatch.setattr(mxg_build, "LIB", str(tmp_path / "lib.so"))
        for p in glob.glob(os.path.join(mxg_build.CSRC, "*.cu")):
            (tmp_path / (os.path.basename(p)[:-3] + ".o")).touch()
        (tmp_path / "lib.so").touch()
        ok = types.SimpleNamespace(returncode=0, stdout="", stderr="")
        monkeypatch.setattr(mxg_build.subprocess, "run", lambda c, **kw: commands.append(c) or ok)
        monkeypatch.setattr(mxg_build.os, "replace", lambda a, b: None)
        made = lambda p: str(p).startswith(str(tmp_path))  # noqa: E731
        monkeypatch.setattr(mxg_build.os.path, "getmtime",
                            lambda p: 3.0 if p == newer else 2.0 if made(p) else 1.0)
        mxg_build.build()
        monkeypatch.undo()
        return sorted(c[c.index("-c") + 1] for c in commands if "-c" in c)
    return run


@pytest.mark.parametrize("header", HEADERS, ids=os.path.basename)
def test_a_newer_header_rebuilds_what_includes_it(compiled, header):
    name = '#include "%s"' % os.path.basename(header)
    direct = [p for p in glob.glob(os.path.join(mxg_build.CSRC, "*.cu")) if name in open(p).read()]
    got = compiled(header)
    assert got and set(direct) <= set(got)


def test_nothing_newer_rebuilds_nothing(compiled):
    assert compiled(None) == []
