"""The build without what only the Python module needs (nothing is compiled: the steps are recorded)."""
import importlib.util
import os
import subprocess

import pytest

from lora_serving_amd import build


@pytest.fixture
def steps(monkeypatch, tmp_path):
    """Commands that a build runs, which write empty outputs into tmp_path."""
    ran = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done

    for name in ("BUILD", "LIB", "MARSHAL"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(subprocess, "run", run)
    return ran


def without_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_library_without_torch(steps, monkeypatch):
    """The C library does not need torch: without it there is no binding to make."""
    without_torch(monkeypatch)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.MARSHAL)
    assert len(steps) == len(build.sources()) + 1


def test_stale_module_does_not_stay(steps, monkeypatch):
    """A module of an earlier build, of another library, is not left beside the new one."""
    open(build.MARSHAL, "w").close()
    without_torch(monkeypatch)
    build.build()
    assert not os.path.exists(build.MARSHAL)


def test_one_compiler(steps):
    """hipcc compiles the module too: no second compiler is needed."""
    assert build.build() == build.LIB and os.path.exists(build.MARSHAL)
    assert {c[0] for c in steps} == {build.HIPCC}
    assert len(steps) == len(build.sources()) + 2
