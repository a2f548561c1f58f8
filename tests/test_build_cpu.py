"""The build of the library and of the Python module beside it: with and without torch, and when torch changes (CPU)."""
import os

import pytest

import __graft_entry__
from differentiable_gaussian_splatting_gs_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def _runs(monkeypatch):
    """The commands that a build would run; the module's output is a file of the test's own."""
    ran = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **_):
        ran.append(cmd)
        if "-o" in cmd:
            with open(cmd[cmd.index("-o") + 1], "a"):
                pass
        return Done()

    monkeypatch.setattr(build.subprocess, "run", run)
    return ran


def test_what_is_built_is_not_built_again(monkeypatch):
    ran = _runs(monkeypatch)
    assert build.build_library() == build.LIB and ran == []


def test_the_library_is_built_without_torch(monkeypatch):
    ran = _runs(monkeypatch)
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    monkeypatch.setattr(build, "_stale", lambda target, deps: target == build.LIB)
    monkeypatch.setattr(build.os, "replace", lambda a, b: os.remove(a))
    assert build.build_library() == build.LIB
    assert len(ran) == 1 and "-shared" in ran[0] and "-cudart" in ran[0]  # linked; no module


def test_another_torch_makes_the_module_stale(monkeypatch):
    nvcc = build._nvcc()
    assert not build._bind_jobs(nvcc, False).stale
    where, version = build._torch()
    assert "__version__" in version
    monkeypatch.setattr(build, "_torch", lambda: (where, version + "\n__version__ = 'another'"))
    assert build._bind_jobs(nvcc, False).stale
    monkeypatch.setattr(build, "_torch", lambda: (where + "/elsewhere", version))
    assert build._bind_jobs(nvcc, False).stale
