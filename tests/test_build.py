"""The build's two parts: the library needs neither torch's headers nor calls.cpp (CPU; the compilers are
stand-ins that write empty files)."""
import os
import subprocess

import pytest

from nvfp4_paged_kv_02_gb300 import _build


class Compilers:
    def __init__(self):
        self.ran, self.broken = [], ()

    def __call__(self, cmd, **kw):
        what = next((s for s in _build.SOURCES + [_build.CALLS_SOURCE] if any(str(a).endswith(s) for a in cmd)), "link")
        tool = os.path.basename(cmd[0])
        self.ran.append((tool, what))
        if (tool, what) in self.broken:
            return subprocess.CompletedProcess(cmd, 1, "", "error: not today")
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", "")


@pytest.fixture()
def tools(monkeypatch, tmp_path):
    t = Compilers()
    monkeypatch.setattr(_build.subprocess, "run", t)
    monkeypatch.setattr(_build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(_build, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(_build, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "CALLS_PATH", str(tmp_path / "calls.so"))
    return t


def test_build_makes_both_once(tools):
    assert _build.build() == _build.LIB_PATH
    assert os.path.exists(_build.LIB_PATH) and os.path.exists(_build.CALLS_PATH)
    assert sorted(tools.ran) == sorted([("nvcc", s) for s in _build.SOURCES] + [("nvcc", "link"), ("g++", "link"),
                                                                                ("g++", _build.CALLS_SOURCE)])
    tools.ran.clear()
    assert _build.build() == _build.LIB_PATH and _build.build_calls() == _build.CALLS_PATH and not tools.ran


def test_library_without_the_calls(tools):
    tools.broken = (("g++", _build.CALLS_SOURCE),)
    assert _build.build_library() == _build.LIB_PATH and os.path.exists(_build.LIB_PATH)
    assert all(tool == "nvcc" for tool, _ in tools.ran)


def test_a_broken_calls_module_is_an_error_and_leaves_the_library(tools):
    tools.broken = (("g++", _build.CALLS_SOURCE),)
    with pytest.raises(RuntimeError, match="calls.cpp"):
        _build.build()
    assert os.path.exists(_build.LIB_PATH) and not os.path.exists(_build.CALLS_PATH)
    tools.ran.clear()
    assert _build.build_library() == _build.LIB_PATH and not tools.ran
    tools.broken = ()
    assert _build.build() == _build.LIB_PATH and os.path.exists(_build.CALLS_PATH)
    assert tools.ran == [("g++", _build.CALLS_SOURCE), ("g++", "link")]


def test_a_broken_kernel_is_an_error(tools):
    tools.broken = (("nvcc", "pages.cu"),)
    with pytest.raises(RuntimeError, match="pages.cu"):
        _build.build()
    assert not os.path.exists(_build.LIB_PATH)
