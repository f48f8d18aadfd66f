"""What the in-tree build needs: the library nvcc alone, the marshalling module torch and g++ besides."""

import importlib.metadata
import os
import subprocess
import types

import pytest

from kernelized_causal_self_gb300 import build as labuild


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """Compilers that only write their output files, in a folder of the test's own. `tools.fails`: a
    word of the commands that fail."""
    monkeypatch.setattr(labuild, "BUILD", str(tmp_path))
    monkeypatch.setattr(labuild, "LIB", str(tmp_path / "liblagb300.so"))
    monkeypatch.setattr(labuild, "MARSHAL", str(tmp_path / "la_marshal.so"))
    monkeypatch.setattr(labuild, "_nvcc", lambda: "/opt/cuda/bin/nvcc")
    t = types.SimpleNamespace(ran=[], fails=None, torch="9.9")

    def run(cmd, **kw):
        source = next((c for c in cmd if c.endswith((".cu", ".cpp"))), "link")
        t.ran.append(os.path.basename(source))
        rc = int(t.fails is not None and any(t.fails in c for c in cmd))
        if rc == 0:
            with open(cmd[cmd.index("-o") + 1], "w"):
                pass
        return types.SimpleNamespace(returncode=rc, stdout="", stderr="no such header" if rc else "")

    def version(name):
        assert name == "torch"
        if t.torch is None:
            raise importlib.metadata.PackageNotFoundError(name)
        return t.torch
    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(importlib.metadata, "version", version)
    return t


def test_everything_is_built_once(tools):
    assert not labuild.up_to_date() and labuild.build() == labuild.LIB
    sources = [os.path.basename(s) for s in labuild._sources()]
    assert sorted(tools.ran) == sorted([*sources, "link", "la_marshal.cpp"])
    assert labuild.up_to_date() and os.path.exists(labuild.MARSHAL)
    tools.ran.clear()
    labuild.build()
    assert not tools.ran
    labuild.build(force=True)
    assert len(tools.ran) == len(sources) + 2


def test_the_library_is_built_where_the_marshalling_does_not_compile(tools):
    tools.fails = "la_marshal"
    with pytest.raises(RuntimeError, match="library is built.*la_marshal.cpp.*\\n.*no such header"):
        labuild.build()
    assert os.path.exists(labuild.LIB) and not os.path.exists(labuild.MARSHAL) and not labuild.up_to_date()
    tools.fails = None
    tools.ran.clear()
    labuild.build()
    assert tools.ran == ["la_marshal.cpp"] and labuild.up_to_date()


def test_the_library_takes_nvcc_alone(tools):
    tools.torch = None
    assert labuild.build() == labuild.LIB and labuild.up_to_date()
    assert "la_marshal.cpp" not in tools.ran and not os.path.exists(labuild.MARSHAL)
    tools.ran.clear()
    labuild.build(force=True)
    assert "la_marshal.cpp" not in tools.ran and tools.ran


def test_another_torch_has_the_marshalling_built_again(tools):
    labuild.build()
    tools.ran.clear()
    tools.torch = "9.10"
    assert not labuild.up_to_date()
    labuild.build()
    assert tools.ran == ["la_marshal.cpp"] and labuild.up_to_date()


def test_a_library_that_does_not_compile_is_none(tools):
    tools.fails = "la_api.cu"
    with pytest.raises(RuntimeError, match="compilation failed"):
        labuild.build()
    assert not os.path.exists(labuild.LIB)
