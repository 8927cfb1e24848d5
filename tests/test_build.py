"""What the build makes of which inputs, with the compilers replaced by a record of their calls (no GPU)."""
import os
import subprocess
import sys
import types

import pytest

from paged_kv_attention_24_gb300 import build


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """Compilers that write an empty file where -o says; .fail names one that reports an error."""
    calls = types.SimpleNamespace(fail=None, ran=[])

    def fake(cmd, **kw):
        tool = os.path.basename(cmd[0])
        calls.ran.append(tool)
        if tool == calls.fail:
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    for name in ("LIB", "BINDING"):
        if hasattr(build, name):
            monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "nvcc", lambda: "/opt/cuda/bin/nvcc")
    monkeypatch.setattr(build.subprocess, "run", fake)
    return calls


def bindings(tmp_path):
    return sorted(p.name for p in tmp_path.glob("_msgl_binding*.so"))


def test_library_and_binding(tools, tmp_path):
    assert build.build() == str(tmp_path / "libmsgl_attn.so")
    assert os.path.exists(tmp_path / "libmsgl_attn.so") and len(bindings(tmp_path)) == 1
    assert build.up_to_date()
    tools.ran.clear()
    build.build()
    assert tools.ran == []


def test_the_c_library_needs_no_torch(tools, tmp_path, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)   # an import of torch raises ImportError
    build.build()
    assert os.path.exists(tmp_path / "libmsgl_attn.so") and bindings(tmp_path) == []
    assert "g++" not in tools.ran
    assert build.up_to_date()


def test_the_c_library_stands_when_the_binding_does_not_compile(tools, tmp_path):
    tools.fail = "g++"
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()
    assert os.path.exists(tmp_path / "libmsgl_attn.so") and bindings(tmp_path) == []
    assert not build.up_to_date()


def test_another_torch_gets_a_binding_of_its_own(tools, tmp_path, monkeypatch):
    import torch
    build.build()
    before = bindings(tmp_path)
    monkeypatch.setattr(torch, "__version__", "99.1+cu999")
    assert not build.up_to_date()
    tools.ran.clear()
    build.build()
    assert set(tools.ran) == {"g++"}                  # the library does not depend on it
    assert len(bindings(tmp_path)) == 2 and set(before) < set(bindings(tmp_path))
    assert build.up_to_date()


def test_the_loaded_binding_is_the_one_of_this_torch(monkeypatch):
    import torch

    from paged_kv_attention_24_gb300 import ops
    build.build()
    assert ops._binding().__file__ == build.binding_path()
    monkeypatch.setattr(torch, "__version__", "99.1+cu999")
    with pytest.raises(RuntimeError, match="not built"):
        ops._binding()
