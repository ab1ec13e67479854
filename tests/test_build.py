"""When the build makes the binding's C++ part anew (the compiler is a stand-in that writes the
file; no GPU needed)."""
import os
import sys
import types

import pytest
import torch

from paged_kv_cache_241_gb300 import build


@pytest.fixture
def compiler(monkeypatch, tmp_path):
    """Commands that the build runs for the module, which goes to a folder of its own."""
    ran = types.SimpleNamespace(commands=[], code=0)

    def run(cmd, **kw):
        ran.commands.append(cmd)
        if ran.code == 0:
            open(cmd[cmd.index("-o") + 1], "w").write("module")
        return types.SimpleNamespace(returncode=ran.code, stdout="", stderr="no")

    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build, "OBJ_DIR", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "run", run)
    return ran


def made(compiler):
    compiler.commands.clear()
    build._build_call_module()
    return len(compiler.commands)


def test_made_once(compiler):
    assert made(compiler) == 1 and made(compiler) == 0
    assert f'-DPKV_TORCH_VERSION="{torch.__version__}"' in " ".join(map(str, build_command(compiler)))


def build_command(compiler):
    os.remove(build.call_module())
    assert made(compiler) == 1
    return compiler.commands[0]


def test_made_anew_for_another_torch_whatever_its_files_times(compiler, monkeypatch):
    assert made(compiler) == 1
    later = os.path.getmtime(build.call_module()) + 1e6
    os.utime(build.call_module(), (later, later))
    monkeypatch.setattr(torch, "__version__", "0.1")
    assert made(compiler) == 1 and made(compiler) == 0
    monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    assert made(compiler) == 1 and made(compiler) == 0


def test_made_anew_for_another_toolkit(compiler, monkeypatch):
    assert made(compiler) == 1
    monkeypatch.setattr(build, "nvcc", lambda: "/nowhere/cuda/bin/nvcc")
    assert made(compiler) == 1 and made(compiler) == 0


def test_a_compilation_that_fails_is_tried_again(compiler, monkeypatch):
    assert made(compiler) == 1
    version = torch.__version__
    monkeypatch.setattr(torch, "__version__", "0.1")
    compiler.code = 1
    for _ in range(2):
        with pytest.raises(RuntimeError, match="failed"):
            build._build_call_module()
    # (what is there may be half of a file)
    monkeypatch.setattr(torch, "__version__", version)
    compiler.code = 0
    assert made(compiler) == 1 and made(compiler) == 0


@pytest.fixture
def library(monkeypatch, tmp_path):
    """The whole build with a stand-in for every compiler, in a folder of its own."""
    def run(cmd, **kw):
        assert "pycall.cc" not in " ".join(cmd)
        open(cmd[cmd.index("-o") + 1], "w").write("made")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    for name, to in (("HERE", ""), ("OBJ_DIR", "objects"), ("LIB", "libpkv.so")):
        monkeypatch.setattr(build, name, str(tmp_path / to))
    monkeypatch.setattr(build.subprocess, "run", run)
    return tmp_path / "libpkv.so"


def test_the_library_is_built_without_torch(library, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == str(library) and library.exists()
    assert "torch" in capsys.readouterr().err


def test_the_library_is_built_with_a_torch_that_has_no_cuda(library, monkeypatch, capsys):
    monkeypatch.setattr(torch.version, "cuda", None)
    assert build.build() == str(library) and library.exists()
    assert "CUDA" in capsys.readouterr().err


def test_the_library_is_built_where_the_module_cannot_be(library, monkeypatch):
    """Its error is told of behind the library's link."""
    def no_module():
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(build, "_build_call_module", no_module)
    with pytest.raises(RuntimeError, match="g.. failed"):
        build.build()
    assert library.exists()
