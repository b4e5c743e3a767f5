"""The build step without a compiler: the library does not depend on the Python module beside it,
and that module belongs to the torch that it was compiled against."""
import os
import subprocess

import pytest
import torch

from moe_grouped_gemm_ragged_b200 import _build, _layer


@pytest.fixture
def compiler(monkeypatch, tmp_path):
    """Compilers that write an empty file, or fail where `failing` says so; their commands."""
    run = type("Run", (), {"commands": [], "failing": None})()

    def call(cmd, *args, **kw):
        run.commands.append(cmd)
        if run.failing is not None and run.failing in os.path.basename(cmd[0]):
            raise run.error
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(subprocess, "check_call", call)
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libgg.so"))
    monkeypatch.setattr(_build, "NATIVE", str(tmp_path / "_native.so"))
    return run


def test_build_makes_both(compiler):
    assert _build.build() == _build.LIB
    assert os.path.exists(_build.LIB) and os.path.exists(_build.NATIVE)
    made = len(compiler.commands)
    _build.build()
    assert len(compiler.commands) == made  # up to date


@pytest.mark.parametrize("error", [subprocess.CalledProcessError(1, "g++"),
                                   FileNotFoundError("g++")])
def test_library_is_built_without_the_module(compiler, error):
    """Without g++ or torch's headers the library is made all the same, and a module of older
    sources, which would call it with the old arguments, does not stay."""
    compiler.failing, compiler.error = "g++", error
    open(_build.NATIVE, "w").close()
    os.utime(_build.NATIVE, (1, 1))
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert _build.build() == _build.LIB
    assert os.path.exists(_build.LIB)
    assert not os.path.exists(_build.NATIVE)


def test_a_failing_library_fails_the_build(compiler):
    compiler.failing, compiler.error = "nvcc", subprocess.CalledProcessError(1, "nvcc")
    with pytest.raises(subprocess.CalledProcessError):
        _build.build()


def test_module_of_another_torch_is_not_loaded(monkeypatch):
    """The module's name tells the torch that it was compiled against, so that neither an import
    nor the build takes one of another torch."""
    _build.build()
    assert _layer._load_native() is not None
    name = _build.native_name()
    assert os.path.basename(_build.NATIVE).startswith(name + ".")
    monkeypatch.setattr(torch, "__version__", "2.99.0")
    assert _build.native_name() != name
    assert _layer._load_native() is None
    monkeypatch.undo()
    monkeypatch.setattr(torch.version, "git_version", "0" * 40)
    assert _build.native_name() != name
    assert _layer._load_native() is None


def test_module_built_after_the_import_is_taken_when_the_library_loads(monkeypatch):
    import moe_grouped_gemm_ragged_b200 as gg
    _build.build()
    monkeypatch.setattr(_layer, "_native", None)
    _layer.declare(gg.lib())
    assert _layer._native is not None
