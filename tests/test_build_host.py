"""The build's two parts, without a GPU and without compiling: the library is
linked whether or not the Python module of the tensor calls can be made."""
import os
import types

import pytest

from tensor_transformer_mlp_tcgen05_gb300 import build as build_mod


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    """Compilers that write their output and succeed; all paths under
    tmp_path.  Returns the commands that were run."""
    runs = []

    def run(cmd, **_):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("made")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build_mod.subprocess, "run", run)
    monkeypatch.setattr(build_mod, "nvcc_path", lambda: "nvcc")
    monkeypatch.setattr(build_mod, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(build_mod, "LIB_PATH", str(tmp_path / "libtpmlp.so"))
    return runs


def test_the_library_does_not_need_the_python_module(compilers, monkeypatch):
    def fails(force=False):
        raise RuntimeError("g++ failed for pycall.cpp")

    monkeypatch.setattr(build_mod, "build_pycall", fails)
    with pytest.raises(RuntimeError, match="pycall"):
        build_mod.build(force=True)
    assert os.path.exists(build_mod.LIB_PATH)
    assert len(compilers) == len(build_mod.SOURCES) + 1


def test_without_torch_the_library_is_all_there_is(compilers, monkeypatch):
    monkeypatch.setattr(build_mod, "has_torch", lambda: False)
    monkeypatch.setattr(build_mod, "build_pycall", lambda force=False: 1 / 0)
    for _ in range(2):   # made, and found made
        assert build_mod.build() == build_mod.LIB_PATH
    assert os.path.exists(build_mod.LIB_PATH)
    assert len(compilers) == len(build_mod.SOURCES) + 1


def test_the_python_module_is_one_torchs_and_one_pythons(monkeypatch):
    """Built for another torch or Python it is not loaded, but asked for."""
    import sys

    import torch
    from tensor_transformer_mlp_tcgen05_gb300 import binding
    build_mod.build()
    path = build_mod.pycall_path()
    assert os.path.exists(path) and torch.__version__ in path
    assert sys.implementation.cache_tag in os.path.basename(path)
    assert binding.tensor_calls().__name__.endswith("._pycall")
    for where, name in ((torch, "__version__"),
                        (sys.implementation, "cache_tag")):
        with monkeypatch.context() as m:
            m.setattr(binding, "_calls", None)
            m.setattr(where, name, "0.0.0")
            with pytest.raises(RuntimeError, match="0.0.0.* is missing"):
                binding.tensor_calls()
