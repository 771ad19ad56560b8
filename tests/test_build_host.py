"""The build script without its compilers: what it makes where PyTorch, or PyTorch's headers, are missing."""
import importlib.util
import os

import pytest

from conftest import ROOT


@pytest.fixture
def script(tmp_path, monkeypatch):
    """The build script with its outputs in tmp_path and commands that only write their output files."""
    path = os.path.join(ROOT, "exact_tiled_attention_26_gb300", "build.py")
    spec = importlib.util.spec_from_file_location("_build_script", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for name in ("LIB", "CALLS"):
        monkeypatch.setattr(mod, name, str(tmp_path / os.path.basename(getattr(mod, name))))
    monkeypatch.setattr(mod, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(mod, "_nvcc", lambda: "/opt/cuda/bin/nvcc")
    mod.commands = []

    def run(cmd, verbose):
        mod.commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return ""
    monkeypatch.setattr(mod, "_run", run)
    return mod


def test_both_libraries(script):
    script.build()
    assert os.path.exists(script.LIB) and os.path.exists(script.CALLS)
    links = [c for c in script.commands if "-shared" in c]
    assert [c[0] for c in links] == ["/opt/cuda/bin/nvcc", "g++"]  # the module links against the library


def test_the_library_without_pytorch(script, monkeypatch, capsys):
    """The C library needs nvcc alone."""
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert script.build() == script.LIB
    assert os.path.exists(script.LIB) and not os.path.exists(script.CALLS)
    assert not any(c[0] == "g++" for c in script.commands)
    assert "tensor_calls.so" in capsys.readouterr().err


def test_the_library_is_made_before_the_module_fails(script, monkeypatch):
    run = script._run

    def failing(cmd, verbose):
        if cmd[0] == "g++":
            raise RuntimeError("no header")
        return run(cmd, verbose)
    monkeypatch.setattr(script, "_run", failing)
    with pytest.raises(RuntimeError):
        script.build()
    assert os.path.exists(script.LIB) and not os.path.exists(script.CALLS)
