"""The build where the binding's short way cannot be compiled, on the CPU and in a copy of the package:
the library is linked all the same, and what an earlier build left of the short way goes."""
import importlib.util
import os
import shutil
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "speculative_decoding_verification_65_gb300"


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The copy's build module, whose compiler and linker of the library only make their files."""
    for part in (os.path.join(NAME, "csrc"), "include"):
        shutil.copytree(os.path.join(ROOT, part), tmp_path / part,
                        ignore=shutil.ignore_patterns("*.o", "*.so"))
    shutil.copy(os.path.join(ROOT, NAME, "build.py"), tmp_path / NAME)
    spec = importlib.util.spec_from_file_location("build_copy", tmp_path / NAME / "build.py")
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    monkeypatch.setattr(module, "compile_command", lambda src, obj, extra=(): ["touch", obj])
    monkeypatch.setattr(module, "link_command", lambda objs, out: ["touch", out])
    return module


def torch_at(monkeypatch, place):
    """PyTorch is found at `place` (None: not at all)."""
    spec = place and types.SimpleNamespace(submodule_search_locations=[str(place)])
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec)


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_a_pytorch_without_headers(build, tmp_path, monkeypatch, capsys):
    (tmp_path / "torch").mkdir()
    torch_at(monkeypatch, tmp_path / "torch")
    open(build.CALLS, "w").close()
    assert build.build(force=True) == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS)
    said = capsys.readouterr().out.splitlines()
    assert len(said) == 1 and "_calls.so is left out" in said[0] and "error" in said[0]
    assert sorted(f for f in os.listdir(build.PKG) if ".tmp" in f) == []


def test_no_compiler_for_it(build, tmp_path, monkeypatch, capsys):
    torch_at(monkeypatch, tmp_path)
    monkeypatch.setattr(build, "calls_command", lambda out: [str(tmp_path / "no-such-compiler")])
    build.build()
    assert os.path.exists(build.LIB)
    assert "_calls.so is left out" in capsys.readouterr().out
    # and where the library is there already
    build.build()
    assert os.path.exists(build.LIB)


def test_no_pytorch(build, monkeypatch, capsys):
    torch_at(monkeypatch, None)
    build.build(force=True)
    assert os.path.exists(build.LIB) and capsys.readouterr().out == ""


def test_what_can_be_built_is(build, tmp_path, monkeypatch):
    torch_at(monkeypatch, tmp_path)
    monkeypatch.setattr(build, "calls_command", lambda out: ["touch", out])
    build.build(force=True)
    assert os.path.exists(build.LIB) and os.path.exists(build.CALLS)


def test_a_failure_of_the_library_is_one(build, tmp_path, monkeypatch):
    torch_at(monkeypatch, None)
    monkeypatch.setattr(build, "link_command", lambda objs, out: ["false"])
    with pytest.raises(RuntimeError, match="linking"):
        build.build(force=True)
    monkeypatch.setattr(build, "compile_command", lambda src, obj, extra=(): ["false"])
    with pytest.raises(RuntimeError, match="compiling"):
        build.build(force=True)
