"""When the binding's short way is compiled anew, and when it is loaded, on the CPU: it belongs to one
PyTorch, whose inline functions it holds, and to the status codes of the library's header."""
import os
import time

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from speculative_decoding_verification_65_gb300 import build as sv_build  # noqa: E402
from tests.test_build_without_calls import build, torch_at  # noqa: E402, F401


@pytest.fixture
def made(build, tmp_path, monkeypatch):  # noqa: F811
    """The build module of a copy that has been built against a PyTorch 1.0."""
    (tmp_path / "torch").mkdir()
    (tmp_path / "torch" / "version.py").write_text("__version__ = '1.0'\n")
    torch_at(monkeypatch, tmp_path / "torch")
    count = []

    def command(out):
        count.append(out)
        return ["touch", out]
    monkeypatch.setattr(build, "calls_command", command)
    build.build()
    assert len(count) == 1 and build.calls_match() and not build.calls_stale()
    build.build()
    assert len(count) == 1
    return build, count


def test_another_version_of_pytorch(made, tmp_path):
    build, count = made  # noqa: F811
    (tmp_path / "torch" / "version.py").write_text("__version__ = '1.1'\n")
    assert not build.calls_match() and build.calls_stale()
    build.build()
    assert len(count) == 2 and build.calls_match()


def test_a_pytorch_elsewhere(made, tmp_path, monkeypatch):
    build, count = made  # noqa: F811
    (tmp_path / "other").mkdir()
    (tmp_path / "other" / "version.py").write_text("__version__ = '1.0'\n")
    torch_at(monkeypatch, tmp_path / "other")
    assert not build.calls_match() and build.calls_stale()


@pytest.mark.parametrize("name", ["CALLS_SRC", "CALLS_HEADER"])
def test_a_newer_source(made, name):
    build, count = made  # noqa: F811
    later = time.time() + 60
    os.utime(getattr(build, name), (later, later))
    assert build.calls_stale()


def test_one_that_says_nothing_of_what_it_was_made_for(made):
    build, count = made  # noqa: F811
    os.remove(build.CALLS_FOR)
    assert not build.calls_match() and build.calls_stale()


def test_a_failed_build_leaves_none(made, monkeypatch, capsys):
    build, count = made  # noqa: F811
    monkeypatch.setattr(build, "calls_command", lambda out: ["false"])
    build.build(force=True)
    assert "left out" in capsys.readouterr().out
    assert not os.path.exists(build.CALLS) and not os.path.exists(build.CALLS_FOR)


def test_another_pytorchs_is_not_loaded(monkeypatch):
    monkeypatch.setattr(sv, "_short", None)
    monkeypatch.setattr(sv, "_run", None)
    monkeypatch.setattr(sv_build, "calls_match", lambda: False)
    assert sv._load_calls() is False and sv._run is None
