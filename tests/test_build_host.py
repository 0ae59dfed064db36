"""When the call module is built again, and what the build does where it cannot be."""
import os
import sys

import pytest

from smc_reweight_resample_gb300 import build


@pytest.fixture
def calls(tmp_path, monkeypatch):
    """The module's build with another output and a compiler that writes a line into it."""
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "CALLS_KEY", str(tmp_path / "_build" / "calls.key"))
    monkeypatch.setattr(build, "_calls_command", lambda out: [sys.executable, "-c", f"open({out!r}, 'w').write('built')"])
    return build


def test_the_module_is_built_again_for_another_torch_or_python(calls, monkeypatch):
    import torch

    started = calls._start_calls()
    assert started is not None
    calls._finish_calls(started)
    assert os.path.exists(calls.CALLS)
    assert calls._start_calls() is None  # up to date
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        again = calls._start_calls()
        assert again is not None
        again[0].communicate()
    assert calls._start_calls() is None
    with monkeypatch.context() as m:
        m.setattr(sys, "version", "3.99")
        again = calls._start_calls()
        assert again is not None
        again[0].communicate()
    os.remove(calls.CALLS_KEY)  # a module of unknown origin
    again = calls._start_calls()
    assert again is not None
    calls._finish_calls(again)
    assert calls._start_calls() is None


def test_without_a_compiler_the_library_is_built_and_the_build_fails(calls, monkeypatch):
    built = []
    monkeypatch.setattr(calls, "_calls_command", lambda out: ["/nonexistent/compiler", out])
    monkeypatch.setattr(calls, "_build_library", lambda *a: built.append(a))
    with pytest.raises(RuntimeError, match="no compiler"):
        calls.build(force=True)
    assert len(built) == 1


def test_without_torch_only_the_library_is_built(calls, monkeypatch):
    built = []
    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.setattr(calls, "_build_library", lambda *a: built.append(a))
    assert calls.build(force=True) == calls.LIB
    assert len(built) == 1 and not os.path.exists(calls.CALLS)


def test_a_compiler_that_fails_leaves_the_module_as_it_was(calls, monkeypatch):
    calls._finish_calls(calls._start_calls())
    monkeypatch.setattr(calls, "_calls_command", lambda out: [sys.executable, "-c", "raise SystemExit(3)"])
    with pytest.raises(RuntimeError, match="compiler failed"):
        calls._finish_calls(calls._start_calls())
    assert open(calls.CALLS).read() == "built"
