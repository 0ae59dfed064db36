"""What a build leaves behind: nothing beside the package's sources but the library and the call module, and no compiled file in the tree."""
import os
import subprocess
import sys
import time

import pytest

from smc_reweight_resample_gb300 import build

ROOT = os.path.dirname(build.HERE)
WRITES = "import sys; open({out!r}, 'w').write('half'); sys.exit({code})"


@pytest.fixture
def calls(tmp_path, monkeypatch):
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "CALLS_KEY", str(tmp_path / "_build" / "calls.key"))
    return build


def left(tmp_path):
    return sorted(os.path.join(os.path.relpath(at, tmp_path), f) for at, _, files in os.walk(tmp_path) for f in files)


def test_a_compiler_that_fails_after_it_wrote_leaves_nothing(calls, tmp_path, monkeypatch):
    monkeypatch.setattr(calls, "_calls_command", lambda out: [sys.executable, "-c", WRITES.format(out=out, code=3)])
    with pytest.raises(RuntimeError, match="compiler failed"):
        calls._finish_calls(calls._start_calls())
    assert left(tmp_path) == []


def test_a_library_that_fails_stops_the_modules_compiler(calls, tmp_path, monkeypatch):
    monkeypatch.setattr(calls, "_calls_command", lambda out: [sys.executable, "-c", WRITES.format(out=out, code=0) + "; import time; time.sleep(60)"])

    def fails(*a):
        end = time.monotonic() + 10
        while not left(tmp_path) and time.monotonic() < end:
            time.sleep(0.01)
        raise RuntimeError("nvcc failed")
    monkeypatch.setattr(calls, "_build_library", fails)
    with pytest.raises(RuntimeError, match="nvcc"):
        calls.build(force=True)
    assert left(tmp_path) == []


def test_unfinished_output_lies_below_the_build_folder(calls, tmp_path, monkeypatch):
    """A build that is killed cannot clean up: its output must lie where it is ignored."""
    monkeypatch.setattr(calls, "_calls_command", lambda out: [sys.executable, "-c", WRITES.format(out=out, code=0)])
    started = calls._start_calls()
    started[0].communicate()
    assert [os.path.dirname(f) for f in left(tmp_path)] == ["_build"]


def test_no_compiled_file_is_in_the_tree():
    if not os.path.isdir(os.path.join(ROOT, ".git")):
        pytest.skip("not a working tree")
    names = subprocess.run(["git", "-C", ROOT, "ls-files", "-z"], capture_output=True, check=True).stdout.decode().split("\0")
    compiled = []
    for name in filter(None, names):
        path = os.path.join(ROOT, name)
        if os.path.isfile(path):
            with open(path, "rb") as f:
                if f.read(4) in (b"\x7fELF", b"!<ar"):
                    compiled.append(name)
    assert compiled == []
