"""Build the CUDA library ``libsmcsd.so`` in-tree for sm_103a (GB300).

Each translation unit is compiled in its own nvcc process, in parallel, then linked into one
shared library with the CUDA runtime linked statically; the host-only call module ``_calls.so`` is
compiled beside them. Objects go to ``_build/`` beside this
file; the library is written next to this file. Run ``python -m smc_reweight_resample_gb300.build``
or call ``build()``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libsmcsd.so")
SOURCES = ["api.cu", "verify_stream.cu", "stream_tma.cu", "finish.cu", "sd_sample.cu", "resample_pacer.cu",
           "static_scratch.cu", "serve_api.cu", "kv_cache.cu", "tree_attention.cu",
           "tree_attention_wide.cu",
           "tree_attention_narrow.cu", "logits_process.cu", "ops_api.cu", "beam_select.cu", "kv_pages.cu", "distill_loss.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


# CPython module that marshals tensors for the calls around the verify (csrc/py_calls.cpp): host code only
CALLS = os.path.join(HERE, "_calls.so")
CALLS_KEY = os.path.join(BUILD, "calls.key")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _flags():
    return ["-std=c++17", "-O3", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC",
            "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]


def _stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")] + [os.path.join(INCLUDE, "smcsd.h")]
    return any(os.path.getmtime(d) > t for d in deps)


# The library with the opt-in device self-checks (-DSMCSD_CHECKS): every check site records its
# code and the offending value in the workspace instead of making the access. Built on request
# (build_checks) into its own folder, for the tests that run the parity cases against it.
CHECKS_BUILD = os.path.join(HERE, "_build_checks")
CHECKS_LIB = os.path.join(CHECKS_BUILD, "libsmcsd_checks.so")


def build_checks(force: bool = False, verbose: bool = False) -> str:
    return build(force, verbose, extra_flags=("-DSMCSD_CHECKS",), out=CHECKS_LIB,
                 objdir=CHECKS_BUILD)


def _calls_command(out: str):
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    inc = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[x for d in inc for x in ("-I", d)],
            os.path.join(CSRC, "py_calls.cpp"), "-o", out, "-L", os.path.join(root, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]


def _calls_key() -> str:
    """What the module is good for: one Python, one torch with its C++ ABI, one compiler line."""
    import torch

    return "\n".join([sys.version, torch.__version__, *_calls_command(CALLS)])


def _start_calls():
    """The module's compiler, running, with its output and key; None if the module is up to date, or if there is no torch that
    it could be called from; or the error that kept the compiler from running."""
    deps = [os.path.join(CSRC, "py_calls.cpp"), os.path.join(INCLUDE, "smcsd.h")]
    try:
        key = _calls_key()
    except ImportError:
        return None
    if os.path.exists(CALLS) and all(os.path.getmtime(d) <= os.path.getmtime(CALLS) for d in deps):
        try:
            with open(CALLS_KEY) as f:
                if f.read() == key:
                    return None
        except OSError:
            pass
    folder = os.path.dirname(CALLS_KEY)  # what a build that is stopped leaves behind lies among the objects
    os.makedirs(folder, exist_ok=True)
    tmp = os.path.join(folder, f"{os.path.basename(CALLS)}.tmp{os.getpid()}")
    try:
        return subprocess.Popen(_calls_command(tmp), stdout=subprocess.PIPE, stderr=subprocess.STDOUT), tmp, key
    except OSError as e:
        return e


def _remove(path):
    if os.path.exists(path):
        os.remove(path)


def _drop_calls(started):
    """Ends the module's compiler and takes its output away."""
    if isinstance(started, tuple):
        started[0].kill()
        started[0].communicate()
        _remove(started[1])


def _finish_calls(started):
    if started is None:
        return
    if isinstance(started, OSError):
        raise RuntimeError(f"no compiler for py_calls.cpp: {started}") from started
    proc, tmp, key = started
    log, _ = proc.communicate()
    if proc.returncode != 0:
        _remove(tmp)
        sys.stdout.write(log.decode(errors="replace"))
        raise RuntimeError("the compiler failed for py_calls.cpp")
    _remove(CALLS_KEY)
    os.replace(tmp, CALLS)
    with open(CALLS_KEY, "w") as f:
        f.write(key)


def build(force: bool = False, verbose: bool = False, extra_flags=(), out: str = LIB,
          objdir: str = BUILD) -> str:
    """The library, and the call module beside it, where they are not up to date. The library is there even if the module
    cannot be built, which raises all the same."""
    calls = _start_calls()
    try:
        if force or _stale(out):
            _build_library(verbose, extra_flags, out, objdir)
    except BaseException:
        _drop_calls(calls)
        raise
    _finish_calls(calls)
    return out


def _build_library(verbose, extra_flags, out, objdir):
    os.makedirs(objdir, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [cc, *_flags(), *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, pr in procs:
        log, _ = pr.communicate()
        if verbose or pr.returncode != 0:
            sys.stdout.write(log.decode(errors="replace"))
        if pr.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError(f"nvcc failed for {failed}")
    tmp = os.path.join(objdir, f"{os.path.basename(out)}.tmp{os.getpid()}")
    try:
        subprocess.check_call([cc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, out)
    finally:
        _remove(tmp)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
