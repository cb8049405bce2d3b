"""Compile libattn_sink.so for sm_103a with nvcc (in-tree, no torch extension), and
beside it the native side of the binding's small calls, attn_sink_fast.so, with
g++ against the installed torch's headers."""
from __future__ import annotations

import os
import platform
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libattn_sink.so")
# Test build: the same sources with the bounded waits lowered to 2 ms and the
# hooks that let a test withhold one tile (exercises the timeout path).
TEST_LIB_PATH = os.path.join(LIB_DIR, "libattn_sink_test.so")
TEST_FLAGS = ["-DATTN_SINK_TEST_HOOKS", "-DATTN_SINK_WAIT_LIMIT_NS=2000000ull"]
FAST_PATH = os.path.join(LIB_DIR, "attn_sink_fast.so")
FAST_SOURCE = os.path.join(CSRC, "fast_calls.cpp")
FAST_STAMP = FAST_PATH + ".built-for"    # which torch and Python the module is for
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libattn_sink.so")


def _sources() -> list[str]:
    files = [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))
             if f.endswith((".cu", ".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in ("attn_sink.h", "attn_sink_step.h",
                                                   "attn_sink_cache.h")]
    return files


def _up_to_date(path: str, sources: list[str]) -> bool:
    return (os.path.exists(path)
            and os.path.getmtime(path) >= max(os.path.getmtime(s) for s in sources))


def fast_target() -> str:
    """What the native module depends on beside its sources."""
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}, {platform.machine()}"


def fast_built_for() -> str | None:
    """The fast_target() the native module was built for, None without one."""
    try:
        with open(FAST_STAMP) as f:
            return f.read()
    except OSError:
        return None


def _start(cmd: list[str], verbose: bool) -> subprocess.Popen:
    if verbose:
        print(" ".join(cmd))
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _finish(proc: subprocess.Popen, tmp: str, path: str, verbose: bool) -> None:
    said = proc.communicate()[0]
    if proc.returncode != 0:
        raise RuntimeError(f"{proc.args[0]} failed ({proc.returncode}):\n{said}")
    if verbose:
        print(said)
    os.replace(tmp, path)


def _fast_command(out: str) -> list[str]:
    import torch
    root = os.path.dirname(torch.__file__)
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("g++ not found: it is required to build attn_sink_fast.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
            "-I", os.path.join(root, "include"),
            "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"), "-I", cuda,
            FAST_SOURCE, "-o", out, "-L" + os.path.join(root, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False, test: bool = False) -> str:
    """Build the shared library (or, with test=True, the test build) if any
    source is newer than it, and the binding's native module; return the
    library's path."""
    path = TEST_LIB_PATH if test else LIB_PATH
    os.makedirs(LIB_DIR, exist_ok=True)
    jobs = []
    tmp = path + ".tmp"
    if force or not _up_to_date(path, _sources()):
        cmd = [_nvcc(), *ARCH_FLAGS, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
               "-shared", "-I", INCLUDE, *(TEST_FLAGS if test else []), "-o", tmp,
               os.path.join(CSRC, "attn_sink_api.cu")]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        jobs.append((_start(cmd, verbose), tmp, path))
    fast = not test and (force or fast_built_for() != fast_target() or not _up_to_date(
        FAST_PATH, [FAST_SOURCE, os.path.join(INCLUDE, "attn_sink_step.h"),
                    os.path.join(INCLUDE, "attn_sink_cache.h")]))
    if fast:
        tmp = FAST_PATH + ".tmp"
        jobs.append((_start(_fast_command(tmp), verbose), tmp, FAST_PATH))
    for job in jobs:                       # they compile side by side
        _finish(*job, verbose)
    if fast:
        with open(FAST_STAMP, "w") as f:
            f.write(fast_target())
    return path


if __name__ == "__main__":
    print(build(force=True, verbose=True))
