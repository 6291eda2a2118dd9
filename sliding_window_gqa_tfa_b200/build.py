"""Build libtfa.so (the C-ABI CUDA library) in-tree with nvcc for sm_100a, and
_calls.so (the binding's native calls, against the installed torch) with g++.

    python -m sliding_window_gqa_tfa_b200.build [--verbose] [--changed]

Every source is compiled again unless --changed is given (then only those whose
source, or any header, is newer than the object).

The library is written next to this file; it links the CUDA runtime
statically and resolves the driver's cuTensorMapEncodeTiled at run time, so it
needs no library path beyond the NVIDIA driver.  _calls.so takes the library's
addresses from it and resolves torch's from the torch that is imported, which must
be the one it was built for; the binding goes without it otherwise.
"""
from __future__ import annotations

import contextlib
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtfa.so")
CALLS = os.path.join(HERE, "_calls.so")
CALLS_SOURCE = os.path.join(CSRC, "calls.cpp")
OBJ = os.path.join(HERE, "_build")  # object files (git-ignored)
SOURCES = [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith(".cu")]
HEADERS = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
    os.path.join(ROOT, "include", "tfa.h")]


def nvcc() -> str:
    for cand in [os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"]:
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    raise RuntimeError("nvcc not found")


def needs_build() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(CALLS):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
    return any(os.path.getmtime(f) > t for f in SOURCES + HEADERS + [CALLS_SOURCE])


def calls_command(out: str) -> list[str]:
    """g++'s command for _calls.so."""
    import torch

    base = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DTFA_BUILT_FOR="torch {torch.__version__}, Python {sys.version_info.major}.{sys.version_info.minor}"',
            "-isystem", base, "-isystem",
            sysconfig.get_paths()["include"], "-isystem", cuda, "-o", out, CALLS_SOURCE,
            "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python"]


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    base = [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
            "-Xcompiler", "-fPIC,-O2", "-I", os.path.join(ROOT, "include")]
    if verbose:
        base.insert(1, "-Xptxas=-v")
    # one object per source, compiled side by side; an object newer than its
    # source and every header is kept
    os.makedirs(OBJ, exist_ok=True)
    header_time = max(os.path.getmtime(f) for f in HEADERS)
    objs, running = [], []
    for src in SOURCES:
        obj = os.path.join(OBJ, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), header_time):
            cmd = base + ["-c", "-o", obj + f".tmp{os.getpid()}", src]
            running.append((cmd, obj, subprocess.Popen(cmd)))
    calls_tmp = CALLS + f".tmp{os.getpid()}"
    if force or not os.path.exists(CALLS) or os.path.getmtime(CALLS) < max(os.path.getmtime(CALLS_SOURCE), header_time):
        cmd = calls_command(calls_tmp)
        running.append((cmd, None, subprocess.Popen(cmd)))
    failed = [(cmd, p.returncode) for cmd, _, p in running if p.wait() != 0]
    if failed:
        for _, obj, _ in running:  # what the others have written
            with contextlib.suppress(FileNotFoundError):
                os.remove(calls_tmp if obj is None else obj + f".tmp{os.getpid()}")
        raise subprocess.CalledProcessError(failed[0][1], failed[0][0])
    for _, obj, _ in running:
        if obj is None:
            os.replace(calls_tmp, CALLS)
        else:
            os.replace(obj + f".tmp{os.getpid()}", obj)
    subprocess.run(base + ["-shared", "-o", tmp] + objs, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--changed" not in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
