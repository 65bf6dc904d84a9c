"""Build step for libsq.so, the CUDA library behind the C ABI in include/sq.h.

Compiles the translation units of csrc/ (sq_api.cu: the int8 layer, sq_mx4_api.cu:
the microscaled 4-bit operators) for sm_100a with nvcc, side by side, and links
them into ``libsq.so`` next to this file (in-tree, so it travels with the source
tree).  cudart is linked statically; only the ABI symbols are exported.

    python -m w8a8_int8_gemm_channel_b200._build [--force] [-v]
"""
from __future__ import annotations

import contextlib
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libsq.so")
MAIN = os.path.join(CSRC, "sq_api.cu")
UNITS = [MAIN, os.path.join(CSRC, "sq_mx4_api.cu")]
# object files, kept between builds (their names hold the process id until done), and the flags that they and the
# library were made with
OBJ = os.path.join(PKG, "_build.d")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = [
    *ARCH,
    "-lineinfo",
    "-O3",
    "-std=c++17",
    "--expt-relaxed-constexpr",
    "-Xcompiler",
    "-fPIC,-fvisibility=hidden",
]
LINK_FLAGS = ["-shared", "-cudart", "static", "-ldl", "-lrt", "-lpthread"]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def sources():
    return sorted(
        os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))
    ) + [os.path.join(INCLUDE, "sq.h")]


def _flags(path, extra=None) -> str:
    """The flags an object, or the library, is made with."""
    return " ".join([*NVCC_FLAGS, *(extra or []), *(LINK_FLAGS if path == LIB else [])])


def _flags_file(path):
    return os.path.join(OBJ, os.path.basename(path) + ".flags")


def _older(path, files, extra) -> bool:
    """Whether a built file is missing, older than one of the files, or made with other flags."""
    if not os.path.exists(path) or not os.path.exists(_flags_file(path)):
        return True
    with open(_flags_file(path)) as f:
        if f.read() != _flags(path, extra):
            return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(s) > t for s in files)


def _place(tmp, path, extra):
    """A finished file takes its name; without its flags it counts as missing, so they come last."""
    with contextlib.suppress(FileNotFoundError):
        os.remove(_flags_file(path))
    os.replace(tmp, path)
    new = _flags_file(path) + f".tmp{os.getpid()}"
    with open(new, "w") as f:
        f.write(_flags(path, extra))
    os.replace(new, _flags_file(path))


def stale(extra=None) -> bool:
    return _older(LIB, sources(), extra)


def _headers(unit, seen=None):
    """The headers of csrc/ and include/ that a unit includes, directly or through one another."""
    seen = set() if seen is None else seen
    with open(unit) as f:
        names = re.findall(r'^#include "([^"]+)"', f.read(), re.M)
    for name in names:
        for d in (CSRC, INCLUDE):
            p = os.path.join(d, name)
            if os.path.exists(p) and p not in seen:
                seen.add(p)
                _headers(p, seen)
    return seen


def _object(unit):
    return os.path.join(OBJ, os.path.basename(unit)[:-3] + ".o")


def _object_stale(unit, extra=None) -> bool:
    return _older(_object(unit), [unit, *_headers(unit)], extra)


def objects(force: bool = False, verbose: bool = False, extra=None) -> list:
    """Compile the units whose objects are stale; return the objects' paths."""
    os.makedirs(OBJ, exist_ok=True)
    running = []
    for unit in UNITS:
        if force or _object_stale(unit, extra):
            tmp = _object(unit) + f".tmp{os.getpid()}.o"
            cmd = [nvcc(), *NVCC_FLAGS, *(extra or []), "-I", INCLUDE, "-I", CSRC, "-c", "-o", tmp, unit]
            if verbose:
                print(" ".join(cmd), flush=True)
            running.append((subprocess.Popen(cmd), cmd, tmp, _object(unit)))
    failed = None
    for p, cmd, tmp, obj in running:
        if p.wait() != 0:
            failed = failed or subprocess.CalledProcessError(p.returncode, cmd)
        else:
            _place(tmp, obj, extra)
    if failed:
        raise failed
    return [_object(unit) for unit in UNITS]


def build(force: bool = False, verbose: bool = False, extra=None) -> str:
    """Compile libsq.so if it is missing, older than any source or made with other flags; return its path."""
    if not force and not stale(extra):
        return LIB
    objs = objects(force, verbose, extra)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-o", tmp, *objs, *LINK_FLAGS]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    _place(tmp, LIB, extra)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None)
    print(LIB)
