"""The library linked with a stand-in for the CUDA runtime (fake_cudart.cpp), so
that what its host code does after an error, or plans for a launch, can be seen
on a machine without a GPU.  No kernel runs and no pointer is read.
"""
import ctypes
import os
import shutil
import subprocess
import tempfile

import w8a8_int8_gemm_channel_b200 as sq
from w8a8_int8_gemm_channel_b200 import _build

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "fake_cudart.cpp")


def load(folder):
    """The library, built in `folder`, with the fake's own functions beside the entry points."""
    include = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    path = os.path.join(str(folder), "libsq_fake.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-Wl,-z,defs", "-I", include,
                           "-o", path, SOURCE, *_build.objects()])
    return _open(path)


def another(lib):
    """The same library once more, as if nothing of it had been called."""
    fd, path = tempfile.mkstemp(".so", dir=os.path.dirname(lib._name))
    os.close(fd)
    shutil.copy(lib._name, path)
    new = _open(path)
    os.remove(path)
    return new


def _open(path):
    lib = ctypes.CDLL(path)
    sq._declare(lib)
    lib.fake_launch_name.restype = ctypes.c_char_p
    lib.fake_launch_arg0.restype = lib.fake_variable.restype = ctypes.c_void_p
    lib.fake_variable.argtypes = [ctypes.c_char_p, ctypes.c_int]
    return lib


def launches(lib):
    return [lib.fake_launch_name(i).decode() for i in range(lib.fake_launches())]
