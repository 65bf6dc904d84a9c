"""The build keeps what is up to date and nothing else: a library or an object
made with other flags is made again.  A compiler that only writes its arguments
down stands in for nvcc.
"""
import os
import subprocess

import pytest

from w8a8_int8_gemm_channel_b200 import _build


@pytest.fixture
def made(tmp_path, monkeypatch):
    """A copy of the build's paths in an empty folder; made() lists what has been compiled or linked since it was last asked."""
    csrc, log = tmp_path / "csrc", tmp_path / "log"
    csrc.mkdir()
    for name, text in (("a.cu", '#include "both.cuh"\n'), ("b.cu", '#include "both.cuh"\n#include "b.cuh"\n'), ("both.cuh", ""), ("b.cuh", "")):
        (csrc / name).write_text(text)
        os.utime(csrc / name, (1, 1))
    (tmp_path / "sq.h").write_text("")
    os.utime(tmp_path / "sq.h", (1, 1))
    fake = tmp_path / "nvcc"
    fake.write_text(f"""#!/bin/sh
case "$*" in *-Dbroken*) exit 1;; esac
while [ "$1" != -o ]; do shift; done
echo "$2" >> {log}
echo made > "$2"
""")
    fake.chmod(0o755)
    monkeypatch.setenv("NVCC", str(fake))
    for k, v in (("CSRC", csrc), ("INCLUDE", tmp_path), ("LIB", tmp_path / "lib.so"), ("OBJ", tmp_path / "obj")):
        monkeypatch.setattr(_build, k, str(v))
    monkeypatch.setattr(_build, "UNITS", [str(csrc / "a.cu"), str(csrc / "b.cu")])

    def since():
        lines = log.read_text().split() if log.exists() else []
        log.write_text("")
        return sorted(os.path.basename(x).split(".")[0] for x in lines)

    return since


def touch(path):
    t = os.path.getmtime(_build.LIB) + 10
    os.utime(path, (t, t))


def test_nothing_is_made_twice(made):
    _build.build()
    assert made() == ["a", "b", "lib"]
    assert _build.build() == _build.LIB
    assert made() == []


def test_sources_and_headers(made):
    _build.build()
    made()
    touch(os.path.join(_build.CSRC, "b.cuh"))
    _build.build()
    assert made() == ["b", "lib"]


def test_other_flags(made, monkeypatch):
    _build.build()
    made()
    monkeypatch.setattr(_build, "NVCC_FLAGS", [*_build.NVCC_FLAGS, "-DOTHER"])
    _build.build()
    assert made() == ["a", "b", "lib"]
    _build.build(extra=["-DMORE"])
    assert made() == ["a", "b", "lib"]
    _build.build(extra=["-DMORE"])
    assert made() == []
    _build.build()  # none of them is left in the next link
    assert made() == ["a", "b", "lib"]
    monkeypatch.setattr(_build, "LINK_FLAGS", [*_build.LINK_FLAGS, "-lother"])
    _build.build()
    assert made() == ["lib"]


def test_a_build_that_failed_is_made_again(made):
    _build.build()
    made()
    with pytest.raises(subprocess.CalledProcessError):
        _build.build(extra=["-Dbroken"])
    made()
    _build.build()
    assert made() == []
    os.remove(_build._flags_file(_build._object(_build.UNITS[0])))  # stopped between an object and its flags
    touch(os.path.join(_build.CSRC, "b.cu"))
    _build.build()
    assert made() == ["a", "b", "lib"]
