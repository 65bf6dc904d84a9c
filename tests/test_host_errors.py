"""What the host code does about errors, on a stand-in for the CUDA runtime."""
import ctypes
import itertools

import pytest

import w8a8_int8_gemm_channel_b200 as sq
from tests import fake_cuda

PIVOT, WAIT, WAIT2 = 0xA00, 0x200, 0x400


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return fake_cuda.load(tmp_path_factory.mktemp("fake"))


def words(lib):
    found = [lib.fake_variable(b"g_sq_device_error", i) for i in range(3)]
    assert found[0] and found[1] and not found[2]
    return [ctypes.c_uint32.from_address(p) for p in found[:2]]


def status(lib):
    code = ctypes.c_uint32(99)
    return lib.sq_device_status(None, ctypes.byref(code)), code.value


def test_no_pending_error_is_lost(lib):
    """Each translation unit has an error word (only the int8 one's kernels meet pivots).  A wait that gave up, which
    makes outputs wrong, is reported before a pivot, and the pivot by the next call."""
    lib.fake_reset(-1)
    kind = {0: sq.SQ_OK, PIVOT: sq.SQ_ERR_INVALID_ARG, WAIT: sq.SQ_ERR_TIMEOUT, WAIT2: sq.SQ_ERR_TIMEOUT}
    cases = set(itertools.product((0, PIVOT, WAIT, WAIT2), (0, WAIT, WAIT2)))
    for int8, mx4 in sorted(cases):
        for w, v in zip(words(lib), (int8, mx4)):
            w.value = v
        want = sorted({kind[v] for v in (int8, mx4) if v}, key=lambda k: k != sq.SQ_ERR_TIMEOUT)
        for k in want:
            st, code = status(lib)
            assert st == k and code in (int8, mx4) and kind[code] == k, (int8, mx4)
        assert status(lib) == (sq.SQ_OK, 0)
        assert [w.value for w in words(lib)] == [0, 0]
