"""What the host code does about errors, on a stand-in for the CUDA runtime."""
import ctypes
import itertools
import os
import subprocess
import sys

import pytest

import w8a8_int8_gemm_channel_b200 as sq
from tests import fake_cuda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


WS = 0x7F0000100000


def moe(lib, T=4, topk=2, E=8, H=256, I=160):
    """An experts layer on fake addresses, which nothing reads: (status, address of the tile words)."""
    A = 0x7F0000001000
    size = lib.sq_mx4_moe_workspace_size(T, topk, E, H, I)
    st = lib.sq_mx4_moe(A, A, A, A, T, topk, E, H, I, A, A, A, A, A, A, A, sq.SQ_BF16, WS, size, None)
    groups = min(E, T * topk)
    return st, WS + -(-groups * T * I // 2 // 256) * 256 + groups * lib.sq_mx4_scale_size(1, I)


def test_experts_layer_whose_second_half_is_not_launched(lib):
    """The first half counts in words that the second half sets back.  Where that one cannot be launched they are
    cleared, or the next call on the workspace would go by what this one counted."""
    lib.fake_reset(-1)
    assert moe(lib)[0] == sq.SQ_OK
    names = fake_cuda.launches(lib)
    assert len(names) == 2 and "moe_up" in names[0] and "stream" in names[1]
    for fails in (0, 1):
        lib.fake_reset(fails)
        st, words = moe(lib)
        names = fake_cuda.launches(lib)
        assert st == sq.SQ_ERR_CUDA
        assert len(names) == fails + 2 and "clear" in names[-1], names
        last = len(names) - 1
        assert lib.fake_launch_arg0(last) == words
        assert lib.fake_launch_arg1(last) * 4 >= 8 * lib.fake_launch_grid(0)  # a word for each CTA
    lib.fake_reset(-1)
    assert moe(lib)[0] == sq.SQ_OK  # nothing of the error is left


def test_a_launch_that_fails_is_reported(lib):
    A, size = 0x7F0000001000, 1 << 40
    calls = [lambda: lib.sq_mx4_linear(A, 1, A, A, A, 8, 256, 256, A, 1, WS, size, None),
             lambda: lib.sq_mx4_gemm(A, A, A, A, 8, 256, 256, A, 1, WS, size, None),
             lambda: lib.sq_mx4_gemm(A, A, A, A, 300, 256, 256, A, 1, WS, size, None),
             lambda: lib.sq_mx4_quant_weight(A, 0, 8, 256, None, A, A, None),
             lambda: lib.sq_residual_norm_quant(A, 1, 8, 256, A, None, 1, 1.0, A, WS, A, 1e-5, A, A, None)]
    for call in calls:
        lib.fake_reset(-1)
        assert call() == sq.SQ_OK
        n = lib.fake_launches()
        for fails in range(n):
            lib.fake_reset(fails)
            assert call() == sq.SQ_ERR_CUDA and lib.fake_launches() == fails + 1


CHILD = """
import sys, tempfile
import w8a8_int8_gemm_channel_b200 as sq
from tests import fake_cuda
A = 0x7F0000001000
with tempfile.TemporaryDirectory() as d:
    lib = fake_cuda.load(d)
    lib.fake_reset(-1)
    lib.fake_no_memory(1)
    calls = [lambda: lib.sq_mx4_gemm(A, A, A, A, 300, 256, 256, A, 1, A, 1 << 40, None),
             lambda: lib.sq_quant_act(A, 1, 2000, 4096, A, A, A, None),
             lambda: lib.sq_quant_act(A, 0, 2000, 1040, A, A, A, None),
             lambda: lib.sq_silu_mul_quant(A, 1, 2000, 1040, A, A, A, None, None),
             lambda: lib.sq_linear_noalloc(A, 1, A, A, A, 8, 256, 256, A, 1, None),
             lambda: lib.sq_w8a8_gemm(A, A, A, A, 300, 256, 256, A, 1, None)]
    got = [f() for f in calls]
    lib.fake_no_memory(0)
    print(got)
"""


def test_no_exception_leaves_the_library():
    """Without host memory a call does its work or returns an error; an exception would end the process."""
    out = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    assert eval(out.stdout) == [sq.SQ_OK] * 6


def test_a_failed_query_is_asked_again(lib):
    """An occupancy query that fails once fails its call alone."""
    A = 0x7F0000001000
    calls = [lambda: lib.sq_mx4_gemm(A, A, A, A, 300, 256, 256, A, sq.SQ_F32, WS, 1 << 40, None),
             lambda: lib.sq_w8a8_gemm(A, A, A, A, 2048, 4096, 4096, A, sq.SQ_F32, None)]
    for call in calls:
        lib.fake_reset(-1)
        lib.fake_fail_queries(1)
        assert call() == sq.SQ_ERR_CUDA and lib.fake_launches() == 0
        assert call() == sq.SQ_OK and lib.fake_launches() > 0


A = 0x7F0000001000
FIRST_CALLS = {
    "mx4_gemm_many": lambda lib: lib.sq_mx4_gemm(A, A, A, A, 300, 256, 256, A, 1, WS, 1 << 40, None),
    "mx4_gemm_few": lambda lib: lib.sq_mx4_gemm(A, A, A, A, 8, 256, 256, A, 1, WS, 1 << 40, None),
    "mx4_linear": lambda lib: lib.sq_mx4_linear(A, 1, A, A, A, 300, 256, 256, A, 1, WS, 1 << 40, None),
    "mx4_moe": lambda lib: moe(lib)[0],
    "mx4_quant": lambda lib: lib.sq_mx4_quant_weight(A, 0, 8, 256, None, A, A, None),
    "residual_norm": lambda lib: lib.sq_residual_norm_quant_mx4(A, 1, 4000, 256, A, None, 1, 1.0, A, WS, A, 1e-5, A, A, None),
    "quant_act": lambda lib: lib.sq_quant_act(A, 1, 2000, 1040, A, A, A, None),
    "w8a8_gemm": lambda lib: lib.sq_w8a8_gemm(A, A, A, A, 2048, 4096, 4096, A, 1, None),
    "linear_noalloc": lambda lib: lib.sq_linear_noalloc(A, 1, A, A, A, 8, 256, 256, A, 1, None),
}


@pytest.mark.parametrize("name", FIRST_CALLS)
def test_an_error_of_the_runtime_is_one_calls_error(lib, name):
    """Whichever call of the runtime fails in a first use, the next use works and is not told of it."""
    call, n = FIRST_CALLS[name], 0
    while True:
        fresh = fake_cuda.another(lib)
        n += 1
        fresh.fake_reset(-1)
        fresh.fake_fail_call(n)
        st = call(fresh)
        if fresh.fake_calls_left() > 0:  # fewer than n calls
            break
        assert st in (sq.SQ_OK, sq.SQ_ERR_CUDA), n
        assert call(fresh) == sq.SQ_OK, f"after call {n} failed"
    assert st == sq.SQ_OK and n > 1
