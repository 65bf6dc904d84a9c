"""The experts layers that the tests of shared tiles run are shared as those
tests say, by the launch code's own printed plan (on a stand-in for the CUDA
runtime with 148 SMs).
"""
import os
import re
import subprocess
import sys

import pytest
import torch

from tests.test_mx4_shared_gpu import SHAPES, definition, make

CHILD = """
import sys, tempfile
from tests import fake_cuda
A = 0x7F0000001000
with tempfile.TemporaryDirectory() as d:
    lib = fake_cuda.load(d)
    for s in {shapes!r}:
        size = lib.sq_mx4_moe_workspace_size(*s)
        assert size > 0 and lib.sq_mx4_moe(A, A, A, A, *s, A, A, A, A, A, A, A, 1, A, size, None) == 0
"""


def test_shared_as_the_gpu_tests_need():
    out = subprocess.run([sys.executable, "-c", CHILD.format(shapes=list(SHAPES))], env={**os.environ, "SQ_DEBUG_PLAN": "1"},
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))), capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    plans = re.findall(r"sq mx4 moe T=(\d+) topk=(\d+) E=(\d+) H=(\d+) I=(\d+): BNX=(\d+) experts=(\d+) up tiles=(\d+) units=(\d+) "
                       r"ctas=(\d+) down tiles=(\d+) units=(\d+) ctas=(\d+)", out.stderr)
    got, token_tiles = {}, set()
    for p in plans:
        T, topk, E, H, I, bnx, experts, *halves = map(int, p)
        assert experts == min(E, T * topk)
        got[T, topk, E, H, I] = tuple("even" if c % t else c // t for t, _, c in (halves[:3], halves[3:]))
        token_tiles |= {(bnx, h, "even" if isinstance(k, str) else k > 1) for h, k in enumerate(got[T, topk, E, H, I])}
    assert got == SHAPES
    # both halves summed both ways for every token tile (the second half of 32 < T < 65 among them)
    assert {(b, h, k) for b in (32, 64, 128) for h in (0, 1) for k in (True, "even")} <= token_tiles


@pytest.mark.parametrize("shape", [(9, 1, 1, 3104, 160), (33, 2, 6, 288, 416), (100, 4, 8, 288, 416)], ids=str)
def test_the_inputs_are_exact(shape):
    T, topk, E, H, I = shape
    _, values = make(*shape, "cpu")
    y = definition(*values, E, I)
    assert torch.equal(y.float().double(), y) and (y != 0).double().mean() > 0.9
