"""Host-side checks of the microscaled 4-bit entry points and the block norms (no
GPU needed): every malformed argument is refused before anything is enqueued,
and the NumPy definitions the GPU tests compare with are themselves pinned.
"""
import numpy as np
import pytest

import w8a8_int8_gemm_channel_b200 as sq
from oracle import mx4
from w8a8_int8_gemm_channel_b200 import _build

A, B, C, D, E = (0x7F0000001000 + 0x1000 * i for i in range(5))  # aligned fake device addresses (never dereferenced)
MIS = 0x7F0000001004
INV, UNS = sq.SQ_ERR_INVALID_ARG, sq.SQ_ERR_UNSUPPORTED
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sq.lib()


def test_quantisers_refuse(lib):
    for f in (lib.sq_mx4_quant_act, lib.sq_mx4_quant_weight):
        assert f(None, 1, 4, 64, B, C, D, None) == INV
        assert f(A, 1, 4, 64, B, None, D, None) == INV
        assert f(A, 1, 4, 64, B, C, None, None) == INV
        assert f(MIS, 1, 4, 64, B, C, D, None) == INV
        assert f(A, 1, 4, 64, MIS, C, D, None) == INV
        assert f(A, 1, 4, 64, None, MIS, D, None) == INV
        assert f(A, 2, 4, 64, B, C, D, None) == INV        # bad dtype
        assert f(A, 1, 0, 64, B, C, D, None) == INV        # no rows
        assert f(A, 1, 4, 48, B, C, D, None) == INV        # K % 32
        assert f(A, 1, 4, 0, B, C, D, None) == INV
        assert f(A, 1, 4, -32, B, C, D, None) == INV
        assert f(A, 1, (1 << 24) + 1, 64, B, C, D, None) == UNS
        assert f(A, 1, 4, 1 << 25, B, C, D, None) == UNS
    f = lib.sq_mx4_dequant
    assert f(None, B, 4, 64, C, 1, None) == INV
    assert f(A, B, 4, 64, None, 1, None) == INV
    assert f(A, B, 4, 40, C, 1, None) == INV
    assert f(A, B, 4, 64, C, 3, None) == INV


def test_gemm_and_linear_refuse(lib):
    f = lib.sq_mx4_gemm
    assert f(A, B, C, D, 0, 64, 64, E, 1, A, BIG, None) == INV       # M = 0
    assert f(A, B, C, D, 4, 40, 64, E, 1, A, BIG, None) == INV       # N % 16
    assert f(A, B, C, D, 4, 64, 80, E, 1, A, BIG, None) == INV       # K % 32
    assert f(A, B, C, D, 4, 64, 64, E, 5, A, BIG, None) == INV       # dtype
    assert f(A, None, C, D, 4, 64, 64, E, 1, A, BIG, None) == INV
    assert f(A, B, C, MIS, 4, 64, 64, E, 1, A, BIG, None) == INV
    assert f(A, B, C, D, 4, 64, 64, E, 1, None, 0, None) == INV      # few tokens need a workspace
    need = lib.sq_mx4_gemm_workspace_size(4, 64, 64)
    assert need > 0 and f(A, B, C, D, 4, 64, 64, E, 1, A, need - 1, None) == INV
    assert f(A, B, C, D, 4, 64, 64, E, 1, MIS, BIG, None) == INV
    assert f(A, B, C, D, 1 << 25, 64, 64, E, 1, A, BIG, None) == UNS
    assert lib.sq_mx4_gemm_workspace_size(129, 64, 64) == 0
    assert lib.sq_mx4_gemm_workspace_size(4, 65, 64) == 0
    g = lib.sq_mx4_linear
    need = lib.sq_mx4_linear_workspace_size(300, 64, 64)
    assert need >= 300 * 32 + lib.sq_mx4_scale_size(300, 64)
    assert g(A, 1, B, C, D, 300, 64, 64, E, 1, A, need - 1, None) == INV
    assert g(A, 1, B, C, D, 300, 64, 64, E, 1, None, need, None) == INV
    assert g(A, 7, B, C, D, 300, 64, 64, E, 1, A, need, None) == INV
    assert g(A, 1, MIS, C, D, 300, 64, 64, E, 1, A, need, None) == INV
    assert g(None, 1, B, C, D, 300, 64, 64, E, 1, A, need, None) == INV


def test_scale_size(lib):
    for rows, K in ((1, 32), (128, 128), (129, 160), (300, 4096)):
        assert lib.sq_mx4_scale_size(rows, K) == mx4.scale_size(rows, K)
    assert lib.sq_mx4_scale_size(0, 32) == 0 and lib.sq_mx4_scale_size(4, 33) == 0


def test_experts_layer_refuses(lib):
    def call(T=4, topk=2, E_=8, H=64, I=64, ptr=A, ws=A, size=BIG, dt=1):
        return lib.sq_mx4_moe(ptr, B, C, D, T, topk, E_, H, I, A, B, C, D, E, A, B, dt, ws, size, None)

    assert call(ptr=None) == INV and call(ptr=MIS) == INV
    assert call(T=0) == INV and call(topk=0) == INV and call(E_=0) == INV
    assert call(H=40) == INV and call(I=16) == INV and call(dt=2) == INV
    assert call(ws=None) == INV and call(ws=MIS) == INV
    assert call(size=lib.sq_mx4_moe_workspace_size(4, 2, 8, 64, 64) - 1) == INV
    assert call(T=129) == UNS and call(T=128, topk=9) == UNS and call(E_=1025) == UNS
    assert call(E_=1024, H=1 << 21) == UNS
    assert lib.sq_mx4_moe_workspace_size(129, 1, 8, 64, 64) == 0


def test_block_norms_refuse(lib):
    for f, step in ((lib.sq_residual_norm_quant, 16), (lib.sq_residual_norm_quant_mx4, 32)):
        def call(b=A, dt=1, M=4, K=64, gamma=B, gate=C, share=1, c=0.5, r=D, r_out=E, g=B, eps=1e-5, q=C, sx=D):
            return f(b, dt, M, K, gamma, gate, share, c, r, r_out, g, eps, q, sx, None)

        assert call(b=None) == INV and call(r=None) == INV and call(r_out=None) == INV and call(g=None) == INV
        assert call(q=None) == INV and call(sx=MIS) == INV and call(gamma=MIS) == INV and call(gate=MIS) == INV
        assert call(dt=4) == INV and call(M=0) == INV and call(K=step + 8) == INV and call(K=0) == INV
        assert call(share=0) == INV
        assert call(c=float("nan")) == INV and call(c=float("inf")) == INV
        assert call(eps=-1e-6) == INV and call(eps=float("nan")) == INV and call(eps=float("inf")) == INV
        assert call(b=A, r_out=A) == INV                   # the block's output is not overwritten
        assert call(K=32768 + 32) == UNS and call(dt=0, K=16384 + 32) == UNS


def test_definition_pins():
    """The block scale and the ties of the NumPy definition, by hand."""
    x = np.zeros((2, 32))
    x[0, :8] = [7.9, -4.0, 5.0, 2.5, -1.75, 0.75, 0.25, 0.2500001]
    x[1, 0] = 2.0 ** -140
    q, s, v = mx4.quantize(x)
    # top 7.9 in [4, 8): scale 1; 7.9 -> 6 (the largest), ties to the even code
    assert v[0, :8].tolist() == [6.0, -4.0, 4.0, 2.0, -2.0, 1.0, 0.0, 0.5]
    assert s[0] == 127 and s[16] == 0  # row 1: below 2^-127 the smallest scale
    assert q[0, 0] == (7 | (14 << 4)) and mx4.decode(q, s)[0, 1] == -4.0
    assert np.array_equal(mx4.decode(q, s), v)
    # a scale below the largest normal one, and the round trip of every code at every scale
    codes = np.arange(16, dtype=np.uint8)
    row = np.repeat(codes, 2)[None, :16] | (np.repeat(codes, 2)[None, 16:] << 4)
    for b in (0, 1, 2, 127, 200, 252):
        t = np.zeros(512, np.uint8)
        t[0] = b
        d = mx4.decode(row, t)
        if b > 0:  # (a block whose top code is 6 keeps its scale: 6 is in [4, 8))
            assert np.array_equal(mx4.quantize(d)[2], d)


def test_python_calls_refuse_wrong_tensors():
    import torch

    x, q, s = torch.zeros(4, 64), torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensors"):
        sq.sq_mx4_quant_act(x, None, q, s)
    with pytest.raises(ValueError):
        sq.sq_mx4_linear(x, None, q, s, torch.zeros(4, 5), s)      # y's shape
    ids, w = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)
    e = torch.zeros(8, 64, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="int32"):
        sq.sq_mx4_moe(q, s, ids, w, e, s, e, s, e, s, x, s)
    with pytest.raises(ValueError, match="scales"):
        sq.sq_mx4_moe(q, s, ids.int(), w, e, s, e, s, e, s, x, s)
    with pytest.raises(ValueError, match="xq"):
        sq.sq_residual_norm_quant(x, None, None, 1, 1.0, x, x, x[0], 0.0, q, s)
    with pytest.raises(ValueError, match="gate"):
        sq.sq_residual_norm_quant_mx4(x, None, x[:1], 2, 1.0, x, x, x[0], 0.0, q, s)
