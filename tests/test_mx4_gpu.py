"""The microscaled 4-bit (MXFP4) quantiser, read-back and products against the
plain 64-bit definitions in oracle/mx4.py.

Codes and scales are bit-exact.  A product is fp32-accumulated: it may be off by
K 2^-23 of the sum of magnitudes (one unit in the last place an addition) and
half a step of the output type, fp32 2^-24 and bf16 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import w8a8_int8_gemm_channel_b200 as sq
from oracle import mx4

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w8a8_int8_gemm_channel_b200 import _build

    _build.build()
    yield
    st, code = sq.sq_device_status()
    assert st == sq.SQ_OK, f"device error word {code:#x}"


def values(rows, K, seed, dtype=F32, scale=1.0):
    """Values with far channels, quiet blocks, zero blocks and exact ties."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g) * scale
    x[:, torch.randperm(K, generator=g)[: max(1, K // 200)]] *= 60.0
    x[rows // 2, :32] = 0.0
    x[rows // 3, -32:] *= 1e-30
    if rows > 2:
        tie = torch.tensor([0.25, -0.75, 1.25, -1.75, 2.5, -3.5, 5.0, 7.5] * 4) * scale
        x[2, :32] = tie
    return x.to(dtype)


def factors(K, seed):
    return torch.rand(K, generator=torch.Generator().manual_seed(seed)) * 3 + 0.3


def np64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def poisoned(*shape):
    return torch.full(shape, 0xEE, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (5, 96), (33, 160), (128, 128), (129, 256), (200, 4096), (1000, 2336), (7, 16384)])
@pytest.mark.parametrize("side", ["act", "weight", "plain"])
def test_quantise_and_read_back(rows, K, dtype, side):
    x = values(rows, K, rows + K, dtype)
    s = None if side == "plain" else factors(K, K)
    v = mx4.smooth_weight(np64(x), np64(s)) if side == "weight" else mx4.smooth_act(np64(x), np64(s))
    want_q, want_s, want_v = mx4.quantize(v)
    q, sc = poisoned(rows, K // 2), poisoned(sq.sq_mx4_scale_size(rows, K))
    (sq.sq_mx4_quant_weight if side == "weight" else sq.sq_mx4_quant_act)(
        x.cuda(), None if s is None else s.cuda(), q, sc)
    assert np.array_equal(sc.cpu().numpy(), want_s)  # the padding too
    assert np.array_equal(q.cpu().numpy(), want_q)
    for out_dtype in (F32, BF16):
        out = torch.empty(rows, K, dtype=out_dtype, device="cuda")
        sq.sq_mx4_dequant(q, sc, out)
        assert np.array_equal(np64(out), want_v)


def test_quantise_special_values():
    x = torch.zeros(6, 64)
    x[0, 3] = float("nan")
    x[1, 40] = float("inf")
    x[2, 0] = -float("inf")
    x[3, :32] = 3.0e38
    x[3, 32:] = torch.finfo(F32).tiny * 2.0 ** -10  # subnormal
    x[4, :32] = torch.finfo(F32).tiny
    x[5, 31] = -0.0
    q, sc, v = mx4.quantize(np64(x))
    gq, gs = sq.mx4_quantize(x.cuda())
    assert np.array_equal(gs.cpu().numpy(), sc) and np.array_equal(gq.cpu().numpy(), q)
    out = torch.empty(6, 64, device="cuda")
    sq.sq_mx4_dequant(gq, gs, out)
    assert np.array_equal(np64(out), v, equal_nan=True)


def quantised(rows, K, seed, scale=1.0):
    q, sc, v = mx4.quantize(np64(values(rows, K, seed, F32, scale)))
    return torch.from_numpy(q).cuda(), torch.from_numpy(sc).cuda(), v


def check_product(y, xv, wv, K):
    want, mags = mx4.product(xv, wv)
    bound = mx4.product_bound(K, mags, want, torch.finfo(y.dtype).eps)
    off = np.abs(np64(y) - want)
    assert np.isfinite(np64(y)).all()
    assert (off <= bound).all(), f"off by {(off / np.maximum(bound, 1e-300)).max():.3g} times the bound"


FEW = [(1, 16, 32), (1, 128, 256), (2, 272, 96), (8, 1040, 2336), (17, 4096, 512), (32, 640, 4096), (33, 400, 1056),
       (64, 2048, 1024), (65, 528, 288), (128, 1040, 4128), (1, 20000, 288), (128, 40000, 64), (5, 144, 16384)]
MANY = [(129, 16, 32), (256, 192, 256), (300, 208, 96), (257, 1040, 2336), (512, 512, 1024), (1000, 400, 288),
        (2048, 1536, 512), (700, 2064, 160)]


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N,K", FEW + MANY)
def test_product(M, N, K, out):
    xq, sx, xv = quantised(M, K, M + K)
    wq, sw, wv = quantised(N, K, N + K + 1, 0.02)
    y = torch.full((M + 1, N), 7.0, dtype=out, device="cuda")  # a row behind the last: left as it was
    sq.sq_mx4_gemm(xq, sx, wq, sw, y[:M])
    torch.cuda.synchronize()
    assert sq.sq_device_status() == (sq.SQ_OK, 0)
    check_product(y[:M], xv, wv, K)
    assert (y[M] == 7.0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [(1, 1040, 4096), (31, 272, 2336), (100, 640, 1056), (203, 1040, 2336), (1024, 512, 512)])
def test_linear(M, N, K, dtype):
    x, s = values(M, K, M, dtype), factors(K, 5)
    wq, sw, wv = quantised(N, K, N, 0.02)
    _, _, xv = mx4.quantize(mx4.smooth_act(np64(x), np64(s)))
    ws = torch.full((sq.sq_mx4_linear_workspace_size(M, N, K),), 0xAB, dtype=torch.uint8, device="cuda")
    y = torch.empty(M, N, dtype=dtype, device="cuda")
    for _ in range(3):  # the same workspace again: nothing of a call is left for the next
        sq.sq_mx4_linear(x.cuda(), s.cuda(), wq, sw, y, ws)
        check_product(y, xv, wv, K)
    first = y.clone()
    sq.sq_mx4_linear(x.cuda(), s.cuda(), wq, sw, y, ws)
    assert torch.equal(first, y)


@pytest.mark.parametrize("M", [5, 40, 300])
def test_nan_blocks_spoil_their_row_and_column_alone(M):
    N, K = 272, 416
    x, w = values(M, K, M), values(N, K, N, F32, 0.02)
    clean = [sq.mx4_quantize(x.cuda()), sq.mx4_prepare_weight(w.cuda())]
    x[3, 64] = float("nan")
    w[9, 400] = float("inf")
    dirty = [sq.mx4_quantize(x.cuda()), sq.mx4_prepare_weight(w.cuda())]
    a, b = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    sq.sq_mx4_gemm(*clean[0], *clean[1], a)
    sq.sq_mx4_gemm(*dirty[0], *dirty[1], b)
    assert torch.isnan(b[3]).all() and torch.isnan(b[:, 9]).all()
    rows, cols = [i for i in range(M) if i != 3], [j for j in range(N) if j != 9]
    assert torch.equal(a[rows][:, cols], b[rows][:, cols])
