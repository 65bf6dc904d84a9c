"""The norms around a block (sq_residual_norm_quant and its MXFP4 form) against
their definition, every fp32 operation rounded in 64-bit arithmetic.

The mean squares are fp64 sums in an unspecified order, so 1 / RMS can round
either way at a fp32 midpoint; the inputs here are random, and a test fails if
one of them is that near (2^-40 relative), so all comparisons are bit-exact.
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


def np64(t):
    return t.detach().cpu().double().numpy()


def rinv(v, eps):
    ms = (v * v).sum(1, keepdims=True) / v.shape[1] + float(np.float32(eps))
    with np.errstate(divide="ignore"):
        r = np.where(ms > 0, 1 / np.sqrt(ms), 0.0)
    lo = mx4.f32(r)
    near = np.abs((r - lo) / np.maximum(np.spacing(lo.astype(np.float32)).astype(np.float64), 1e-300))
    assert (np.abs(near - 0.5) > 2.0 ** -16).all(), "a row too near a rounding midpoint: take another seed"
    return lo


def definition(b, gamma, gate, share, c, r, g, eps, dt):
    """(r', a) with each fp32 rounding of the definition."""
    u = np64(b)
    if gamma is not None:
        u = mx4.f32(mx4.f32(u * rinv(u, eps)) * np64(gamma))
    if gate is not None:
        u = mx4.f32(u * np64(gate)[np.arange(len(u)) // share])
    v = mx4.f32(np64(r) + mx4.f32(u * float(np.float32(c))))
    out = torch.from_numpy(v).to(F32).to(dt)
    o = np64(out)
    return out, mx4.f32(mx4.f32(o * rinv(o, eps)) * np64(g))


def int8(a):
    sx = mx4.f32(np.abs(a).max(1) / 127)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(sx[:, None] > 0, np.rint(mx4.f32(a / sx[:, None])), 0)
    return np.clip(q, -127, 127).astype(np.int8), sx.astype(np.float32)


def inputs(M, K, dt, seed, share, post):
    g = torch.Generator().manual_seed(seed)
    b = torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    r = torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g) * 2)
    r[:, torch.randperm(K, generator=g)[: max(1, K // 500)]] *= 60
    if M > 4:
        b[1] = 0
        b[2], r[2] = 0, 0  # a row of zeros
        r[3] *= 1e-30
        b[3] *= 1e-30
    gamma = torch.rand(K, generator=g) + 0.5 if post else None
    gate = None if share is None else torch.randn(-(-M // share), K, generator=g).to(dt)
    return b.to(dt), gamma, gate, r.to(dt), torch.rand(K, generator=g) * 2 + 0.1


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


SHAPES = [(1, 32, 1), (5, 96, 2), (7, 160, 7), (3, 2048, 100), (33, 4096, 1), (9, 4128, None), (6, 8192, 4),
          (1000, 256, 512), (700, 1056, None), (640, 4096, 100), (600, 8192, 600), (5, 16384, 2)]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("M,K,share", SHAPES)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("in_place", [False, True])
def test_both_outputs(M, K, share, post, dt, in_place):
    b, gamma, gate, r, g = inputs(M, K, dt, M + K, share, post)
    eps = 0.0 if M == 7 else 1e-5
    want_r, a = definition(b, gamma, gate, share, 0.8, r, g, eps, dt)
    want_q, want_sx = int8(a)
    want_c, want_tiles, _ = mx4.quantize(a)
    db, dgamma, dgate, dg = cuda(b, gamma, gate, g)
    for form in ("int8", "mx4"):
        dr = r.cuda()
        out = dr if in_place else torch.empty_like(dr)
        if form == "int8":
            q, sx = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
            sq.sq_residual_norm_quant(db, dgamma, dgate, share or 1, 0.8, dr, out, dg, eps, q, sx)
            assert np.array_equal(sx.cpu().numpy(), want_sx) and np.array_equal(q.cpu().numpy(), want_q)
        else:
            q = torch.full((M, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
            sx = torch.full((sq.sq_mx4_scale_size(M, K),), 0xEE, dtype=torch.uint8, device="cuda")
            sq.sq_residual_norm_quant_mx4(db, dgamma, dgate, share or 1, 0.8, dr, out, dg, eps, q, sx)
            assert np.array_equal(sx.cpu().numpy(), want_tiles) and np.array_equal(q.cpu().numpy(), want_c)
        assert torch.equal(out.cpu(), want_r)
        if not in_place:
            assert torch.equal(dr.cpu(), r)


@pytest.mark.parametrize("M,K,dt", [(4, 32768, BF16), (3, 16, F32), (700, 48, BF16), (2, 16384, F32), (650, 16384, BF16)])
def test_longest_and_shortest_rows_int8(M, K, dt):
    b, gamma, gate, r, g = inputs(M, K, dt, K, 3, True)
    want_r, a = definition(b, gamma, gate, 3, -1.5, r, g, 1e-6, dt)
    want_q, want_sx = int8(a)
    q, sx, out = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, K, dtype=dt, device="cuda")
    db, dgamma, dgate, dr, dg = cuda(b, gamma, gate, r, g)
    sq.sq_residual_norm_quant(db, dgamma, dgate, 3, -1.5, dr, out, dg, 1e-6, q, sx)
    assert torch.equal(out.cpu(), want_r)
    assert np.array_equal(sx.cpu().numpy(), want_sx) and np.array_equal(q.cpu().numpy(), want_q)


def test_int8_ties_are_divided():
    """Rows whose quotients lie on half-integers: the reciprocal alone would not decide them."""
    K = 256
    n = torch.arange(K, dtype=torch.float32)
    r = (n % 127 + 0.5) * 2.0 ** -7
    r[-1] = 127 * 2.0 ** -7
    r = torch.stack([r, -r, r * 3, r * 1.1])
    b = torch.zeros_like(r)
    g = torch.ones(K)
    want_r, a = definition(b, None, None, 1, 1.0, r, g, 0.0, F32)
    want_q, want_sx = int8(a)
    q, sx, out = torch.empty(4, K, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda"), torch.empty(4, K, device="cuda")
    sq.sq_residual_norm_quant(b.cuda(), None, None, 1, 1.0, r.cuda(), out, g.cuda(), 0.0, q, sx)
    assert np.array_equal(sx.cpu().numpy(), want_sx) and np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("M,K,dt", [(4, 32768, BF16), (130, 20032, BF16), (3, 32, F32), (700, 96, BF16), (600, 16416, BF16), (650, 16384, F32)])
@pytest.mark.parametrize("post", [True, False])
def test_longest_and_shortest_rows_mx4(M, K, dt, post):
    b, gamma, gate, r, g = inputs(M, K, dt, K + 1, 3, post)
    want_r, a = definition(b, gamma, gate, 3, -1.5, r, g, 1e-6, dt)
    want_q, want_s, _ = mx4.quantize(a)
    q = torch.full((M + 1, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
    sx = torch.full((sq.sq_mx4_scale_size(M, K) + 512,), 0xEE, dtype=torch.uint8, device="cuda")
    out = torch.full((M + 1, K), 7.0, dtype=dt, device="cuda")
    db, dgamma, dgate, dr, dg = cuda(b, gamma, gate, r, g)
    sq.sq_residual_norm_quant_mx4(db, dgamma, dgate, 3, -1.5, dr, out[:M], dg, 1e-6, q[:M], sx[:-512])
    assert torch.equal(out[:M].cpu(), want_r)
    assert np.array_equal(sx[:-512].cpu().numpy(), want_s) and np.array_equal(q[:M].cpu().numpy(), want_q)
    assert (out[M] == 7.0).all() and (q[M] == 0xEE).all() and (sx[-512:] == 0xEE).all()
