"""The microscaled 4-bit operators as a model would use them: in a run, captured
and replayed, on several streams, with one workspace after another call, and
past 32-bit offsets.

Every stage is compared with the 64-bit definition on the bytes that the stage
before it left, so no error is carried along.
"""
import numpy as np
import pytest
import torch

import w8a8_int8_gemm_channel_b200 as sq
from oracle import mx4
from tests.test_mx4_gpu import factors, np64, quantised, values
from tests.test_mx4_moe_gpu import definition, make, on_gpu
from tests.test_residual_norm_gpu import definition as norm_definition

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


def empty(*shape, dtype=torch.uint8):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Layer:
    """Two blocks of a feed-forward stack: a linear layer, then an experts layer, a norm before each and after."""

    def __init__(self, T, H, seed):
        self.T, self.H = T, H
        self.w = quantised(H, H, seed, 0.02)
        self.case = make(T, 2, 4, H, 96, seed + 1)
        g = torch.Generator().manual_seed(seed)
        self.gamma, self.g = torch.rand(H, generator=g) + 0.5, torch.rand(H, generator=g) + 0.5
        self.gate = torch.randn(1, H, generator=g).to(BF16)
        self.dev = [t.cuda() for t in (self.gamma, self.g, self.gate)]
        self.block, self.res = (values(T, H, seed + i, BF16).cuda() for i in (2, 3))
        self.r1, self.r2 = empty(T, H, dtype=BF16), empty(T, H, dtype=BF16)
        self.codes = [(empty(T, H // 2), empty(sq.sq_mx4_scale_size(T, H))) for _ in range(2)]
        self.y1, self.y2 = empty(T, H, dtype=BF16), empty(T, H, dtype=BF16)
        self.moe = on_gpu(*self.case)
        self.ws = empty(max(sq.sq_mx4_gemm_workspace_size(T, H, H), sq.sq_mx4_moe_workspace_size(T, 2, 4, H, 96)))

    def run(self, stream=None):
        gamma, g, gate = self.dev
        sq.sq_residual_norm_quant_mx4(self.block, gamma, gate, self.T, 0.5, self.res, self.r1, g, 1e-5, *self.codes[0], stream=stream)
        sq.sq_mx4_gemm(*self.codes[0], *self.w[:2], self.y1, self.ws, stream)
        sq.sq_residual_norm_quant_mx4(self.y1, gamma, None, 1, 1.0, self.r1, self.r2, g, 1e-5, *self.codes[1], stream=stream)
        sq.sq_mx4_moe(*self.codes[1], *self.moe[2:], self.y2, self.ws, stream)

    def outputs(self):
        return [t.clone() for t in (self.r1, self.y1, self.r2, self.y2, *self.codes[0], *self.codes[1])]

    def check(self):
        norms = ((self.block, self.gate, 0.5, self.res, self.r1, self.codes[0]), (self.y1, None, 1.0, self.r1, self.r2, self.codes[1]))
        for b, gate, c, r, out, (q, sc) in norms:
            want_r, a = norm_definition(b.cpu(), self.gamma, gate, self.T, c, r.cpu(), self.g, 1e-5, BF16)
            want_q, want_s, _ = mx4.quantize(a)
            assert torch.equal(out.cpu(), want_r)
            assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(sc.cpu().numpy(), want_s)
        x = mx4.decode(*(t.cpu().numpy() for t in self.codes[0]))
        want, mags = mx4.product(x, self.w[2])
        assert (np.abs(np64(self.y1) - want) <= mx4.product_bound(self.H, mags, want, torch.finfo(BF16).eps)).all()
        q, sc = (t.cpu().numpy() for t in self.codes[1])
        want, bound = definition((q, sc, mx4.decode(q, sc)), *self.case[1:], torch.finfo(BF16).eps)
        assert (np.abs(np64(self.y2) - want) <= bound).all()


@pytest.mark.parametrize("T,H", [(1, 256), (7, 544), (40, 288), (100, 256)])
def test_a_run_of_them(T, H):
    layer = Layer(T, H, T)
    layer.run()
    layer.check()


@pytest.mark.parametrize("T", [3, 40])
def test_captured_and_replayed(T):
    """A captured run gives the eager run's bits, again and again, on the first call's workspace and on new inputs; two
    graphs take turns on one workspace."""
    a, b = Layer(T, 288, 11), Layer(T, 544, 12)
    for layer in (a, b):
        layer.run()
    torch.cuda.synchronize()
    eager = [a.outputs(), b.outputs()]
    size = max(a.ws.numel(), b.ws.numel())
    a.ws = b.ws = torch.randint(0, 256, (size,), dtype=torch.uint8, device="cuda")  # a workspace that never was one
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for layer in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            layer.run()
        graphs.append(g)
    for _ in range(3):
        for layer, g, want in zip((a, b), graphs, eager):
            layer.y1.fill_(0)
            layer.y2.fill_(0)
            g.replay()
            torch.cuda.synchronize()
            for x, y in zip(layer.outputs(), want):
                assert torch.equal(x, y)
    a.block.copy_(values(T, 288, 99, BF16))
    graphs[0].replay()
    torch.cuda.synchronize()
    a.check()


def test_streams_side_by_side():
    """Runs on two streams with workspaces of their own, and a stream given by hand."""
    layers = [Layer(5, 288, 21), Layer(33, 544, 22)]
    for layer in layers:
        layer.run()
    torch.cuda.synchronize()
    want = [layer.outputs() for layer in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    for layer, s in zip(layers, streams):
        for t in (layer.y1, layer.y2, layer.r1, layer.r2):
            t.fill_(0)
        s.wait_stream(torch.cuda.current_stream())
    for i in range(20):
        for layer, s in zip(layers, streams):
            if i % 2:
                layer.run(stream=s)
            else:
                with torch.cuda.stream(s):
                    layer.run()
    torch.cuda.synchronize()
    for layer, w in zip(layers, want):
        for x, y in zip(layer.outputs(), w):
            assert torch.equal(x, y)


def test_calls_back_to_back_on_one_workspace():
    """Products of different sizes and the linear layer share a workspace, one call after another, unsynchronised."""
    shapes = [(1, 1040, 4096), (64, 272, 1056), (17, 4096, 512), (200, 528, 288), (2, 144, 16384)]
    cases = [(quantised(M, K, M), quantised(N, K, N, 0.02)) for M, N, K in shapes]
    ws = empty(max(sq.sq_mx4_gemm_workspace_size(*s) for s in shapes))
    ws.fill_(0x5A)
    ys = [[empty(M, N, dtype=F32) for M, N, K in shapes] for _ in range(3)]
    for round_ in ys:
        for (x, w), y in zip(cases, round_):
            sq.sq_mx4_gemm(*x[:2], *w[:2], y, ws)
    for (M, N, K), (x, w), first, *again in zip(shapes, cases, *ys):
        want, mags = mx4.product(x[2], w[2])
        assert (np.abs(np64(first) - want) <= mx4.product_bound(K, mags, want, 2.0 ** -23)).all()
        assert all(torch.equal(first, y) for y in again)


def test_conveniences_allocate_and_stack():
    torch.manual_seed(0)
    w, x, s = torch.randn(3, 64, 96, device="cuda") * 0.02, torch.randn(5, 96, device="cuda"), factors(96, 1).cuda()
    wq, sw = sq.mx4_prepare_weight(w, s)
    for i in range(3):
        q, t, v = mx4.quantize(mx4.smooth_weight(np64(w[i]), np64(s)))
        assert np.array_equal(wq[i].cpu().numpy(), q) and np.array_equal(sw[i].cpu().numpy(), t)
        y = sq.mx4_linear(x, s, wq[i], sw[i], out_dtype=F32)
        want, mags = mx4.product(mx4.quantize(mx4.smooth_act(np64(x), np64(s)))[2], v)
        assert (np.abs(np64(y) - want) <= mx4.product_bound(96, mags, want, 2.0 ** -23)).all()
    down, sd = sq.mx4_prepare_weight(torch.randn(3, 96, 64, device="cuda"))
    xq, sx = sq.mx4_quantize(x, s)
    ids = torch.tensor([[0, 1], [1, 2], [2, 0], [-1, 1], [0, 0]], dtype=torch.int32, device="cuda")
    y = sq.mx4_moe(xq, sx, ids, torch.ones(5, 2, device="cuda"), wq, sw, wq, sw, down, sd)
    assert y.shape == (5, 96) and y.dtype == BF16 and torch.isfinite(y).all()


def test_offsets_past_32_bits():
    """A matrix of 2.6e9 values: its last rows come out like the same rows quantised alone."""
    rows, K = 40000, 65536
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    x = torch.empty(rows, K, dtype=BF16, device="cuda")
    tail = torch.randn(64, K, device="cuda").to(BF16)
    x[:-64] = 1.0
    x[-64:] = tail
    q, sc = sq.mx4_quantize(x)
    alone_q, _ = sq.mx4_quantize(tail)
    assert torch.equal(q[-64:], alone_q)
    out = x  # the values, in place of the input
    sq.sq_mx4_dequant(q, sc, out)
    want = torch.empty(64, K, dtype=BF16, device="cuda")
    sq.sq_mx4_dequant(alone_q, sq.mx4_quantize(tail)[1], want)
    assert torch.equal(out[-64:], want) and (out[:3] == 1.0).all() and (out[-67:-64] == 1.0).all()
    # two rows of it through a product: the weight's rows lie past 2^31 codes
    y = sq.mx4_linear(tail[:2].contiguous(), None, q, sc, out_dtype=F32)
    v = np64(want)
    exact, mags = mx4.product(v[:2], v)
    assert (np.abs(np64(y[:, -64:]) - exact) <= mx4.product_bound(K, mags, exact, 2.0 ** -23)).all()
