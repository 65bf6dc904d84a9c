"""What a call allocates for itself when it is given a stream: workspaces and
outputs have to belong to that stream.  A block of the current stream may still be
written there by earlier work, and goes to later work there as soon as the call
drops it, while the kernels on the given stream use it.

On the CPU a fake torch and a fake library note where each tensor is allocated
and where each entry point is launched; on the GPU the given stream is held back
while the current one allocates and writes.
"""
import contextlib
import threading
import types

import numpy as np
import pytest
import torch

import w8a8_int8_gemm_channel_b200 as sq

CURRENT, OTHER = 0x100, 0x200  # stream handles of the fake


class FakeTensor:
    is_cuda, device = True, "cuda:0"

    def __init__(self, shape, dtype):
        self.shape, self.dtype = torch.Size(shape), dtype

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def reshape(self, *shape):
        return FakeTensor(torch.empty(self.shape, device="meta").reshape(*shape).shape, self.dtype)

    def __iter__(self):
        return (FakeTensor(self.shape[1:], self.dtype) for _ in range(self.shape[0]))

    get_device = lambda self: 0  # noqa: E731
    is_contiguous = lambda self: True  # noqa: E731
    data_ptr = lambda self: 0x1000  # noqa: E731


class FakeStream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class Fakes:
    """torch and the library as far as the binding uses them, with a log of (what, stream)."""

    def __init__(self):
        self.log, self.at = [], CURRENT
        cuda = types.SimpleNamespace(
            stream=self.stream, ExternalStream=FakeStream, current_device=lambda: 0,
            current_stream=lambda d=None: FakeStream(self.at), default_stream=lambda d=None: FakeStream(0))
        make = lambda *shape, dtype, device=None: self.make(shape, dtype)  # noqa: E731
        self.torch = types.SimpleNamespace(
            uint8=torch.uint8, int8=torch.int8, int32=torch.int32, float32=torch.float32, bfloat16=torch.bfloat16,
            float64=torch.float64, cuda=cuda, _C=object(), empty=make, zeros=make,
            empty_like=lambda t: self.make(t.shape, t.dtype))

    @contextlib.contextmanager
    def stream(self, s):
        before, self.at = self.at, s.cuda_stream
        yield
        self.at = before

    def make(self, shape, dtype):
        self.log.append(("empty", self.at))
        return FakeTensor(shape[0] if isinstance(shape[0], torch.Size) else shape, dtype)

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 4096 if "scale" not in name else -(-a[0] // 128) * -(-a[1] // 128) * 512

        def entry(*args):
            self.log.append((name, args[-1]))
            return 0

        return entry


def t(*shape, dtype=torch.bfloat16):
    return FakeTensor(shape, dtype)


U8, I8, F32, F64 = torch.uint8, torch.int8, torch.float32, torch.float64


def mx4(rows, K):
    return t(rows, K // 2, dtype=U8), t(512, dtype=U8)


def experts():
    return [t(*s, dtype=U8) for s in ((3, 64, 32), (3, 512), (3, 64, 32), (3, 512), (3, 64, 32), (3, 512))]


IDS = t(4, 2, dtype=torch.int32), t(4, 2, dtype=F32)
CALLS = {
    "sq_mx4_gemm": lambda **k: sq.sq_mx4_gemm(*mx4(4, 64), *mx4(64, 64), t(4, 64), **k),
    "sq_mx4_linear": lambda **k: sq.sq_mx4_linear(t(4, 64), None, *mx4(64, 64), t(4, 64), **k),
    "sq_mx4_moe": lambda **k: sq.sq_mx4_moe(*mx4(4, 64), *IDS, *experts(), t(4, 64), **k),
    "sq_w8a8_gemm_ws": lambda **k: sq.sq_w8a8_gemm_ws(t(4, 64, dtype=I8), t(4, dtype=F32), t(64, 64, dtype=I8), t(64, dtype=F32), t(4, 64), **k),
    "sq_gptq_factor": lambda **k: sq.sq_gptq_factor(t(64, 64, dtype=F64), t(64, 64, dtype=F64), **k),
    "mx4_quantize": lambda **k: sq.mx4_quantize(t(4, 64), **k),
    "mx4_prepare_weight": lambda **k: sq.mx4_prepare_weight(t(3, 64, 64), **k),
    "mx4_linear": lambda **k: sq.mx4_linear(t(4, 64), None, *mx4(64, 64), **k),
    "mx4_moe": lambda **k: sq.mx4_moe(*mx4(4, 64), *IDS, *experts(), **k),
    "calibrate": lambda **k: sq.calibrate(t(4, 64), **k),
    "prepare_weight": lambda **k: sq.prepare_weight(t(64, dtype=F32), t(64, 64), 0.5, **k),
    "linear": lambda **k: sq.linear(t(4, 64), t(64, dtype=F32), t(64, 64, dtype=I8), t(64, dtype=F32), **k),
    "gptq_weight": lambda **k: sq.gptq_weight(t(4, 64), t(64, 64), t(64, dtype=F32), **k),
}


@pytest.mark.parametrize("given", ["none", "stream", "handle", "default"])
@pytest.mark.parametrize("name", CALLS)
def test_allocations_are_on_the_stream_of_the_launch(name, given, monkeypatch):
    fakes = Fakes()
    monkeypatch.setattr(sq, "_torch", lambda: fakes.torch)
    monkeypatch.setattr(sq, "lib", lambda: fakes)
    monkeypatch.setattr(sq, "_lib", fakes)
    monkeypatch.setattr(sq, "_codes_of", {})
    want = {"none": CURRENT, "stream": OTHER, "handle": OTHER, "default": 0}[given]
    CALLS[name](**{"none": {}, "stream": {"stream": FakeStream(OTHER)}, "handle": {"stream": OTHER}, "default": {"stream": 0}}[given])
    whats = [w for w, _ in fakes.log]
    assert "empty" in whats and any(w.startswith("sq_") for w in whats)
    assert [s for _, s in fakes.log] == [want] * len(fakes.log), fakes.log
    assert fakes.at == CURRENT


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w8a8_int8_gemm_channel_b200 import _build

    _build.build()
    yield
    assert sq.sq_device_status() == (sq.SQ_OK, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("as_handle", [False, True])
def test_the_current_stream_allocates_and_writes_meanwhile(gpu, as_handle):
    T, H, I, E = 20, 544, 416, 6
    g = torch.Generator().manual_seed(1)
    r = lambda *shape: (torch.randn(*shape, generator=g) * 0.1).cuda()  # noqa: E731
    weights = [x for shape in ((E, I, H), (E, I, H), (E, H, I)) for x in sq.mx4_prepare_weight(r(*shape))]
    wq, sw = sq.mx4_prepare_weight(r(1040, H))
    x = r(T, H)
    ids = torch.from_numpy(np.stack([np.random.default_rng(i).permutation(E)[:2] for i in range(T)]).astype(np.int32)).cuda()
    share = torch.rand(T, 2, generator=g).cuda()

    def calls(**k):
        xq, sx = sq.mx4_quantize(x, **k)
        return sq.mx4_linear(x, None, wq, sw, **k), sq.mx4_moe(xq, sx, ids, share, *weights, out_dtype=F32, **k)

    want = [y.clone() for y in calls()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sizes = [sq.sq_mx4_linear_workspace_size(T, 1040, H), sq.sq_mx4_moe_workspace_size(T, 2, E, H, I), T * 1040 * 4, T * H * 4]
    for _ in range(3):
        # blocks whose last writes on the current stream are still to come when they are dropped
        early = [torch.empty(n, dtype=U8, device="cuda") for n in sizes]
        torch.cuda._sleep(20_000_000)
        for b in early:
            b.fill_(0xC3)
        del early, b
        with torch.cuda.stream(side):
            torch.cuda._sleep(10_000_000)
        ys = calls(stream=side.cuda_stream if as_handle else side)
        # blocks the current stream takes while the calls wait
        late = [torch.full((n,), 0x3C, dtype=U8, device="cuda") for n in sizes for _ in range(2)]
        torch.cuda.synchronize()
        for y, w in zip(ys, want):
            assert torch.equal(y, w)
        for b in late:
            assert (b == 0x3C).all()


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
def test_calls_that_allocate_are_captured(gpu, given):
    """Workspaces and outputs made during a capture belong to the graph; replays give the eager bits."""
    T, H, I, E = 17, 288, 160, 4
    g = torch.Generator().manual_seed(2)
    r = lambda *shape: (torch.randn(*shape, generator=g) * 0.1).cuda()  # noqa: E731
    weights = [x for shape in ((E, I, H), (E, I, H), (E, H, I)) for x in sq.mx4_prepare_weight(r(*shape))]
    wq, sw = sq.mx4_prepare_weight(r(1040, H))
    ids = (torch.arange(2 * T, device="cuda").reshape(T, 2) % E).to(torch.int32)
    share, x = torch.rand(T, 2, generator=g).cuda(), r(T, H)

    def calls(**k):
        xq, sx = sq.mx4_quantize(x, **k)
        return sq.mx4_linear(x, None, wq, sw, **k), sq.mx4_moe(xq, sx, ids, share, *weights, out_dtype=F32, **k)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ys = calls(stream=side) if given else calls()
    for seed in range(3):
        x.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(seed)))
        for y in ys:
            y.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        for y, want in zip(ys, calls()):
            assert torch.equal(y, want)


@pytest.mark.gpu
def test_host_threads_side_by_side(gpu):
    """Threads on streams of their own, each with first calls of other shapes, and without workspaces of theirs."""
    shapes = [(3, 544, 160), (40, 288, 416), (100, 256, 96), (1, 1056, 288)]

    def work(T, H, I, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *shape: (torch.randn(*shape, generator=g) * 0.1).cuda()  # noqa: E731
        weights = [x for shape in ((5, I, H), (5, I, H), (5, H, I)) for x in sq.mx4_prepare_weight(r(*shape))]
        wq, sw = sq.mx4_prepare_weight(r(528, H))
        x, ids, share = r(T, H), (torch.arange(2 * T).reshape(T, 2) % 5).to(torch.int32).cuda(), torch.rand(T, 2, generator=g).cuda()
        ys = []
        for _ in range(30):
            xq, sx = sq.mx4_quantize(x)
            ys.append((sq.mx4_linear(x, None, wq, sw), sq.mx4_moe(xq, sx, ids, share, *weights, out_dtype=F32)))
        torch.cuda.current_stream().synchronize()
        return ys

    out = [None] * len(shapes)

    def thread(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            out[i] = work(*shapes[i], i)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(len(shapes))]
    for t_ in threads:
        t_.start()
    for t_ in threads:
        t_.join()
    for i, shape in enumerate(shapes):
        want = work(*shape, i)[0]
        assert out[i] is not None
        for ys in out[i]:
            assert all(torch.equal(y, w) for y, w in zip(ys, want))
