"""The experts layer for few tokens on MXFP4 weights (sq_mx4_moe) against its
definition in 64 bits, with tolerances from arithmetic.

The quantised h between the two halves is the one step that is not continuous:
a value of h that the fp32 product puts on the other side of a rounding border
gives another code.  The gate and up products are off by at most
K 2^-23 of their sums of magnitudes (oracle/mx4.py), so h by a known amount d;
a code can differ only where a border lies within d, and then by one step (a
sixth of the block's top binade or less is excluded: the step above 4 is 2
units).  The bound on y is the sum of those steps over the down product, plus
the product's own rounding.
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


def make(T, topk, E, H, I, seed):
    rng = np.random.default_rng(seed)
    x = mx4.quantize(rng.standard_normal((T, H)) * np.where(rng.random(H) < 0.01, 30.0, 1.0))
    w = {k: [mx4.quantize(rng.standard_normal(shape) * 0.05) for _ in range(E)]
         for k, shape in (("g", (I, H)), ("u", (I, H)), ("d", (H, I)))}
    ids = np.stack([rng.permutation(E)[:topk] if topk <= E else rng.integers(0, E, topk) for _ in range(T)]).astype(np.int32)
    return x, w, ids, rng.random((T, topk)).astype(np.float32)


def silu(v):
    return v / (1 + np.exp(-v))


def definition(x, w, ids, weights, out_eps):
    """(y, bound) of the layer in 64 bits."""
    T, topk = ids.shape
    H, I = x[2].shape[1], w["g"][0][2].shape[0]
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    for e in sorted(set(ids[(ids >= 0) & (ids < len(w["g"]))].tolist())):
        rows = np.flatnonzero((ids == e).any(1))
        v = np.where(ids[rows] == e, weights[rows].astype(np.float64), 0.0).sum(1)[:, None]
        xv = x[2][rows]
        (g, gm), (u, um) = mx4.product(xv, w["g"][e][2]), mx4.product(xv, w["u"][e][2])
        dg, du = mx4.product_bound(H, gm, g, 0.0), mx4.product_bound(H, um, u, 0.0)
        h = silu(g) * u
        # |silu'| <= 1.1; e^x, the division and the products round by a few 2^-24
        dh = 1.1 * dg * np.abs(u) + np.abs(silu(g)) * du + 1.1 * dg * du + 2.0 ** -21 * np.abs(h)
        _, _, hv = mx4.quantize(h)
        lo, hi = mx4.quantize(np.abs(h) - np.minimum(dh, np.abs(h)))[2], mx4.quantize(np.abs(h) + dh)[2]
        # a block whose top crosses a power of two may take the scale next to it: its codes move by a step of that scale
        top, dt = np.abs(h).reshape(len(rows), -1, 32).max(-1), dh.reshape(len(rows), -1, 32).max(-1)
        crosses = np.frexp(top - np.minimum(dt, top * 0.5))[1] != np.frexp(top + dt)[1]
        step = np.maximum(np.abs(hi - np.abs(hv)), np.abs(lo - np.abs(hv)))
        step = np.where(np.repeat(crosses, 32, 1), np.abs(h) * 0.5 + np.repeat(top, 32, 1) / 4, step)
        out, om = mx4.product(hv, w["d"][e][2])
        y[rows] += v * out
        wd = np.abs(w["d"][e][2]).T
        bound[rows] += np.abs(v) * (step @ wd + mx4.product_bound(I, om + step @ wd, out, 0.0)) + 2.0 ** -22 * topk * np.abs(v * out)
    return y, bound + out_eps / 2 * np.abs(y) + 2.0 ** -126


def on_gpu(x, w, ids, weights):
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    t = [cuda(x[0]), cuda(x[1]), cuda(ids), cuda(weights)]
    for k in ("g", "u", "d"):
        t += [cuda(np.stack([q[0] for q in w[k]])), cuda(np.stack([q[1] for q in w[k]]))]
    return t


def check(y, want, bound):
    off = np.abs(y.double().cpu().numpy() - want)
    assert np.isfinite(y.double().cpu().numpy()).all()
    assert (off <= bound).all(), f"off by {(off / bound).max():.3g} times the bound"


@pytest.mark.parametrize("T,topk,E,H,I", [(1, 1, 1, 32, 32), (1, 2, 8, 256, 128), (3, 2, 4, 96, 160), (17, 4, 16, 544, 416),
                                          (33, 2, 6, 288, 96), (64, 6, 32, 512, 288), (65, 3, 5, 160, 640),
                                          (128, 8, 40, 256, 224), (128, 1, 3, 1056, 64), (5, 8, 4, 128, 96), (2, 2, 64, 2048, 1408)])
@pytest.mark.parametrize("out", [F32, BF16])
def test_layer(T, topk, E, H, I, out):
    case = make(T, topk, E, H, I, T + H)
    want, bound = definition(*case, torch.finfo(out).eps)
    t = on_gpu(*case)
    ws = torch.full((sq.sq_mx4_moe_workspace_size(T, topk, E, H, I),), 0xFF, dtype=torch.uint8, device="cuda")
    y = torch.full((T + 1, H), 9.0, dtype=out, device="cuda")
    for _ in range(2):
        sq.sq_mx4_moe(*t, y[:T], ws)
        check(y[:T], want, bound)
    assert (y[T] == 9.0).all()
    first = y.clone()
    ws.fill_(0x7F)
    sq.sq_mx4_moe(*t, y[:T], ws)
    assert torch.equal(first, y)  # nothing hangs on the workspace's contents


def test_choices_that_name_no_expert():
    """-1, E and far values count for nothing; a token without any expert gets zeros; all tokens so: all zeros."""
    T, topk, E, H, I = 9, 3, 6, 256, 160
    x, w, ids, weights = make(T, topk, E, H, I, 3)
    ids[0] = -1
    ids[1] = [E, 2 ** 31 - 1, -(2 ** 31)]
    ids[2, 1] = -1
    want, bound = definition(x, w, ids, weights, torch.finfo(F32).eps)
    y = torch.empty(T, H, device="cuda")
    sq.sq_mx4_moe(*on_gpu(x, w, ids, weights), y)
    check(y, want, bound)
    assert (y[:2] == 0).all()
    for out in (F32, BF16):
        y = torch.full((T, H), 5.0, dtype=out, device="cuda")
        sq.sq_mx4_moe(*on_gpu(x, w, np.full_like(ids, -1), weights), y)
        assert (y == 0).all()


def test_one_expert_twice_and_for_all():
    T, topk, E, H, I = 40, 4, 7, 160, 96
    x, w, ids, weights = make(T, topk, E, H, I, 4)
    ids[:] = 5
    ids[3] = [2, 5, 2, 2]
    want, bound = definition(x, w, ids, weights, torch.finfo(F32).eps)
    y = torch.empty(T, H, device="cuda")
    sq.sq_mx4_moe(*on_gpu(x, w, ids, weights), y)
    check(y, want, bound)


def test_a_token_with_nan_spoils_itself_alone():
    T, topk, E, H, I = 6, 2, 4, 128, 128
    x, w, ids, weights = make(T, topk, E, H, I, 5)
    t = on_gpu(x, w, ids, weights)
    y, z = torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda")
    sq.sq_mx4_moe(*t, y)
    sx = x[1].copy()
    sx[mx4.tile_index(T, H)[2, 1]] = 255
    t[1] = torch.from_numpy(sx).cuda()
    sq.sq_mx4_moe(*t, z)
    assert torch.isnan(z[2]).all()
    keep = [i for i in range(T) if i != 2]
    assert torch.equal(y[keep], z[keep])


@pytest.mark.parametrize("below", [0, 1, 2, 3, 70000])
def test_workspace_contents_around_the_counts_tag(below):
    """A workspace of words that a few adds turn into tagged ones (and of what a finished call leaves, 0 below)."""
    T, topk, E, H, I = 2, 2, 64, 2048, 1408  # three CTAs a tile of the first half
    g = torch.Generator(device="cuda").manual_seed(6)

    def matrix(*shape):  # any codes, every scale 1/16
        return [torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, dtype=torch.uint8, device="cuda"),
                torch.full((*shape[:-2], sq.sq_mx4_scale_size(*shape[-2:])), 123, dtype=torch.uint8, device="cuda")]

    ids = torch.tensor([[3, 60], [17, 41]], dtype=torch.int32, device="cuda")
    t = [*matrix(T, H), ids, torch.rand(T, topk, generator=g, device="cuda"), *matrix(E, I, H), *matrix(E, I, H), *matrix(E, H, I)]
    n = sq.sq_mx4_moe_workspace_size(T, topk, E, H, I)
    y = [torch.empty(T, H, device="cuda") for _ in range(2)]
    sq.sq_mx4_moe(*t, y[0], torch.zeros(n, dtype=torch.uint8, device="cuda"))
    assert torch.isfinite(y[0]).all() and (y[0] != 0).any()
    tag = (0x9E3779B97F4A << 16) - below
    ws = torch.full((n // 8,), tag - (1 << 64), dtype=torch.int64, device="cuda").view(torch.uint8)
    assert ws.numel() == n
    for _ in range(2):
        sq.sq_mx4_moe(*t, y[1], ws)
        assert torch.equal(*y)


def digits(v, n):
    """Integers [rows] as E2M1 codes [rows, 32 n]: a hexadecimal digit in each block of 32, the lowest first."""
    out = np.zeros((len(v), 32 * n), np.uint8)
    for row, x in enumerate(v):
        for i in range(n):
            d, at = (int(x) >> 4 * i) & 15, 32 * i
            while d:
                part = max(p for p in (6, 4, 3, 2, 1) if p <= d)
                out[row, at] = {1: 2, 2: 4, 3: 5, 4: 6, 6: 7}[part]
                d, at = d - part, at + 1
    return out


def near_borders(count, low, high):
    """(a, p, b, q, border, above): gate values a 2^p and up values b 2^q whose h = silu(gate) up lies between low and
    high steps of 2^-24 from a border between two E2M1 values."""
    rng = np.random.default_rng(12)
    a = np.arange(2048, 4096)
    exps = np.arange(-14, -5)  # |gate| from 1/8 to 64
    A, P, S = (x.ravel() for x in np.meshgrid(a, exps, (1, -1), indexing="ij"))
    g = S * A * 2.0 ** P
    s = silu(g)
    found = []
    for border in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        m, e = np.frexp(border / np.abs(s))
        b = np.rint(m * 65536)  # 16 bits
        off = b / (m * 65536) - 1
        hit = (np.abs(off) >= low * 2.0 ** -24) & (np.abs(off) <= high * 2.0 ** -24)
        found += list(zip(S[hit] * A[hit], P[hit], b[hit].astype(np.int64), e[hit] - 16, np.full(hit.sum(), border), off[hit] > 0))
    assert len(found) >= count
    return [found[i] for i in rng.permutation(len(found))[:count]]


def test_silu_is_as_accurate_as_it_says():
    """The activation's error, up to 5 steps of 2^-24 and a little, and one of the product with up: an h that lies 6.5 to
    13 such steps from a border has the code of its own side.  The gate and up products are exact here, and the down
    projection hands h out as it is."""
    n = 4096
    levels = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    cases = near_borders(n // 32 * 31, 6.5, 13.0)
    cases = [c for i in range(n // 32) for c in [(2048, -5, 6 * 4096, -18, None, True), *cases[31 * i:31 * i + 31]]]
    # each block's first channel: 64 times 6/64, which sets the scale to 1
    a, p, b, q = (np.array([c[i] for c in cases]) for i in range(4))
    codes = {"g": digits(np.abs(a), 3) | ((digits(np.abs(a), 3) != 0) * np.where(a < 0, 8, 0)[:, None]).astype(np.uint8), "u": digits(b, 4)}
    at = mx4.tile_index(n, n)
    t = {}
    for k, base, num in (("g", p, 3), ("u", q, 4)):
        nib = np.zeros((n, n), np.uint8)
        nib[:, :32 * num] = codes[k]
        tiles = np.full(mx4.scale_size(n, n), 127, np.uint8)
        byte = 127 + base[:, None] + 4 * np.arange(num)
        assert (byte > 0).all() and (byte < 255).all()
        tiles[at[:, :num]] = byte
        t[k] = (nib[:, 0::2] | (nib[:, 1::2] << 4), tiles)
    g, u = (mx4.decode(t[k][0], t[k][1]).sum(1) for k in ("g", "u"))
    assert np.array_equal(g, a * 2.0 ** p) and np.array_equal(u, b * 2.0 ** q)
    h = silu(g) * u
    want = []
    for c, v in zip(cases, h):
        border, above = c[4:]
        assert border is None or abs(v) / border > 1 if above else abs(v) / border < 1
        low = 7 if border is None else max(i for i in range(8) if levels[i] < border) + bool(above)
        want.append(np.copysign(levels[low], v))
    one = np.zeros((1, n), np.uint8)
    one[:, :128] = 2
    ident = np.zeros((n, n), np.uint8)
    np.fill_diagonal(ident, 2)
    pack = lambda c: c[:, 0::2] | (c[:, 1::2] << 4)  # noqa: E731
    ones = lambda rows: np.full(mx4.scale_size(rows, n), 127, np.uint8)  # noqa: E731
    args = [(pack(one), ones(1)), (t["g"][0][None], t["g"][1][None]), (t["u"][0][None], t["u"][1][None]), (pack(ident)[None], ones(n)[None])]
    x, wg, wu, wd = [[torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in m] for m in args]
    ids, weights = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, 1, device="cuda")
    y = sq.mx4_moe(*x, ids, weights, *wg, *wu, *wd, out_dtype=F32).cpu().numpy()[0]
    wrong = np.flatnonzero(y != np.array(want))
    assert wrong.size == 0, [(cases[i], g[i], h[i], y[i]) for i in wrong[:5]]
