"""Experts layers whose tiles are shared by several CTAs, compared without a tolerance.

How many CTAs share a tile is chosen from the sizes, in each half: one (nothing
is summed), some for each tile, or all of them with ranges that cross the borders
of tiles and experts.  SHAPES names what each layer has to get at 148 SMs;
test_mx4_plan_host.py holds the launch code to it, so that another choice cannot
leave the sums untested.

The inputs make every sum exact in fp32, in any order, so the outputs have one
right value.  Codes are 0, 1 or 2 with a sign and scales span two binades.  The
gate products are multiples of 256: above 0, v / (1 + e^-v) is v in fp32, and
below, a zero.  Then h is one fp32 product, its codes have no border to miss, and
the down products and routing weights (powers of two) are whole multiples of one
step.  definition() asserts that their sum of magnitudes stays below 2^24 steps.
"""
import numpy as np
import pytest
import torch

import w8a8_int8_gemm_channel_b200 as sq
from oracle import mx4

F32, BF16 = torch.float32, torch.bfloat16

# (tokens, choices, experts, H, I): CTAs a tile of the first and the second half ("even": ranges across borders)
SHAPES = {
    (1, 1, 1, 4128, 3104): ("even", 1),
    (9, 1, 1, 3104, 160): (3, 1),
    (2, 2, 64, 2048, 1408): (3, 8),
    (20, 2, 40, 3104, 32): ("even", "even"),
    (20, 3, 6, 288, 3104): ("even", 13),
    (33, 1, 1, 6176, 96): (2, 1),
    (33, 1, 16, 3104, 160): ("even", 1),
    (33, 2, 6, 288, 3104): ("even", 6),
    (48, 2, 40, 5152, 288): (1, "even"),
    (64, 6, 64, 2048, 1408): ("even", 9),
    (65, 1, 2, 6176, 160): (3, 1),
    (65, 1, 24, 1568, 96): (4, 4),
    (100, 4, 40, 288, 416): ("even", 8),
    (128, 8, 16, 2048, 1024): (1, 6),
    (100, 4, 8, 4096, 4096): ("even", "even"),
}


def codes(g, *shape, density):
    """Codes and values, the magnitudes 0, 1 and 2."""
    v = torch.randint(1, 3, shape, generator=g, device=g.device) * (torch.rand(shape, generator=g, device=g.device) < density)
    v *= torch.randint(0, 2, shape, generator=g, device=g.device) * 2 - 1
    c = (v.abs() * 2 + 8 * (v < 0)).to(torch.uint8)  # E2M1: 1 is code 2, 2 is code 4
    return c[..., 0::2] | (c[..., 1::2] << 4), v.to(torch.int8)


def matrix(g, E, rows, K, base, density):
    """(codes [E, rows, K / 2], scale tiles [E, bytes], values of an expert's matrix in 64 bits)."""
    q, v = codes(g, E, rows, K, density=density)
    byte = torch.randint(base - 1, base + 2, (E, rows, K // 32), generator=g, device=g.device)
    tiles = torch.zeros(E, mx4.scale_size(rows, K), dtype=torch.uint8, device=g.device)
    at = torch.from_numpy(mx4.tile_index(rows, K)).to(g.device)
    tiles[:, at] = byte.to(torch.uint8)
    unit = torch.tensor([2.0 ** (b - 127) for b in range(256)], dtype=torch.float64, device=g.device)  # (pow is not exact there)
    return q, tiles, lambda e: v[e].double() * unit[byte[e]].repeat_interleave(32, 1)


def make(T, topk, E, H, I, device, seed=0):
    """(arguments of the call, values): every expert is chosen, each by as many tokens as any other, or one more."""
    g = torch.Generator(device=device).manual_seed(T + H + I + seed)
    x, wg, wu = matrix(g, 1, T, H, 127, 0.5), matrix(g, E, I, H, 137, 0.5), matrix(g, E, I, H, 127, 0.5)
    wd = matrix(g, E, H, I, 127, 0.25)
    ids = (torch.arange(T * topk, device=device).reshape(T, topk) % E)[torch.randperm(T, generator=g, device=device)]
    weights = torch.tensor([1.0, 0.5, -1.0, 2.0], device=device)[torch.randint(0, 4, (T, topk), generator=g, device=device)]
    args = [x[0][0], x[1][0], ids.to(torch.int32).contiguous(), weights, wg[0], wg[1], wu[0], wu[1], wd[0], wd[1]]
    return args, (x[2](0), wg[2], wu[2], wd[2], ids, weights)


def definition(x, wg, wu, wd, ids, weights, E, I):
    """The layer in 64 bits; asserts that fp32 holds every sum of it."""
    T, H = x.shape
    y, mags = torch.zeros(T, H, dtype=torch.float64, device=x.device), torch.zeros(T, H, dtype=torch.float64, device=x.device)
    step = float("inf")
    for e in range(E):
        rows = (ids == e).any(1).nonzero().squeeze(1)
        if not rows.numel():
            continue
        v = torch.where(ids[rows] == e, weights[rows], 0.0).sum(1).double().unsqueeze(1)
        g, u = x[rows] @ wg(e).t(), x[rows] @ wu(e).t()
        assert (g % 256 == 0).all() and (u % 0.25 == 0).all()
        assert max(g.abs().max() / 256, u.abs().max() * 4) < 2 ** 24
        assert (x[rows].abs() @ wg(e).abs().t()).max() < 2 ** 32 and (x[rows].abs() @ wu(e).abs().t()).max() < 2 ** 22
        h = (g.clamp(min=0).float() * u.float()).cpu().numpy()
        hv = torch.from_numpy(mx4.quantize(h)[2]).to(x.device)
        block = hv.reshape(len(rows), I // 32, 32).abs()
        least = block[block > 0].min().item() if (block > 0).any() else float("inf")
        # the least value of a code is half of its scale, which is a value's at the lowest
        step = min(step, 2.0 ** (np.floor(np.log2(least)) - 2) * 0.5 * v.abs().min().item()) if least < float("inf") else step
        d = wd(e)
        y[rows] += v * (hv @ d.t())
        mags[rows] += v.abs() * (hv.abs() @ d.abs().t())
    assert mags.max().item() < 2 ** 24 * step, f"sums of {np.log2(mags.max().item() / step):.1f} bits"
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shared_tiles_are_summed_exactly(shape):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    T, topk, E, H, I = shape
    args, values = make(*shape, "cuda")
    want = definition(*values, E, I)
    assert torch.equal(want.float().double(), want) and (want != 0).any()
    for out in (F32, BF16):
        ws = torch.full((sq.sq_mx4_moe_workspace_size(*shape),), 0xFF, dtype=torch.uint8, device="cuda")
        y = torch.full((T + 1, H), 9.0, dtype=out, device="cuda")
        for _ in range(4):  # the first call finds no tagged words
            y[:T] = float("nan")
            sq.sq_mx4_moe(*args, y[:T], ws)
            assert torch.equal(y[:T], want.to(out))
        assert (y[T] == 9.0).all()
    # some tokens' choices live elsewhere: fewer a tile, or fewer experts and other ranges
    args[2][::3] = -1
    values[4][::3] = -1
    y = sq.mx4_moe(*args, out_dtype=F32)
    assert torch.equal(y, definition(*values, E, I).float())
    assert sq.sq_device_status() == (sq.SQ_OK, 0)
