"""Plain NumPy definitions of the microscaled 4-bit (OCP MXFP4) operators, for
the tests: element by element in 64 bits with the fp32 roundings that
include/sq.h names.  Shares no code with the library.

Arrays are fp32 or fp64 values; codes are uint8 [rows, K / 2] and scales uint8
in tiles (see tile_index).
"""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def f32(v):
    """One rounding to fp32, kept in fp64."""
    return np.asarray(v, np.float64).astype(np.float32).astype(np.float64)


def tile_index(rows, K):
    """Byte offset of the scale of row r, block i: an array [rows, K / 32]."""
    r = np.arange(rows)[:, None]
    i = np.arange(K // 32)[None, :]
    return ((r // 128) * (-(-K // 128)) + i // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + i % 4


def scale_size(rows, K):
    return -(-rows // 128) * -(-K // 128) * 512


def round_e2m1(a):
    """Codes 0..7 of the magnitudes a: the nearest level, ties to the even code, above 6 the 7th."""
    a = np.asarray(a, np.float64)
    code = np.zeros(a.shape, np.int64)
    for c in range(1, 8):
        mid = (LEVELS[c - 1] + LEVELS[c]) / 2
        code = np.where((a > mid) | ((a == mid) & (c % 2 == 0)), c, code)
    return code


def quantize(v):
    """(codes, scale tiles, the values they stand for [rows, K]) of v [rows, K]."""
    v = np.asarray(v, np.float64)
    rows, K = v.shape
    blocks = v.reshape(rows, K // 32, 32)
    finite = np.isfinite(blocks).all(-1)
    top = np.abs(np.where(finite[..., None], blocks, 0.0)).max(-1)
    _, e = np.frexp(top)  # top = m 2^e, m in [.5, 1)
    byte = np.where(top > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
    unit = np.ldexp(1.0, byte - 127)
    safe = np.where(finite[..., None], blocks, 0.0)
    code = round_e2m1(np.abs(safe) / unit[..., None])
    neg = np.signbit(safe) & finite[..., None]
    value = np.where(neg, -1.0, 1.0) * LEVELS[code] * unit[..., None]
    value = np.where(finite[..., None], value, np.nan).reshape(rows, K)
    nib = (code + 8 * neg).astype(np.uint8)
    nib = np.where(finite[..., None], nib, 0).astype(np.uint8).reshape(rows, K)
    tiles = np.zeros(scale_size(rows, K), np.uint8)
    tiles[tile_index(rows, K)] = np.where(finite, byte, 255)
    return nib[:, 0::2] | (nib[:, 1::2] << 4), tiles, value


def decode(codes, tiles):
    """The values of codes [rows, K / 2] with their scale tiles, in fp64."""
    rows, half = codes.shape
    K = 2 * half
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(rows, K)
    v = np.where(nib & 8, -1.0, 1.0) * LEVELS[nib & 7]
    b = tiles[tile_index(rows, K)].astype(np.int64)
    unit = np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))
    return v * np.repeat(unit, 32, axis=1)


def smooth_act(x, s):
    """x / s as the quantiser computes it: RN(x * RN(1 / s))."""
    x = np.asarray(x, np.float64)
    return x if s is None else f32(x * f32(1.0 / np.asarray(s, np.float64)))


def smooth_weight(w, s):
    w = np.asarray(w, np.float64)
    return w if s is None else f32(w * np.asarray(s, np.float64))


def product(x, w):
    """(y, sum of magnitudes): x [M, K] times w [N, K] transposed, in fp64."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def product_bound(K, mags, y, out_eps):
    """How far an fp32-accumulated product may be from y: every one of at most
    K additions is off by one unit of the running sum's last place (2^-23 of at
    most the sum of magnitudes) or, below fp32's normal numbers, by the smallest
    of them (a sum of 4.5e-61 has no fp32 value but 0); then one rounding to the
    output type."""
    return K * (2.0 ** -23 * mags + 2.0 ** -126) + out_eps / 2 * np.abs(y)
