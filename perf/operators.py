"""The microscaled 4-bit operators of the library as they are measured: the quantiser, the linear layer, the norms
around a block with their gate and residual, and the mixture-of-experts layer for a few tokens.

Format (OCP microscaling MXFP4).  A block of 32 consecutive values along K shares one power-of-two scale 2^(b - 127)
(b one byte, E8M0) and each value is an E2M1 number 0, .5, 1, 1.5, 2, 3, 4, 6 with a sign:
    b = max(floor(log2 max|v|) - 2 + 127, 0),  code = round-half-even(v / 2^(b - 127)), at most 6.
Two codes share a byte (the even one low).  Scale bytes lie in tiles of 128 rows x 4 blocks (512 bytes), row tile by
row tile: byte (r % 32) * 16 + (r % 128 / 32) * 4 + block % 4 of a tile; the padding holds 0.
"""
import torch

own = False
DEVICE = "cuda"
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------------
def _quant(side, rows, K, dtype, smooth):
    return {"op": "quant", "side": side, "rows": rows, "K": K, "dtype": dtype, "smooth": smooth}


def _linear(M, N, K, dtype, out):
    return {"op": "linear", "M": M, "N": N, "K": K, "dtype": dtype, "out": out}


def _norm(M, K, dtype, to, gate_tokens, post):
    return {"op": "norm", "M": M, "K": K, "dtype": dtype, "to": to, "gate_tokens": gate_tokens, "post": post}


def _moe(T, topk, E, H, I, holes):
    return {"op": "moe", "T": T, "topk": topk, "E": E, "H": H, "I": I, "holes": holes}


def listed():
    return [
        # a decode batch's activations, quantised and read back: latency
        {"name": "quantise 8 tokens", **_quant("act", 8, 4096, "bf16", True)},
        # a fused gate/up weight quantised once offline: bandwidth
        {"name": "quantise a weight", **_quant("weight", 28672, 4096, "bf16", True)},
        # one token through the fused QKV projection: the weight is streamed
        {"name": "linear 1 token", **_linear(1, 6144, 4096, "bf16", "bf16")},
        # a decode batch through the fused gate/up projection
        {"name": "linear 32 tokens", **_linear(32, 28672, 4096, "bf16", "bf16")},
        # sizes that end inside every tile, in 32 bits
        {"name": "linear ragged f32", **_linear(203, 1040, 2336, "f32", "f32")},
        # a prompt through the fused QKV projection
        {"name": "linear prompt", **_linear(4096, 6144, 4096, "bf16", "bf16")},
        # a long prompt through a large down projection: the tensor cores' rate
        {"name": "linear long prompt", **_linear(8192, 8192, 28672, "bf16", "bf16")},
        # one token between two blocks
        {"name": "norm 1 token", **_norm(1, 4096, "bf16", "mx4", 0, True)},
        # a prompt between two blocks, one gate for each sequence of 512 tokens
        {"name": "norm prompt", **_norm(4096, 8192, "bf16", "mx4", 512, True)},
        # one token through two of eight large experts
        {"name": "moe 1 token", **_moe(1, 2, 8, 4096, 14336, False)},
        # a small batch over many small experts: nearly every expert has a token or two
        {"name": "moe 16 tokens", **_moe(16, 8, 128, 2048, 768, False)},
        # a batch on one part of the experts: choices that live elsewhere are marked -1
        {"name": "moe 64 tokens", **_moe(64, 6, 64, 2048, 1408, True)},
    ]


def _log(rng, lo, hi, step=1):
    """Whole multiples of `step` from lo to hi, even over the logarithm."""
    v = lo * (hi / lo) ** rng.random()
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("quant", "linear", "linear", "norm", "moe", "moe"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "quant":
        K = _log(rng, 32, 16384, 32)
        return _quant(rng.choice(("act", "weight")), _log(rng, 1, max(1, min(28672, 100_000_000 // K))), K, dtype, rng.random() < 0.7)
    if op == "linear":
        N, K = _log(rng, 64, 16384, 16), _log(rng, 64, 16384, 32)
        return _linear(_log(rng, 1, 8192), N, K, dtype, rng.choice(("bf16", "bf16", "f32")))
    if op == "norm":
        to = rng.choice(("mx4", "mx4", "int8"))
        K = _log(rng, 256, 16384, 32 if to == "mx4" else 16)
        M = _log(rng, 1, min(8192, 32_000_000 // K))
        return _norm(M, K, dtype, to, rng.choice((-1, 0, 1, 100, 512)), rng.random() < 0.7)
    E = rng.choice((4, 8, 16, 40, 64, 128))
    H = _log(rng, 256, 4096, 32)
    I = _log(rng, 256, max(256, min(8192, 400_000_000 // (E * H))), 32)
    return _moe(_log(rng, 1, 128), min(E, rng.choice((1, 2, 4, 6, 8))), E, H, I, rng.random() < 0.5)


# ----------------------------------------------------------------------------------------------------------------------
# the format in elementary operations
# ----------------------------------------------------------------------------------------------------------------------
def _round_mx4(v):
    """(values as the codes stand for them divided by their scale, scale bytes) of v [..., K] in 32 bits."""
    blocks = v.reshape(*v.shape[:-1], -1, 32)
    top = blocks.abs().amax(-1)
    byte = ((top.view(torch.int32) >> 23) - 2).clamp(min=0)
    a = blocks * ((254 - byte) << 23).view(torch.float32).unsqueeze(-1)  # a power of two: exact
    m = a.abs()
    q = torch.where(m < 2, (m * 2).round() / 2, torch.where(m < 4, m.round(), (m / 2).round() * 2)).clamp(max=6)
    return torch.copysign(q, a), byte


def _scale(byte):
    """2^(byte - 127) in 32 bits, byte 0 (below the normal numbers) among them."""
    return torch.where(byte > 0, byte << 23, torch.full_like(byte, 1 << 22)).view(torch.float32)


def _values(q, byte):
    return (q * _scale(byte).unsqueeze(-1)).flatten(-2)


def _pack(q):
    m = q.abs()
    code = torch.where(m < 2, m * 2, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(q).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _tile(byte):
    """Scale bytes [..., rows, blocks] laid out in tiles, [..., bytes]."""
    R, B = byte.shape[-2:]
    p = torch.zeros(*byte.shape[:-2], -(-R // 128) * 128, -(-B // 4) * 4, dtype=torch.uint8, device=byte.device)
    p[..., :R, :B] = byte.to(torch.uint8)
    p = p.reshape(-1, p.shape[-2] // 128, 4, 32, p.shape[-1] // 4, 4).permute(0, 1, 4, 3, 2, 5)
    return p.reshape(*byte.shape[:-2], -1).contiguous()


def _untile(t, R, B):
    rt, bt = -(-R // 128), -(-B // 4)
    p = t.reshape(-1, rt, bt, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(*t.shape[:-1], rt * 128, bt * 4)
    return p[..., :R, :B].to(torch.int32)


def _decode(codes, tiles):
    """The values of codes [..., R, K / 2] with their tiled scales [..., bytes], in 32 bits."""
    R, K = codes.shape[-2], codes.shape[-1] * 2
    table = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int32)
    return _values(table[c].reshape(*codes.shape[:-1], K // 32, 32), _untile(tiles, R, K // 32))


def _smooth(v, s, side):
    v = v.float()
    if s is None:
        return v
    return v * s if side == "weight" else v * (1.0 / s)


# ----------------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed))


def _acts(g, M, K, dtype):
    """Activations with a few channels far above the others, as a transformer's have."""
    x = torch.randn(M, K, generator=g, device=DEVICE)
    x[:, torch.randperm(K, generator=g, device=DEVICE)[: max(1, K // 1000)]] *= 60.0
    return x.to(dtype)


def _factors(g, K):
    return torch.rand(K, generator=g, device=DEVICE) * 3.0 + 0.3


def _weights(g, E, N, K):
    """E quantised weights: codes [E, N, K / 2] and tiled scales [E, bytes]."""
    codes, tiles = [], []
    for _ in range(E):
        q, byte = _round_mx4(torch.randn(N, K, generator=g, device=DEVICE) * 0.02)
        codes.append(_pack(q))
        tiles.append(_tile(byte))
    return torch.stack(codes), torch.stack(tiles)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    empty = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device=DEVICE)  # noqa: E731
    tiles = lambda rows, K: empty(-(-rows // 128) * -(-K // 128) * 512, dtype=torch.uint8)  # noqa: E731
    if c["op"] == "quant":
        R, K = c["rows"], c["K"]
        c["x"] = _acts(g, R, K, _dtype(c["dtype"])) if c["side"] == "act" else (torch.randn(R, K, generator=g, device=DEVICE) * 0.02).to(_dtype(c["dtype"]))
        c["s"] = _factors(g, K) if c["smooth"] else None
        c |= {"xq": empty(R, K // 2, dtype=torch.uint8), "sx": tiles(R, K), "y": empty(R, K, dtype=torch.bfloat16)}
    elif c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        c["x"] = _acts(g, M, K, _dtype(c["dtype"]))
        c["s"] = _factors(g, K)
        w, sw = _weights(g, 1, N, K)
        c |= {"wq": w[0], "sw": sw[0], "y": empty(M, N, dtype=_dtype(c["out"]))}
    elif c["op"] == "norm":
        M, K, dt = c["M"], c["K"], _dtype(c["dtype"])
        c["b"] = torch.randn(M, K, generator=g, device=DEVICE).to(dt)
        c["r"] = _acts(g, M, K, dt)
        c["gamma"] = torch.rand(K, generator=g, device=DEVICE) + 0.5 if c["post"] else None
        c["g"] = torch.rand(K, generator=g, device=DEVICE) * 1.5 + 0.1
        # a gate for every token, for each group of tokens, one for all (0), or none (-1)
        t = c["gate_tokens"] or M
        c["gate"] = None if t < 0 else torch.randn(-(-M // t), K, generator=g, device=DEVICE).to(dt)
        c["share"] = t
        c["r_out"] = empty(M, K, dtype=dt)
        if c["to"] == "mx4":
            c |= {"xq": empty(M, K // 2, dtype=torch.uint8), "sx": tiles(M, K), "y": empty(M, K, dtype=torch.bfloat16)}
        else:
            c |= {"xq": empty(M, K, dtype=torch.int8), "sx": empty(M, dtype=torch.float32)}
    else:
        T, E, H, I = c["T"], c["E"], c["H"], c["I"]
        q, byte = _round_mx4(_acts(g, T, H, torch.bfloat16).float())
        c |= {"xq": _pack(q), "sx": _tile(byte)}
        chosen = torch.rand(T, E, generator=g, device=DEVICE).topk(c["topk"], -1)
        weights = chosen.values.softmax(-1)
        ids = chosen.indices.to(torch.int32)
        if c["holes"]:
            ids = torch.where(torch.rand(ids.shape, generator=g, device=DEVICE) < 0.25, torch.full_like(ids, -1), ids)
        c |= {"ids": ids.contiguous(), "weights": weights.contiguous()}
        c["wg"], c["sg"] = _weights(g, E, I, H)
        c["wu"], c["su"] = _weights(g, E, I, H)
        c["wd"], c["sd"] = _weights(g, E, H, I)
        c["y"] = empty(T, H, dtype=torch.bfloat16)
    return c


# ----------------------------------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------------------------------
def _workspace(c, size):
    if "ws" not in c:
        c["ws"] = torch.empty(max(16, size), dtype=torch.uint8, device=DEVICE)
    return c["ws"]


def _run_own(c):
    import w8a8_int8_gemm_channel_b200 as sq

    if c["op"] == "quant":
        (sq.sq_mx4_quant_act if c["side"] == "act" else sq.sq_mx4_quant_weight)(c["x"], c["s"], c["xq"], c["sx"])
        sq.sq_mx4_dequant(c["xq"], c["sx"], c["y"])
        return c["y"]
    if c["op"] == "linear":
        ws = c["ws"] if "ws" in c else _workspace(c, sq.sq_mx4_linear_workspace_size(c["M"], c["N"], c["K"]))
        sq.sq_mx4_linear(c["x"], c["s"], c["wq"], c["sw"], c["y"], ws)
        return c["y"]
    if c["op"] == "norm":
        if c["to"] == "mx4":
            sq.sq_residual_norm_quant_mx4(c["b"], c["gamma"], c["gate"], c["share"], 0.8, c["r"], c["r_out"], c["g"], 1e-5, c["xq"], c["sx"])
            sq.sq_mx4_dequant(c["xq"], c["sx"], c["y"])
            return {"r": c["r_out"], "a": c["y"]}
        sq.sq_residual_norm_quant(c["b"], c["gamma"], c["gate"], c["share"], 0.8, c["r"], c["r_out"], c["g"], 1e-5, c["xq"], c["sx"])
        return {"r": c["r_out"], "a": torch.mul(c["xq"], c["sx"].unsqueeze(1))}
    ws = c["ws"] if "ws" in c else _workspace(c, sq.sq_mx4_moe_workspace_size(c["T"], c["topk"], c["E"], c["H"], c["I"]))
    sq.sq_mx4_moe(c["xq"], c["sx"], c["ids"], c["weights"], c["wg"], c["sg"], c["wu"], c["su"], c["wd"], c["sd"], c["y"], ws)
    return c["y"]


def _rinv(v, eps):
    """1 / RMS, the mean square in 64 bits and rounded once (codes next to a border hang on its last bit)."""
    return (1.0 / (v.double().square().mean(-1, keepdim=True) + eps).sqrt()).float()


def run(state):
    c = state
    if own:
        return _run_own(c)
    if c["op"] == "quant":
        return _values(*_round_mx4(_smooth(c["x"], c["s"], c["side"]))).to(torch.bfloat16)
    if c["op"] == "linear":
        x = _values(*_round_mx4(_smooth(c["x"], c["s"], "act")))
        return torch.matmul(x, _decode(c["wq"], c["sw"]).t()).to(_dtype(c["out"]))
    if c["op"] == "norm":
        u = c["b"].float()
        if c["gamma"] is not None:
            u = u * _rinv(u, 1e-5) * c["gamma"]
        if c["gate"] is not None:
            u = u * c["gate"].float()[torch.arange(c["M"], device=DEVICE) // c["share"]]
        c08 = torch.tensor(0.8, device=DEVICE)
        r = (c["r"].float() + u * c08).to(c["r"].dtype)
        a = r.float() * _rinv(r, 1e-5) * c["g"]
        if c["to"] == "mx4":
            return {"r": r, "a": _values(*_round_mx4(a)).to(torch.bfloat16)}
        sx = a.abs().amax(-1, keepdim=True) / 127
        q = torch.where(sx > 0, (a / sx).round(), torch.zeros_like(a)).clamp(-127, 127)
        return {"r": r, "a": q * sx}
    x = _decode(c["xq"], c["sx"])
    gate = torch.matmul(x, _decode(c["wg"], c["sg"]).transpose(1, 2))  # every expert for every token: [E, T, I]
    up = torch.matmul(x, _decode(c["wu"], c["su"]).transpose(1, 2))
    h = _values(*_round_mx4(gate / (1 + torch.exp(-gate)) * up))
    out = torch.matmul(h, _decode(c["wd"], c["sd"]).transpose(1, 2))  # [E, T, H]
    here = c["ids"] >= 0
    picked = out[c["ids"].clamp(min=0).long(), torch.arange(c["T"], device=DEVICE).unsqueeze(1)]  # [T, topk, H]
    return (picked * torch.where(here, c["weights"], torch.zeros_like(c["weights"])).unsqueeze(-1)).sum(1).to(torch.bfloat16)


# ----------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------------------------------------------
def work(case):
    c = case
    size = lambda name: 2 if name == "bf16" else 4  # noqa: E731
    mx4 = 0.5 + 1 / 32  # bytes a value
    if c["op"] == "quant":  # the values in, the codes out and in again, the values they stand for out
        n = c["rows"] * c["K"]
        return {"bytes": n * (size(c["dtype"]) + 2 * mx4 + 2) + (4 * c["K"] if c["smooth"] else 0), "flops": 3 * n}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K * size(c["dtype"]) + 4 * K + N * K * mx4 + M * N * size(c["out"]), "flops": 2 * M * N * K}
    if c["op"] == "norm":
        n, d = c["M"] * c["K"], size(c["dtype"])
        gates = 0 if c["gate_tokens"] < 0 else -(-c["M"] // (c["gate_tokens"] or c["M"])) * c["K"] * d
        back = 2 * mx4 + 2 if c["to"] == "mx4" else 2 * 1 + 4
        return {"bytes": n * (3 * d + back) + gates + c["K"] * 4 * (1 + bool(c["post"])), "flops": 14 * n}
    T, E, H, I = c["T"], c["E"], c["H"], c["I"]
    kept = 0.75 if c["holes"] else 1.0
    experts = E * (1 - (1 - kept * c["topk"] / E) ** T)  # expected number of different experts
    return {"bytes": experts * 3 * H * I * mx4 + T * H * (mx4 + 2) + 8 * T * c["topk"], "flops": 6 * T * c["topk"] * kept * H * I}


# ----------------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------------------------------------------------
def _f32(v):
    """One rounding to 32 bits that the definition names."""
    return v.float().double()


def _exact_mx4(v):
    """What the codes of v [..., K] (64 bits) stand for."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    e = (torch.frexp(b.abs().amax(-1, keepdim=True)).exponent - 3).clamp(min=-127)
    unit = torch.ldexp(torch.ones_like(e, dtype=torch.float64), e)
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=v.device)
    border[1::2] = torch.nextafter(border[1::2], torch.zeros_like(border[1::2]))  # a tie goes to the even code
    level = torch.tensor(LEVELS, dtype=torch.float64, device=v.device)[torch.bucketize((b / unit).abs(), border)]
    return (torch.sign(b) * level * unit).flatten(-2)


def _exact_decode(codes, tiles):
    R, K = codes.shape[0], codes.shape[1] * 2
    r = torch.arange(R, device=codes.device).unsqueeze(1)
    k = torch.arange(K // 32, device=codes.device).unsqueeze(0)
    at = ((r // 128) * -(-K // 128) + k // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + k % 4
    unit = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=codes.device), tiles[at].double() - 127)
    v = torch.empty(R, K, dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        c = (codes >> (4 * half)) & 15
        m, e = (c & 1).double(), ((c >> 1) & 3).double()
        mag = torch.where(e > 0, (1 + m / 2) * torch.pow(torch.full_like(e, 2.0), e - 1), m / 2)
        v[:, half::2] = torch.where(c >= 8, -mag, mag)
    return v * unit.repeat_interleave(32, 1)


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] in ("quant", "linear"):
        x = c["x"].double()
        if c["s"] is not None:
            x = _f32(x * (c["s"].double() if c.get("side") == "weight" else _f32(1 / c["s"].double())))
        x = _exact_mx4(x)
        return x if c["op"] == "quant" else x @ _exact_decode(c["wq"], c["sw"]).t()
    if c["op"] == "norm":
        u = c["b"].double()
        if c["gamma"] is not None:
            u = _f32(_f32(u * _f32((u.square().sum(1, keepdim=True) / c["K"] + 1e-5).rsqrt())) * c["gamma"].double())
        if c["gate"] is not None:
            u = _f32(u * c["gate"].double().repeat_interleave(c["share"], 0)[: c["M"]])
        r = _f32(c["r"].double() + _f32(u * torch.tensor(0.8).double().item())).to(c["r"].dtype).double()
        a = _f32(_f32(r * _f32((r.square().sum(1, keepdim=True) / c["K"] + 1e-5).rsqrt())) * c["g"].double())
        if c["to"] == "mx4":
            return {"r": r, "a": _exact_mx4(a)}
        sx = _f32(a.abs().amax(1, keepdim=True) / 127)
        return {"r": r, "a": torch.round(_f32(a / sx.clamp(min=1e-300))).clamp(-127, 127) * sx}
    x = _exact_decode(c["xq"], c["sx"])
    y = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEVICE)
    for e in range(c["E"]):
        w = torch.where(c["ids"] == e, c["weights"].double(), torch.zeros((), dtype=torch.float64, device=DEVICE)).sum(1)
        rows = (c["ids"] == e).any(1).nonzero().squeeze(1)
        if rows.numel():
            g = x[rows] @ _exact_decode(c["wg"][e], c["sg"][e]).t()
            u = x[rows] @ _exact_decode(c["wu"][e], c["su"][e]).t()
            y[rows] += w[rows].unsqueeze(1) * (_exact_mx4(g * torch.sigmoid(g) * u) @ _exact_decode(c["wd"][e], c["sd"][e]).t())
    return y
