"""Cases that time and check what stands around a product with 4-bit weights: the
root-mean-square norm with the residual's addition and a quantised output, its
backward pass, the product of 8-bit activations with 4-bit weight shards, and
the product of a few unquantised tokens with them.

``run`` computes each operator in plain torch operations, or, with ``own`` set,
makes the calls a user of this package makes.  Both start from the same buffers.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BLOCK = {"mxfp4": 32, "nvfp4": 16, "mxfp8": 32}
BITS = {"mxfp4": 4, "nvfp4": 4, "mxfp8": 8}


def dtype(word):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[word]


# --- the cases ---------------------------------------------------------------------

def listed():
    return [
        # one token entering a layer while it is served: all launch latency
        {"name": "norm 1x4096 to 8 bits", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "weight": "bf16", "residual": True, "format": "mxfp8"},
        # a GPT-2-small-wide model in fp32, the norm before anything is quantised
        {"name": "norm 1000x768 fp32", "op": "norm", "rows": 1000, "cols": 768, "dtype": "f32", "weight": "f32", "residual": False, "format": "none"},
        # ragged rows of a packed batch, straight to the operand of a 4-bit product
        {"name": "norm 2050x1120 to nvfp4", "op": "norm", "rows": 2050, "cols": 1120, "dtype": "bf16", "weight": "f32", "residual": True, "format": "nvfp4"},
        # the tokens of a training step entering a large layer
        {"name": "norm 8192x4096 to 8 bits", "op": "norm", "rows": 8192, "cols": 4096, "dtype": "bf16", "weight": "bf16", "residual": True, "format": "mxfp8"},
        # backward of the small layer of the all-gather fixture
        {"name": "norm grad 128x512", "op": "norm_grad", "rows": 128, "cols": 512, "dtype": "bf16", "weight": "bf16", "residual": True},
        # odd sizes in fp32: no row starts on a boundary
        {"name": "norm grad 1031x1601 fp32", "op": "norm_grad", "rows": 1031, "cols": 1601, "dtype": "f32", "weight": "f32", "residual": False},
        # backward of the large layer
        {"name": "norm grad 8192x4096", "op": "norm_grad", "rows": 8192, "cols": 4096, "dtype": "bf16", "weight": "bf16", "residual": True},
        # the small all-gather product
        {"name": "8-bit x, 128x512x512", "op": "product8", "M": 128, "D": 512, "K": 8, "F_shard": 64},
        # ragged tokens, features and shards
        {"name": "8-bit x, 777x1056x832", "op": "product8", "M": 777, "D": 1056, "K": 4, "F_shard": 208},
        # the large all-gather product
        {"name": "8-bit x, 8192x4096x4096", "op": "product8", "M": 8192, "D": 4096, "K": 8, "F_shard": 512},
        # one token through the large layer
        {"name": "one token, 4096x4096", "op": "tokens", "M": 1, "D": 4096, "K": 8, "F_shard": 512, "format": "nvfp4"},
        # sixteen sequences' tokens through a vocabulary-wide layer
        {"name": "16 tokens, 8192x65536", "op": "tokens", "M": 16, "D": 8192, "K": 8, "F_shard": 8192, "format": "mxfp4"},
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "product8", "tokens"])
    if op in ("norm", "norm_grad"):
        c = {"op": op, "rows": log_int(rng, 1, 8192), "dtype": rng.choice(["bf16", "bf16", "f32"]), "weight": rng.choice(["bf16", "f32"]), "residual": rng.random() < 0.6}
        if op == "norm":
            c["format"] = rng.choice(["none", "mxfp8", "mxfp8", "mxfp4", "nvfp4"])
        c["cols"] = 32 * log_int(rng, 2, 192) if rng.random() < 0.6 or c.get("format", "none") != "none" else log_int(rng, 33, 6000)
        return c
    K = rng.choice([1, 2, 4, 8])
    if op == "product8":
        return {"op": op, "M": log_int(rng, 1, 8192), "D": 32 * log_int(rng, 2, 128), "K": K, "F_shard": 16 * log_int(rng, 1, 32)}
    return {"op": op, "M": log_int(rng, 1, 32), "D": 32 * log_int(rng, 2, 256), "K": K, "F_shard": 16 * log_int(rng, 1, 256), "format": rng.choice(["mxfp4", "nvfp4"])}


# --- what a program has in hand -----------------------------------------------------

def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed % (1 << 62))


def loud(x, g):
    """Activations: a few channels are many times louder than the others."""
    return x * (1 + 10 * (torch.rand(x.shape[1], device=DEV, generator=g) > 0.99))


def prepare(c, seed):
    g = gen(seed)
    if c["op"] in ("norm", "norm_grad"):
        T, shape = dtype(c["dtype"]), (c["rows"], c["cols"])
        x = loud(torch.randn(shape, device=DEV, generator=g), g).to(T)
        w = (1 + 0.2 * torch.randn(c["cols"], device=DEV, generator=g)).to(dtype(c["weight"]))
        more = torch.randn(shape, device=DEV, generator=g)
        s = {"c": c, "w": w}
        if c["op"] == "norm":
            s.update(x=x, residual=more.to(T) if c["residual"] else None)
            # calibrated beforehand, as the tensor scale of activations is
            s["scale"] = torch.full((1,), 8.0 / 2688.0, device=DEV) if c["format"] == "nvfp4" else None
            return s
        # what the forward pass left, and the gradients that arrive
        s.update(h=x, rstd=torch.rsqrt(x.double().square().mean(1) + EPS).float(), dy=(more * 1e-3).to(T))
        s["dh"] = (torch.randn(shape, device=DEV, generator=g) * 1e-3).to(T) if c["residual"] else None
        return s
    x = loud(torch.randn(c["M"], c["D"], device=DEV, generator=g), g).to(torch.bfloat16)
    w = torch.randn(c["K"] * c["F_shard"], c["D"], device=DEV, generator=g) * 0.02
    fmt = c.get("format", "mxfp4")
    t = (w.abs().amax() / 2688.0).view(1) if fmt == "nvfp4" else None
    codes, byte = encode4(w, fmt, t)
    packed, tiled = pack4(codes), tile_scales(byte, c["K"], c["F_shard"])
    s = {"c": c, "x": x, "w": packed, "w_scales": tiled, "w_scale": t}
    if own:
        from ring_allreduce_gradient_gb300 import mx4
        s["shards"] = [mx4.Mx4Tensor(a, b, c["F_shard"], c["D"], fmt, t) for a, b in zip(packed.chunk(c["K"]), tiled.unbind(0))]
    return s


# --- plain forms ----------------------------------------------------------------------

def power(e):
    return torch.ldexp(torch.ones(e.shape, device=e.device), e)


def encode4(x, fmt, t):
    """4-bit values (as fp32) and one 8-bit scale (as its byte) per block along the rows of x."""
    b = x.unflatten(1, (-1, BLOCK[fmt]))
    top = b.abs().amax(2)
    if fmt == "mxfp4":      # a power of two: floor(log2(largest)) - 2
        e = torch.where(top > 0, (torch.frexp(top)[1] - 3).clamp(-127, 127), -127)
        byte, step = (e + 127).to(torch.uint8), power(e)
    else:
        f8 = (top * (1.0 / 6.0) / t).clamp(max=448.0).to(torch.float8_e4m3fn)
        byte, step = f8.view(torch.uint8), f8.float() * t
    y = torch.where(step[..., None] > 0, b / step[..., None], 0.0)
    a = y.abs()
    unit = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = ((a / unit).round() * unit).clamp(max=6.0).copysign(y)
    return q.flatten(1), byte


def steps_of(byte, fmt, t):
    return power(byte.to(torch.int32) - 127) if fmt == "mxfp4" else byte.view(torch.float8_e4m3fn).float() * t


def decode4(q, byte, fmt, t):
    return (q.unflatten(1, (-1, BLOCK[fmt])) * steps_of(byte, fmt, t)[..., None]).flatten(1)


def values8(x):
    """The values that x stands for in 8 bits: e4m3 times the smallest power of two that keeps a block of 32 below 448."""
    b = x.unflatten(1, (-1, BLOCK["mxfp8"]))
    top = b.abs().amax(2, keepdim=True)
    m, e = torch.frexp(top)                              # top = m 2^e, m in [0.5, 1)
    e = (e - 9 + (m > 0.875).int()).clamp(min=-127)      # 448 = 0.875 2^9
    return ((b * power(-e)).to(torch.float8_e4m3fn).float() * power(e)).flatten(1)


def magnitudes(device):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)


def pack4(q):
    """Two values a byte, the first in the low half; bit 3 is the sign."""
    code = torch.bucketize(q.abs(), magnitudes(q.device)).to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def unpack4(packed):
    code = torch.stack([packed & 15, packed >> 4], 2).flatten(1).int()
    return magnitudes(packed.device)[code & 7] * (1.0 - 2.0 * (code >> 3))


def tile_scales(byte, K, rows):
    """[K * rows, blocks] scale bytes as each shard's 512-byte tiles of 128 rows x 4 blocks:
    row r, block b of a tile at (r % 32) * 16 + (r // 32) * 4 + b; zero where there is none."""
    R, B = -(-rows // 128), -(-byte.shape[1] // 4)
    full = byte.new_zeros(K, R * 128, B * 4)
    full[:, :rows, :byte.shape[1]] = byte.view(K, rows, -1)
    return full.view(K, R, 4, 32, B, 4).permute(0, 1, 4, 3, 2, 5).reshape(K, -1)


def untile_scales(tiled, K, rows, blocks):
    R, B = -(-rows // 128), -(-blocks // 4)
    full = tiled.view(K, R, B, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(K, R * 128, B * 4)
    return full[:, :rows, :blocks].reshape(K * rows, blocks)


def plain_weights(s):
    c = s["c"]
    fmt = c.get("format", "mxfp4")
    byte = untile_scales(s["w_scales"], c["K"], c["F_shard"], c["D"] // BLOCK[fmt])
    return decode4(unpack4(s["w"]), byte, fmt, s["w_scale"])


def plain_norm(s):
    c, x = s["c"], s["x"]
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    v = h.float()
    rstd = torch.rsqrt(v.square().mean(1) + EPS)
    y = v * rstd[:, None] * s["w"].float()
    if c["format"] == "mxfp8":
        y = values8(y)
    elif c["format"] != "none":
        y = decode4(*encode4(y, c["format"], s["scale"]), c["format"], s["scale"])
    return {"y": y.to(x.dtype if c["format"] == "none" else torch.bfloat16), "h": h, "rstd": rstd}


def plain_norm_grad(s):
    xh = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = (g - xh * (g * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dw": (dy * xh).sum(0)}


# --- one pass --------------------------------------------------------------------------

def run(s):
    c = s["c"]
    if not own:
        if c["op"] == "norm":
            return plain_norm(s)
        if c["op"] == "norm_grad":
            return plain_norm_grad(s)
        x = values8(s["x"].float()) if c["op"] == "product8" else s["x"].float()
        return (x @ plain_weights(s).t()).to(torch.bfloat16)
    from ring_allreduce_gradient_gb300 import mx4, mx8, norm
    if c["op"] == "norm":
        if c["format"] == "none":
            n = norm.rms_norm(s["x"], s["w"], residual=s["residual"], eps=EPS)
            return {"y": n.y, "h": n.h, "rstd": n.rstd}
        n = norm.rms_norm(s["x"], s["w"], residual=s["residual"], eps=EPS, format=c["format"], tensor_scale=s["scale"])
        y = mx8.dequantize(n.q) if c["format"] == "mxfp8" else mx4.dequantize(n.q)
        return {"y": y, "h": n.h, "rstd": n.rstd}
    if c["op"] == "norm_grad":
        dx, dw = norm.rms_norm_backward(s["dy"], s["h"], s["w"], s["rstd"], dh=s["dh"])
        return {"dx": dx, "dw": dw}
    if c["op"] == "product8":
        return mx8.linear(s["x"], s["shards"])
    return mx4.linear_w4(s["x"], s["shards"])


def work(c):
    wide = {"f32": 4, "bf16": 2}
    if c["op"] in ("norm", "norm_grad"):
        n, e = c["rows"] * c["cols"], wide[c["dtype"]]
        if c["op"] == "norm_grad":
            return {"bytes": n * e * (4 if c["residual"] else 3) + 4 * c["rows"] + c["cols"] * (wide[c["weight"]] + 4), "flops": 12 * n}
        f = c["format"]
        out = e if f == "none" else BITS[f] / 8 + 1 / BLOCK[f] + 2      # the quantised form, and its values in bf16
        return {"bytes": n * (e * (3 if c["residual"] else 1) + out) + 4 * c["rows"] + c["cols"] * wide[c["weight"]], "flops": 6 * n}
    M, D, F = c["M"], c["D"], c["K"] * c["F_shard"]
    per = 0.5 + 1 / BLOCK[c.get("format", "mxfp4")]      # bytes of a weight with its share of a scale
    return {"bytes": 2 * M * D + per * F * D + 2 * M * F, "flops": 2 * M * D * F}


# --- the definitions in 64 bits --------------------------------------------------------

def power_below(a):
    """The largest power of two that is no larger than a (a > 0)."""
    return a / (2 * torch.frexp(a).mantissa)


def nearest(x, low, high, top, parts):
    """Nearest value with `parts` steps to a power of two between low and high, ties to even, saturated at top."""
    a = x.abs()
    grid = power_below(a.clamp(min=low, max=high)) / parts
    return (torch.round(a / grid) * grid).clamp(max=top) * torch.sign(x)


def exact_values(y, fmt, t):
    """What 64-bit y [rows, cols] stands for in a format, blocks along its rows."""
    b = y.reshape(y.shape[0], -1, BLOCK[fmt])
    top = b.abs().max(2, keepdim=True).values
    if fmt == "nvfp4":
        step = nearest(top / (6.0 * t), 2.0 ** -6, 256.0, 448.0, 8) * t
    elif fmt == "mxfp4":
        step = power_below(top.clamp(min=2.0 ** -125)) / 4
    else:
        step = power_below(top.clamp(min=2.0 ** -119)) / 256
        step = torch.where(top > 448.0 * step, 2 * step, step)
    z = b / torch.where(step == 0, 1.0, step)
    q = nearest(z, 2.0 ** -6, 256.0, 448.0, 8) if fmt == "mxfp8" else nearest(z, 1.0, 4.0, 6.0, 2)
    return (q * step).reshape(y.shape)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(s["x"].dtype).double()
        rstd = 1 / torch.sqrt((h * h).sum(1) / c["cols"] + EPS)
        y = h * rstd.unsqueeze(1) * s["w"].double()
        if c["format"] != "none":
            y = exact_values(y, c["format"], None if s["scale"] is None else s["scale"].double())
        return {"y": y, "h": h, "rstd": rstd}
    if c["op"] == "norm_grad":
        h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double().unsqueeze(1)
        g = dy * s["w"].double()
        dx = r * g - h * r ** 3 * ((g * h).sum(1, keepdim=True) / c["cols"])
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dw": torch.einsum("mn,mn->n", dy, h * r)}
    F = c["K"] * c["F_shard"]
    w = torch.empty(F, c["D"], dtype=torch.float64, device=DEV)
    code = s["w"].long()
    table = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=DEV) / 2
    table = torch.cat([table, -table])
    w[:, 0::2], w[:, 1::2] = table[code % 16], table[code // 16]
    fmt = c.get("format", "mxfp4")
    rows = torch.arange(F, device=DEV).unsqueeze(1)
    blocks = torch.arange(c["D"] // BLOCK[fmt], device=DEV).unsqueeze(0)
    r, per = rows % c["F_shard"], -(-(c["D"] // BLOCK[fmt]) // 4)
    at = (r // 128 * per + blocks // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + blocks % 4
    byte = s["w_scales"][rows // c["F_shard"], at].long()
    if fmt == "mxfp4":
        step = torch.pow(2.0, (byte - 127).double())
    else:
        e, m = byte // 8, (byte % 8).double() / 8
        step = torch.where(e > 0, (1 + m) * torch.pow(2.0, (e - 7).double()), m * 2.0 ** -6) * s["w_scale"].double()
    w.view(F, -1, BLOCK[fmt]).mul_(step.unsqueeze(2))
    x = s["x"].double()
    if c["op"] == "product8":
        x = exact_values(x, "mxfp8", None)
    return x @ w.t()
