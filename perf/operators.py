"""Cases that time and check the sharded training step's operators: the AdamW
step with 32- and 8-bit states, the global gradient norm with its clip
coefficient, the microscaled 4-bit quantisation and the 4-bit all-gather
product.

``run`` computes each operator in plain torch operations in 32 bits, or, with
``own`` set, makes the calls a user of this package makes.  Both start from
the same buffers.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
BETAS, EPS, LR, DECAY = (0.9, 0.95), 1e-8, 3e-4, 0.1
START = 100          # steps already taken: the states are those of a run under way
QBLOCK = 256         # elements that share one scale of an 8-bit state
MAX_NORM = 1.0
BLOCK = {"mxfp4": 32, "nvfp4": 16}
NAN = float("nan")


# --- tensor lists ----------------------------------------------------------------

def gpt2_small(layers=12, d=768, vocab=50257, ctx=1024):
    """(matrices, vectors) of a GPT-2-small-shaped model: the first decay, the second do not."""
    mats, vecs = [vocab * d, ctx * d], [d, d]
    for _ in range(layers):
        mats += [3 * d * d, d * d, 4 * d * d, 4 * d * d]
        vecs += [d, d, 3 * d, d, d, d, 4 * d, d]
    return mats, vecs


def sizes(c):
    """(decayed, undecayed) element counts of a case's tensors."""
    if c["layout"] == "gpt2":
        return gpt2_small()
    if c["layout"] == "vectors":
        return [], gpt2_small()[1]
    if c["layout"] == "layer":
        mats, vecs = gpt2_small(layers=1)
        return mats[2:], vecs[2:]
    if c["layout"] == "shards":
        return [c["elems"] // c["tensors"]] * c["tensors"], []
    rng = random.Random(c["elems"] * 1000 + c["tensors"])   # "odd": ragged sizes that sum to about elems
    parts = [rng.random() ** 2 + 1e-3 for _ in range(c["tensors"])]
    ns = [max(1, int(c["elems"] * p / sum(parts))) for p in parts]
    cut = (len(ns) + 1) // 2
    return ns[:cut], ns[cut:]


def place(c):
    """Offsets of the tensors in one flat buffer, its length, and where the undecayed ones begin."""
    dec, rest = sizes(c)
    pad = QBLOCK if c.get("states") == "8bit" else 1
    offs, at = [], 0
    for n in dec + rest:
        offs.append(at)
        at += -(-n // pad) * pad
    split = offs[len(dec)] if rest else at
    return dec + rest, offs, at, split


def views(flat, ns, offs):
    return [flat[o:o + n] for n, o in zip(ns, offs)]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed % (1 << 62))


def filled(ns, offs, flat):
    """Zeroes the padding between the tensors of a flat buffer."""
    for n, o, nxt in zip(ns, offs, offs[1:] + [flat.numel()]):
        flat[o + n:nxt] = 0
    return flat


def dtype(word):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[word]


# --- the cases ---------------------------------------------------------------------

def listed():
    return [
        # the biases and norms of a GPT-2-small-shaped model: 98 vectors, all launch latency
        {"name": "adamw vectors", "op": "adamw", "layout": "vectors", "states": "f32", "param": "f32", "grad": "f32", "copy": True},
        # the whole GPT-2-small-shaped model of the DDP benchmark, fp32 masters with a bf16 copy
        {"name": "adamw gpt2", "op": "adamw", "layout": "gpt2", "states": "f32", "param": "f32", "grad": "f32", "copy": True},
        # ragged tensors packed back to back at odd offsets, bf16 parameters and gradients
        {"name": "adamw ragged bf16", "op": "adamw", "layout": "odd", "elems": 30000001, "tensors": 61, "states": "f32", "param": "bf16", "grad": "bf16", "copy": False},
        # one transformer layer's tensors with 8-bit states
        {"name": "adamw8 layer", "op": "adamw", "layout": "layer", "states": "8bit", "param": "f32", "grad": "f32", "copy": True},
        # eight ranks' shards of 8 Mi elements (the FSDP gradient benchmark), bf16 gradients
        {"name": "adamw8 shards", "op": "adamw", "layout": "shards", "elems": 8 << 23, "tensors": 8, "states": "8bit", "param": "f32", "grad": "bf16", "copy": True},
        # clip before a small step: one layer's gradients
        {"name": "norm layer", "op": "norm", "layout": "layer", "grad": "f32"},
        # clip before the GPT-2-small step
        {"name": "norm gpt2", "op": "norm", "layout": "gpt2", "grad": "f32"},
        # activations of the small all-gather product
        {"name": "mx quantize 128x512", "op": "quantize", "rows": 128, "cols": 512, "format": "mxfp4", "transpose": False},
        # a layer's activations for the weight gradient: blocks run along the tokens
        {"name": "nv quantize t 8192x4096", "op": "quantize", "rows": 8192, "cols": 4096, "format": "nvfp4", "transpose": True},
        # the small all-gather product
        {"name": "mx product 128x512x512", "op": "product", "M": 128, "D": 512, "K": 8, "F_shard": 64, "format": "mxfp4"},
        # one token through the large layer: all weight traffic
        {"name": "nv product 1x4096x4096", "op": "product", "M": 1, "D": 4096, "K": 8, "F_shard": 512, "format": "nvfp4"},
        # the large all-gather product
        {"name": "nv product 8192x4096x4096", "op": "product", "M": 8192, "D": 4096, "K": 8, "F_shard": 512, "format": "nvfp4"},
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "adamw8", "norm", "quantize", "product"])
    if op in ("adamw", "adamw8", "norm"):
        c = {"op": "norm" if op == "norm" else "adamw", "layout": "odd", "elems": log_int(rng, 3000, 120000000),
             "tensors": log_int(rng, 1, 300), "grad": rng.choice(["f32", "bf16"])}
        if op != "norm":
            c.update(states="8bit" if op == "adamw8" else "f32", param=rng.choice(["f32", "f32", "bf16"]))
            c["copy"] = c["param"] == "f32" and rng.random() < 0.5
        return c
    fmt = rng.choice(["mxfp4", "nvfp4"])
    if op == "quantize":
        t = rng.random() < 0.5
        a, b = log_int(rng, 1, 8192), 32 * log_int(rng, 1, 128)     # b: along the blocks
        return {"op": "quantize", "rows": b if t else a, "cols": a if t else b, "format": fmt, "transpose": t}
    return {"op": "product", "M": log_int(rng, 1, 8192), "D": 32 * log_int(rng, 2, 128), "K": rng.choice([1, 2, 4, 8]),
            "F_shard": 16 * log_int(rng, 1, 32), "format": fmt}


# --- what a program has in hand -----------------------------------------------------

def start_values(c, seed):
    """Parameters, gradients and 32-bit states of a run under way, in flat buffers."""
    ns, offs, total, split = place(c)
    g = gen(seed)
    grad = filled(ns, offs, torch.randn(total, device=DEV, generator=g) * 1e-3).to(dtype(c["grad"]))
    if c["op"] == "norm":
        return ns, offs, split, None, grad, None, None
    param = filled(ns, offs, torch.randn(total, device=DEV, generator=g) * 0.02).to(dtype(c["param"]))
    m = filled(ns, offs, torch.randn(total, device=DEV, generator=g) * 3e-4)
    v = filled(ns, offs, torch.randn(total, device=DEV, generator=g).mul_(1e-3).square_() + 1e-10)
    return ns, offs, split, param, grad, m, v


def prepare(c, seed):
    if c["op"] in ("adamw", "norm"):
        ns, offs, split, param, grad, m, v = start_values(c, seed)
        s = {"c": c, "grad": grad}
        grads = views(grad, ns, offs)
        if c["op"] == "norm":
            if own:
                from ring_allreduce_gradient_gb300 import optim
                s["norm"] = optim.GradNorm(grads, MAX_NORM)
            return s
        s.update(param=param, split=split, t=START, coef=torch.full((1,), 0.75, device=DEV))
        s["copy"] = torch.zeros(param.numel(), dtype=torch.bfloat16, device=DEV) if c["copy"] else None
        if c["states"] == "f32":
            s.update(m=m, v=v)
        else:
            s["m8"], s["m_scale"] = encode8(m)
            s["r8"], s["r_scale"] = encode8(v.sqrt(), v > 0)
        if own:
            from ring_allreduce_gradient_gb300 import optim
            cut = sum(1 for o in offs if o < split)
            kw = {"copies": views(s["copy"], ns, offs)} if c["copy"] else {}
            if c["states"] == "f32":
                kw.update(exp_avg=views(m, ns, offs), exp_avg_sq=views(v, ns, offs))
            else:
                nb, bo = [-(-n // QBLOCK) for n in ns], [o // QBLOCK for o in offs]
                kw.update(exp_avg=views(s["m8"], ns, offs), exp_avg_scale=views(s["m_scale"], nb, bo),
                          exp_avg_sq=views(s["r8"], ns, offs), exp_avg_sq_scale=views(s["r_scale"], nb, bo))
            s["opt"] = optim.AdamW(views(param, ns, offs), grads, lr=LR, betas=BETAS, eps=EPS,
                                   weight_decay=[DECAY] * cut + [0.0] * (len(ns) - cut), states=c["states"], step=START, **kw)
        return s
    g = gen(seed)
    fmt = c["format"]
    if c["op"] == "quantize":
        x = (torch.randn(c["rows"], c["cols"], device=DEV, generator=g) * 0.02).to(torch.bfloat16)
        return {"c": c, "x": x, "scale": tensor_scale(x) if fmt == "nvfp4" else None}
    # activations with a few loud channels, calibrated once; weights laid out once
    x = torch.randn(c["M"], c["D"], device=DEV, generator=g)
    x = (x * (1 + 10 * (torch.rand(c["D"], device=DEV, generator=g) > 0.99))).to(torch.bfloat16)
    w = torch.randn(c["K"] * c["F_shard"], c["D"], device=DEV, generator=g) * 0.02
    wt = tensor_scale(w) if fmt == "nvfp4" else None
    codes, scales = encode4(w, fmt, wt)
    packed = pack4(codes)
    tiled = tile_scales(scales, c["K"], c["F_shard"])
    s = {"c": c, "x": x, "x_scale": tensor_scale(x) if fmt == "nvfp4" else None, "w": packed, "w_scales": tiled, "w_scale": wt}
    if own:
        from ring_allreduce_gradient_gb300 import mx4
        s["shards"] = [mx4.Mx4Tensor(a, b, c["F_shard"], c["D"], fmt, wt) for a, b in zip(packed.chunk(c["K"]), tiled.unbind(0))]
    return s


# --- plain forms ----------------------------------------------------------------------

def encode8(x, keep=None):
    """8-bit e4m3 codes with one fp32 scale per block; what `keep` marks does not fall to zero."""
    b = x.view(-1, QBLOCK)
    top = b.abs().amax(1)
    codes = b * torch.where(top > 2.0 ** -110, top.reciprocal() * 448.0, 0.0)[:, None]
    if keep is not None:
        codes = torch.where(keep.view(-1, QBLOCK), codes.clamp(min=2.0 ** -9), codes)
    return codes.clamp(-448, 448).to(torch.float8_e4m3fn).view(-1), top * (1.0 / 448.0)


def decode8(codes, scale):
    return (codes.float().view(-1, QBLOCK) * scale[:, None]).view(-1)


def plain_adamw(s):
    c, cut = s["c"], s["split"]
    s["t"] += 1
    fix1, fix2 = 1 - BETAS[0] ** s["t"], 1 - BETAS[1] ** s["t"]
    m = s["m"] if c["states"] == "f32" else decode8(s["m8"], s["m_scale"])
    v = s["v"] if c["states"] == "f32" else decode8(s["r8"], s["r_scale"]).square()
    g = s["grad"].float() * s["coef"]
    m = m * BETAS[0] + g * (1 - BETAS[0])
    v = v * BETAS[1] + g * g * (1 - BETAS[1])
    p = s["param"].float()
    p = torch.cat([p[:cut] * (1 - LR * DECAY), p[cut:]])
    p = p - (LR / fix1) * (m / (v.sqrt() * (1 / math.sqrt(fix2)) + EPS))
    s["param"].copy_(p)
    out = {"param": s["param"]}
    if s["copy"] is not None:
        out["copy"] = s["copy"].copy_(p)
    if c["states"] == "f32":
        out.update(m=s["m"].copy_(m), v=s["v"].copy_(v))
    else:
        s["m8"], s["m_scale"] = encode8(m)
        s["r8"], s["r_scale"] = encode8(v.sqrt(), v > 0)
        out.update(m=s["m8"], m_scale=s["m_scale"], r=s["r8"], r_scale=s["r_scale"])
    return out


def plain_norm(s):
    norm = s["grad"].float().square().sum().sqrt()
    coef = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
    return {"norm": norm.view(1), "coef": torch.where(torch.isfinite(norm), coef, NAN).view(1)}


def tensor_scale(x):
    """The fp32 scale that takes a tensor's largest value to the top of e2m1 times e4m3."""
    return (x.float().abs().amax() * (1.0 / 2688.0)).view(1)


def encode4(x, fmt, scale):
    """4-bit values (as fp32) and one 8-bit scale (as its byte) per block along the rows of x."""
    b = x.float().unflatten(1, (-1, BLOCK[fmt]))
    top = b.abs().amax(2)
    if fmt == "mxfp4":      # a power of two: floor(log2(largest)) - 2
        e = (torch.frexp(top)[1] - 3).clamp(-127, 127)
        e = torch.where(top > 0, e, -127)
        byte, step = (e + 127).to(torch.uint8), torch.ldexp(torch.ones_like(top), e)
    else:
        f8 = (top * (1.0 / 6.0) / scale).clamp(max=448.0).to(torch.float8_e4m3fn)
        byte, step = f8.view(torch.uint8), f8.float() * scale
    y = torch.where(step[..., None] > 0, b / step[..., None], 0.0)
    a = y.abs()
    unit = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = ((a / unit).round() * unit).clamp(max=6.0).copysign(y)
    return q.flatten(1), byte


def steps_of(byte, fmt, scale):
    if fmt == "mxfp4":
        return torch.ldexp(torch.ones(byte.shape, device=byte.device), byte.to(torch.int32) - 127)
    return byte.view(torch.float8_e4m3fn).float() * scale


def decode4(q, byte, fmt, scale):
    return (q.unflatten(1, (-1, BLOCK[fmt])) * steps_of(byte, fmt, scale)[..., None]).flatten(1)


def magnitudes(device):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)


def pack4(q):
    """Two values a byte, the first in the low half; bit 3 is the sign."""
    code = torch.bucketize(q.abs(), magnitudes(q.device)).to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def unpack4(packed):
    code = torch.stack([packed & 15, packed >> 4], 2).flatten(1).long()
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


def plain_quantize(s):
    c = s["c"]
    q, byte = encode4(s["x"].t() if c["transpose"] else s["x"], c["format"], s["scale"])
    return decode4(q, byte, c["format"], s["scale"]).to(torch.bfloat16)


def plain_product(s):
    c, fmt = s["c"], s["c"]["format"]
    q, byte = encode4(s["x"], fmt, s["x_scale"])
    x = decode4(q, byte, fmt, s["x_scale"])
    w = decode4(unpack4(s["w"]), untile_scales(s["w_scales"], c["K"], c["F_shard"], c["D"] // BLOCK[fmt]), fmt, s["w_scale"])
    return (x @ w.t()).to(torch.bfloat16)


# --- one pass --------------------------------------------------------------------------

def run(s):
    c = s["c"]
    if not own:
        return {"adamw": plain_adamw, "norm": plain_norm, "quantize": plain_quantize, "product": plain_product}[c["op"]](s)
    if c["op"] == "adamw":
        s["opt"].step(grad_scale=s["coef"])
        out = {"param": s["param"]}
        if s["copy"] is not None:
            out["copy"] = s["copy"]
        if c["states"] == "f32":
            out.update(m=s["m"], v=s["v"])
        else:
            out.update(m=s["m8"], m_scale=s["m_scale"], r=s["r8"], r_scale=s["r_scale"])
        return out
    if c["op"] == "norm":
        norm, coef = s["norm"]()
        return {"norm": norm, "coef": coef}
    from ring_allreduce_gradient_gb300 import mx4
    if c["op"] == "quantize":
        q = mx4.quantize(s["x"], c["format"], tensor_scale=s["scale"], transpose=c["transpose"])
        return mx4.dequantize(q, torch.bfloat16)
    return mx4.linear(s["x"], s["shards"], x_scale=s["x_scale"])


def work(c):
    if c["op"] in ("adamw", "norm"):
        n = sum(sum(part) for part in sizes(c))
        wide = {"f32": 4, "bf16": 2}
        if c["op"] == "norm":
            return {"bytes": n * wide[c["grad"]] + 8, "flops": 2 * n}
        state = 16 if c["states"] == "f32" else 4 + 16 / QBLOCK
        return {"bytes": n * (2 * wide[c["param"]] + wide[c["grad"]] + state + (2 if c["copy"] else 0)), "flops": 15 * n}
    per = 0.5 + 1 / BLOCK[c["format"]]      # bytes of a value in 4 bits with its share of a scale
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (2 + per + 2), "flops": 4 * n}
    M, D, F = c["M"], c["D"], c["K"] * c["F_shard"]
    return {"bytes": 2 * M * D + per * F * D + 2 * M * F, "flops": 2 * M * D * F}


# --- the definitions in 64 bits --------------------------------------------------------

def power_below(a):
    """The largest power of two that is no larger than a (a > 0); exact, where a logarithm may round."""
    return a / (2 * torch.frexp(a).mantissa)


def nearest_e4m3(x):
    """Nearest e4m3 value, ties to even, saturated, of 64-bit values."""
    a = x.abs()
    grid = power_below(a.clamp(min=2.0 ** -6)) / 8
    return (torch.round(a / grid) * grid).clamp(max=448.0) * torch.sign(x)


def nearest_e2m1(x):
    a = x.abs()
    grid = power_below(a.clamp(min=1.0, max=4.0)) / 2
    return (torch.round(a / grid) * grid).clamp(max=6.0) * torch.sign(x)


def exact_codes8(x, positive=None):
    b = x.reshape(-1, QBLOCK)
    top = b.abs().max(1, keepdim=True).values
    y = b / torch.where(top == 0, 1.0, top) * 448.0
    if positive is not None:
        y = torch.where(positive.reshape(-1, QBLOCK), y.clamp(min=2.0 ** -9), y)
    return nearest_e4m3(y).reshape(-1), top.reshape(-1) / 448.0


def exact_values4(x, fmt, scale):
    """The values that 64-bit x [rows, cols] stands for in 4 bits with blocks along its rows."""
    b = x.reshape(x.shape[0], -1, BLOCK[fmt])
    top = b.abs().max(2, keepdim=True).values
    if fmt == "mxfp4":
        step = power_below(top.clamp(min=2.0 ** -125)) / 4
    else:
        step = nearest_e4m3(top / (6.0 * scale)) * scale
    return (nearest_e2m1(b / torch.where(step == 0, 1.0, step)) * step).reshape(x.shape)


def exact(c, seed):
    if c["op"] in ("adamw", "norm"):
        ns, offs, split, param, grad, m, v = start_values(c, seed)
        g = grad.double()
        if c["op"] == "norm":
            norm = torch.linalg.vector_norm(g).view(1)
            return {"norm": norm, "coef": torch.minimum(MAX_NORM / (norm + 1e-6), torch.ones_like(norm))}
        g.mul_(0.75)
        if c["states"] == "f32":
            m, v = m.double(), v.double()
        else:
            m8, ms = encode8(m)
            r8, rs = encode8(v.sqrt(), v > 0)
            blocks = lambda codes, sc: (codes.double().reshape(-1, QBLOCK) * sc.double().reshape(-1, 1)).reshape(-1)  # noqa: E731
            m, v = blocks(m8, ms), blocks(r8, rs).pow(2)
        t = START + 1
        m.mul_(BETAS[0]).add_(g, alpha=1 - BETAS[0])
        v.mul_(BETAS[1]).addcmul_(g, g, value=1 - BETAS[1])
        p = param.double()
        p[:split] -= LR * DECAY * p[:split]
        p -= LR * (m / (1 - BETAS[0] ** t)) / ((v / (1 - BETAS[1] ** t)).sqrt() + EPS)
        out = {"param": p}
        if c["copy"]:
            out["copy"] = p
        if c["states"] == "f32":
            out.update(m=m, v=v)
        else:
            out["m"], out["m_scale"] = exact_codes8(m)
            out["r"], out["r_scale"] = exact_codes8(v.sqrt(), v > 0)
        return out
    s = prepare(c, seed)
    if c["op"] == "quantize":
        x = s["x"].double()
        sc = s["scale"].double() if s["scale"] is not None else None
        return exact_values4(x.t().contiguous() if c["transpose"] else x, c["format"], sc)
    fmt = c["format"]
    x = exact_values4(s["x"].double(), fmt, s["x_scale"].double() if s["x_scale"] is not None else None)
    w = decode4(unpack4(s["w"]).double(), untile_scales(s["w_scales"], c["K"], c["F_shard"], c["D"] // BLOCK[fmt]), fmt, None if fmt == "mxfp4" else s["w_scale"].double())
    return x @ w.t()
