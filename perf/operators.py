"""Cases of the operators around the convolutions: group norm with an
activation, counter-based dropout, and the replay cache.

Tensors are channels last in the library's order [H][W][N][C]. `run` computes
an operator in its plain form (elementary torch operations in fp32), or, with
`own` set, by the package's entry points.
"""
import math

import numpy as np
import torch

own = False

ACTS = ("none", "relu", "silu", "gelu")
E4M3, E5M2, E2M3, E3M2, E2M1 = 0, 1, 2, 3, 4
FMTS = {"e4m3": E4M3, "e5m2": E5M2, "e2m3": E2M3, "e3m2": E3M2, "e2m1": E2M1}
# (bits, exponent bits, mantissa bits, bias, exponent of the largest binade, largest value)
ELEM = {
    "e4m3": (8, 4, 3, 7, 8, 448.0),
    "e5m2": (8, 5, 2, 15, 15, 57344.0),
    "e2m3": (6, 2, 3, 1, 2, 7.5),
    "e3m2": (6, 3, 2, 3, 4, 28.0),
    "e2m1": (4, 2, 1, 1, 2, 6.0),
}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
EPS = 1e-5


def _norm(name, op, h, w, n, c, groups, act, p, out, bp=32):
    return {"name": name, "op": op, "h": h, "w": w, "n": n, "c": c, "groups": groups, "act": act, "p": p, "out": out,
            "bp": bp}


def _drop(name, h, w, n, c, p, residual, out, bp=32):
    return {"name": name, "op": "dropout", "h": h, "w": w, "n": n, "c": c, "p": p, "residual": residual, "out": out,
            "bp": bp}


def _cache(name, op, slots, h, w, c, fmt, write, read, out, bp=1):
    return {"name": name, "op": op, "slots": slots, "h": h, "w": w, "c": c, "fmt": fmt, "write": write, "read": read,
            "out": out, "bp": bp}


def listed():
    return [
        # the forward-only small layer (2 samples, 32 channels, 16 x 16): one call's latency
        _norm("norm_small", "norm", 16, 16, 2, 32, 8, "silu", 0.0, "f32", 1),
        # the detector's 3x3 layer at batch 16: the next convolution's activation, quantized once in squares
        _norm("norm_detector_e4m3", "norm", 80, 80, 16, 64, 16, "silu", 0.1, "e4m3"),
        # the stride-2 stress layer's input, the largest activation of the workloads
        _norm("norm_stress_f32", "norm", 160, 160, 32, 128, 32, "silu", 0.0, "f32"),
        # gradients of the same layers; the replay head's goes on to the previous convolution as MX codes
        _norm("norm_grad_replay_e5m2", "norm_backward", 20, 20, 128, 256, 32, "silu", 0.2, "e5m2"),
        _norm("norm_grad_detector_f32", "norm_backward", 80, 80, 16, 64, 16, "silu", 0.1, "f32"),
        # odd extents, a channel count that is no multiple of four, five samples
        _norm("norm_grad_odd_f32", "norm_backward", 19, 23, 5, 90, 9, "gelu", 0.0, "f32"),
        # a residual branch at the stress layer's output
        _drop("dropout_stress_f32", 80, 80, 32, 256, 0.1, True, "f32"),
        # the detector layer's gradient through dropout, quantized for the backward products
        _drop("dropout_detector_e5m2", 80, 80, 16, 64, 0.1, False, "e5m2"),
        # a few odd rows
        _drop("dropout_odd_f32", 7, 9, 3, 45, 0.5, False, "f32"),
        # a batch of new latents stored in a replay memory of 1,024 samples
        _cache("cache_write_e4m3", "cache_write", 1024, 20, 20, 256, "e4m3", 128, 0, "e4m3"),
        # a latent replay batch: 16 new samples stored as 4-bit codes, 128 read back as values
        _cache("cache_replay_e2m1", "cache_replay", 4096, 20, 20, 256, "e2m1", 16, 128, "f32"),
        # a batch read back as the squares that the backward products need
        _cache("cache_read_mx_e3m2", "cache_read_mx", 1024, 20, 20, 256, "e3m2", 0, 128, "e4m3", 32),
    ]


LARGEST = 160 * 160 * 32 * 128  # elements of the largest listed tensor


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    c = _log_int(rng, 3, 512)
    if rng.random() < 0.6:  # most layers have a multiple of 8 or 32 channels
        unit = rng.choice((8, 32))
        c = max(unit, c // unit * unit)
    n, h, w = _log_int(rng, 1, 128), _log_int(rng, 1, 160), _log_int(rng, 1, 160)
    while h * w * n * c > LARGEST // 2:
        h, w = max(1, h // 2), max(1, w * 2 // 3)
    op = rng.choice(("norm", "norm_backward", "dropout", "cache_write", "cache_replay", "cache_read_mx"))
    if op in ("norm", "norm_backward"):
        while h * w * c < 64:  # a handful of elements has no statistics: its gradient is rounding noise
            h, w = 2 * h + 1, w + 1
        groups = rng.choice([g for g in range(1, min(c, 64) + 1) if c % g == 0 and h * w * c >= 64 * g])
        out = rng.choice(("f32", "e4m3" if op == "norm" else "e5m2"))
        case = _norm("", op, h, w, n, c, groups, rng.choice(ACTS), rng.choice((0.0, 0.1, 0.25)), out,
                     rng.choice((1, 32)))
    elif op == "dropout":
        out = rng.choice(("f32", "e4m3", "e5m2"))
        case = _drop("", h, w, n, c, round(rng.uniform(0.02, 0.9), 3), out == "f32" and rng.random() < 0.5, out,
                     rng.choice((1, 32)))
    else:
        slots = _log_int(rng, 1, 2048)
        while slots * h * w * c > 1 << 27:
            slots = max(1, slots // 2)
            h, w = max(1, h * 2 // 3), max(1, w * 2 // 3)
        fmt = rng.choice(("e4m3", "e5m2")) if op == "cache_write" else rng.choice(sorted(FMTS))
        write = 0 if op == "cache_read_mx" else min(slots, _log_int(rng, 1, 128))
        read = 0 if op == "cache_write" else n
        out = {"cache_write": fmt, "cache_replay": "f32", "cache_read_mx": rng.choice(("e4m3", "e5m2"))}[op]
        case = _cache("", op, slots, h, w, c, fmt, write, read, out, rng.choice((1, 32)))
    del case["name"]
    return case


# ---- inputs -------------------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _norm_inputs(case, seed):
    """x with its own mean and spread in every channel, as a convolution leaves it, gamma, beta, and for the backward pass
    dy (with one entry in a thousand a hundred times larger) and the statistics that the forward pass kept."""
    g = _generator(seed)
    h, w, n, c, groups = (case[k] for k in ("h", "w", "n", "c", "groups"))
    x = _normal(g, h, w, n, c)
    x.mul_(0.5 + torch.rand(c, generator=g, device="cuda")).add_(_normal(g, c))
    t = {"x": x, "gamma": 1 + 0.1 * _normal(g, c), "beta": 0.1 * _normal(g, c)}
    if case["op"] == "norm_backward":
        dy = _normal(g, h, w, n, c).mul_(1e-3)
        dy.mul_(1 + 99 * (torch.rand(h, w, n, c, generator=g, device="cuda") < 1e-3))
        xg = x.view(h * w, n, groups, c // groups)
        mean = xg.mean(dim=(0, 3), dtype=torch.float64)
        var = xg.var(dim=(0, 3), correction=0).double()
        t |= {"dy": dy, "mean": mean.float(), "rstd": torch.rsqrt(var + EPS).float()}
    return t


def _codes(g, fmt, shape, c):
    """Random codes of a format in [..., Cpad] bytes (no infinity or NaN; zeros past channel c)."""
    bits = ELEM[fmt][0]
    q = torch.randint(0, 1 << bits, (*shape, (c + 31) // 32 * 32), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == "e4m3":
        q[(q & 0x7F) == 0x7F] = 0
    elif fmt == "e5m2":
        q[(q & 0x7C) == 0x7C] = 0
    q[..., c:] = 0
    return q


def _pack(q, bits):
    """Codes [..., 32 k] as packed bytes: little-endian runs of 32 codes."""
    if bits == 8:
        return q
    if bits == 4:
        return q[..., 0::2] | (q[..., 1::2] << 4)
    a, b, c, d = (q[..., i::4].to(torch.int32) for i in range(4))
    word = a | (b << 6) | (c << 12) | (d << 18)  # four codes in three bytes
    return torch.stack([word & 255, (word >> 8) & 255, word >> 16], dim=-1).to(torch.uint8).flatten(-2)


def _unpack(b, bits):
    if bits == 8:
        return b
    if bits == 4:
        return torch.stack([b & 15, b >> 4], dim=-1).flatten(-2)
    b = b.unflatten(-1, (-1, 3)).to(torch.int32)
    word = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
    return torch.stack([(word >> s) & 63 for s in (0, 6, 12, 18)], dim=-1).to(torch.uint8).flatten(-2)


def _cache_inputs(case, seed):
    """A filled cache, the samples that are stored next (post-ReLU latents) and the slots that are written and read."""
    g = _generator(seed)
    slots, h, w, c, fmt = (case[k] for k in ("slots", "h", "w", "c", "fmt"))
    q = _codes(g, fmt, (slots, h, w), c)
    ncb = (c + 31) // 32
    top = 127 - ELEM[fmt][4]
    scales = torch.randint(top - 2, top + 3, (slots, h, w, ncb), generator=g, device="cuda", dtype=torch.uint8)
    t = {"codes": _pack(q, ELEM[fmt][0]).contiguous(), "scales": scales}
    order = torch.randperm(slots, generator=g, device="cuda")
    if case["write"]:
        t["new"] = _normal(g, h, w, case["write"], c).relu_()
        t["to"] = order[: case["write"]].to(torch.int32)
    if case["read"]:
        at = torch.randint(0, slots, (case["read"],), generator=g, device="cuda")
        if case["write"]:  # some of the new samples are replayed at once
            k = min(case["write"], case["read"]) // 2
            at[:k] = order[:k]
        t["from"] = at.to(torch.int32)
    return t


def prepare(case, seed):
    s = {"case": case, "seed": seed * 0x9E3779B97F4A7C15 & (1 << 64) - 1}
    op = case["op"]
    if op.startswith("cache"):
        t = _cache_inputs(case, seed)
        h, w, c, count = case["h"], case["w"], case["c"], case["read"]
    else:
        h, w, c, count = case["h"], case["w"], case["c"], case["n"]
        if op == "dropout":
            g = _generator(seed)
            t = {"x": _normal(g, h, w, count, c)}
            if case["residual"]:
                t["residual"] = _normal(g, h, w, count, c)
        else:
            t = _norm_inputs(case, seed)
    s |= t
    # the buffers that a step keeps for its results
    if count and case["out"] == "f32":
        s["out"] = torch.empty(h, w, count, c, device="cuda")
    elif count:
        ncb, bp = (c + 31) // 32, case["bp"]
        s["out_codes"] = torch.empty(h, w, count, ncb * 32, dtype=torch.uint8, device="cuda")
        s["out_scales"] = torch.empty(h, w, (count + bp - 1) // bp, ncb, dtype=torch.uint8, device="cuda")
    if op == "norm":
        s["mean"] = torch.empty(count, case["groups"], device="cuda")
        s["rstd"] = torch.empty_like(s["mean"])
    if op == "norm_backward":
        s["dgamma"], s["dbeta"] = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    return s


# ---- the plain form -----------------------------------------------------------------------------
MASK = 0xFFFFFFFF


def _halves(rows, c, seed):
    """The 16-bit random numbers of elements (row, channel): half word c % 8 of Philox4x32-10 at counter (row, c / 8, 1, 0)
    with the seed as its key. int64 products wrap, and their bits are what counts."""
    c0 = torch.arange(rows, device="cuda")[:, None]
    c1 = torch.arange((c + 7) // 8, device="cuda")[None, :]
    c2, c3 = torch.ones_like(c1), torch.zeros_like(c1)
    k0, k1 = seed & MASK, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (p1 >> 32 & MASK) ^ c1 ^ k0, p1 & MASK, (p0 >> 32 & MASK) ^ c3 ^ k1, p0 & MASK
        k0, k1 = k0 + 0x9E3779B9 & MASK, k1 + 0xBB67AE85 & MASK
    u = torch.stack([v for q in (c0, c1, c2, c3) for v in (q & 0xFFFF, q >> 16)], dim=-1)
    return u.flatten(-2)[:, :c]


def _dropped(x, p, seed):
    """x [..., C] with a share p of its elements zero and the others scaled."""
    q = math.floor(p * 65536 + 0.5)
    if q == 0:
        return x
    keep = _halves(x.numel() // x.shape[-1], x.shape[-1], seed).view(x.shape) >= q
    return torch.where(keep, x * (65536.0 / (65536 - q)), torch.zeros_like(x))


def _act(u, act):
    if act == "relu":
        return torch.where(u < 0, torch.zeros_like(u), u)
    if act == "silu":
        return u / (1 + torch.exp(-u))
    if act == "gelu":
        return 0.5 * u * (1 + torch.erf(u * math.sqrt(0.5)))
    return u


def _act_slope(u, act):
    if act == "relu":
        return (u > 0).to(u.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-u))
        return s * (1 + u * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(u * math.sqrt(0.5))) + u * torch.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)
    return torch.ones_like(u)


def _blocks(x, bp):
    """x [H][W][N][C] padded with zeros to [H*W][blocks][bp][channel blocks][32]."""
    h, w, n, c = x.shape
    x = torch.nn.functional.pad(x, (0, -c % 32, 0, -n % bp))
    return x.view(h * w, x.shape[2] // bp, bp, x.shape[3] // 32, 32)


def _scales(x, fmt, bp):
    """Scale bytes [H*W][blocks][channel blocks] of x, and the factor 2^(127 - byte) of each block."""
    amax = _blocks(x, bp).abs().amax(dim=(2, 4)).view(torch.int32)
    byte = ((amax >> 23) - ELEM[fmt][4]).clamp_(min=0)
    byte = torch.where(amax >= 0x7F800000, 255, byte)
    inv = torch.where(byte == 255, 0, (254 - byte) << 23).to(torch.int32).view(torch.float32)
    return byte, inv


def _scaled(x, fmt, bp):
    """The blocks of x over their scales, saturated, and the scale bytes."""
    byte, inv = _scales(x, fmt, bp)
    top = ELEM[fmt][5]
    v = (_blocks(x, bp) * inv[:, :, None, :, None]).clamp_(-top, top)
    return torch.where((byte == 255)[:, :, None, :, None], torch.zeros_like(v), v), byte


def _quantized(x, fmt, bp):
    """x [H][W][N][C] as 8-bit codes (float8 values [H][W][N][Cpad]) and scales (powers of two)."""
    h, w, n, _ = x.shape
    v, byte = _scaled(x, fmt, bp)
    codes = v.to(FP8[fmt]).view(torch.uint8).flatten(-2).flatten(1, 2)[:, :n].contiguous()
    scales = byte.to(torch.uint8).view(h, w, *byte.shape[1:])
    return {"codes": codes.view(h, w, n, -1).view(FP8[fmt]), "scales": scales.view(torch.float8_e8m0fnu)}


def _power(e):
    """2^e in fp32 for int32 e in [-127, 127], exactly (2^-127, the scale of a block of zeros, as 0)."""
    return ((e + 127) << 23).view(torch.float32)


def _value_table(fmt):
    bits, eb, mb, bias, _, _ = ELEM[fmt]
    code = torch.arange(1 << bits, device="cuda", dtype=torch.int32)
    e, m = (code >> mb) & ((1 << eb) - 1), (code & ((1 << mb) - 1)).float()
    mag = torch.where(e == 0, m * 2.0 ** (1 - bias - mb), (1 + m * 2.0 ** -mb) * _power(e - bias))
    return torch.where(code >> (bits - 1) == 1, -mag, mag)


def _to_codes(v, fmt):
    """Codes of saturated block values: each to the nearest of the format's values, ties to the even code."""
    bits, _, mb, bias, _, _ = ELEM[fmt]
    if fmt in FP8:
        return v.to(FP8[fmt]).view(torch.uint8)
    a = v.abs()
    e = ((a.view(torch.int32) >> 23) - 127).clamp_(min=1 - bias)  # exponent of the grid's binade
    m = torch.round(a * _power(mb - e)).to(torch.int32)  # mantissa with its leading one; 2 << mb moves on
    mag = ((e + bias - 1) << mb) + m
    sign = torch.signbit(v).to(torch.int32) << (bits - 1)
    return (mag | sign).to(torch.uint8)


def _read(s, slots):
    """Values [H][W][M][C] of the cache's slots."""
    case = s["case"]
    at = slots.long()
    q = _unpack(s["codes"][at], ELEM[case["fmt"]][0]).long()
    scale = _power(s["scales"][at].to(torch.int32) - 127)
    x = _value_table(case["fmt"])[q].unflatten(-1, (-1, 32)) * scale[..., None]
    return x.flatten(-2)[..., : case["c"]].permute(1, 2, 0, 3).contiguous()


def _write(s):
    case = s["case"]
    h, w, n, _ = s["new"].shape
    v, byte = _scaled(s["new"], case["fmt"], 1)
    packed = _pack(_to_codes(v, case["fmt"]).flatten(-2), ELEM[case["fmt"]][0]).view(h, w, n, -1)
    to = s["to"].long()
    s["codes"][to] = packed.permute(2, 0, 1, 3)
    s["scales"][to] = byte.to(torch.uint8).view(h, w, n, -1).permute(2, 0, 1, 3)


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "dropout":
        y = _dropped(s["x"], case["p"], s["seed"])
        if case["residual"]:
            y = y + s["residual"]
        return y if case["out"] == "f32" else _quantized(y, case["out"], case["bp"])
    if op == "norm":
        h, w, n, c = s["x"].shape
        xg = s["x"].view(h * w, n, case["groups"], -1)
        mean = xg.mean(dim=(0, 3))
        d = xg - mean[..., None]
        rstd = 1 / torch.sqrt((d * d).mean(dim=(0, 3)) + EPS)
        u = (d * rstd[..., None]).view(h, w, n, c) * s["gamma"] + s["beta"]
        y = _dropped(_act(u, case["act"]), case["p"], s["seed"])
        y = {"y": y} if case["out"] == "f32" else _quantized(y, case["out"], case["bp"])
        return y | {"mean": mean, "rstd": rstd}
    if op == "norm_backward":
        h, w, n, c = s["x"].shape
        mean, rstd = s["mean"][..., None], s["rstd"][..., None]
        xh = (s["x"].view(h * w, n, case["groups"], -1) - mean) * rstd
        u = xh.view(h, w, n, c) * s["gamma"] + s["beta"]
        g = _dropped(s["dy"], case["p"], s["seed"]) * _act_slope(u, case["act"])
        dbeta = g.sum(dim=(0, 1, 2))
        dgamma = (g * xh.view(h, w, n, c)).sum(dim=(0, 1, 2))
        gg = (g * s["gamma"]).view(xh.shape)
        a, b = gg.mean(dim=(0, 3))[..., None], (gg * xh).mean(dim=(0, 3))[..., None]
        dx = (rstd * (gg - a - xh * b)).view(h, w, n, c)
        dx = {"dx": dx} if case["out"] == "f32" else _quantized(dx, case["out"], case["bp"])
        return dx | {"dgamma": dgamma, "dbeta": dbeta}
    if op == "cache_read_mx":
        return _quantized(_read(s, s["from"]), case["out"], case["bp"])
    _write(s)
    if op == "cache_replay":
        return _read(s, s["from"])
    return {"codes": s["codes"].view(FP8[case["fmt"]]), "scales": s["scales"].view(torch.float8_e8m0fnu)}


# ---- the package's entry points -----------------------------------------------------------------
def _plan(mq, s):
    """What a program keeps between its steps: descriptors, tensor views and a workspace."""
    case, op = s["case"], s["case"]["op"]
    h, w, c = case["h"], case["w"], case["c"]
    count = case["read"] if op.startswith("cache") else case["n"]
    plan = {}
    if "out_codes" in s:
        role = mq.ROLE_GRAD if op == "norm_backward" else mq.ROLE_ACT
        plan["mx"] = mq.MxTensor(s["out_codes"], s["out_scales"], FMTS[case["out"]], case["bp"], role, (h, w, count, c))
    if op.startswith("cache"):
        plan["cache"] = mq.MxCache(s["codes"], s["scales"], FMTS[case["fmt"]], case["slots"], h, w, c)
        return plan
    plan["drop"] = mq.mq_drop(case["p"], s["seed"]) if case["p"] else None
    if op != "dropout":
        plan["norm"] = mq.mq_norm(h, w, count, c, case["groups"], ACTS.index(case["act"]), EPS)
        need = mq.mqconv_group_norm_workspace_bytes(plan["norm"], mq.NORM_BWD if op == "norm_backward" else mq.NORM_FWD)
        plan["ws"] = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    return plan


def _mx_out(s):
    fmt = s["case"]["out"]
    return {"codes": s["out_codes"].view(FP8[fmt]), "scales": s["out_scales"].view(torch.float8_e8m0fnu)}


def _run_own(s):
    import microscaling_quantized_convolution_mxq_amd as mq
    plan = s.get("plan")
    if plan is None:
        plan = s["plan"] = _plan(mq, s)
    case, op = s["case"], s["case"]["op"]
    f32 = case["out"] == "f32"
    if op == "dropout":
        if f32:
            mq.mqconv_dropout(s["x"], plan["drop"], s["out"], residual=s.get("residual"))
            return s["out"]
        mq.mqconv_dropout_mx(s["x"], plan["drop"], plan["mx"])
        return _mx_out(s)
    if op == "norm":
        kept = {"mean": s["mean"], "rstd": s["rstd"]}
        if f32:
            mq.mqconv_group_norm(plan["norm"], s["x"], s["gamma"], s["beta"], s["out"], s["mean"], s["rstd"],
                                 plan["ws"], drop=plan["drop"])
            return {"y": s["out"]} | kept
        mq.mqconv_group_norm_mx(plan["norm"], s["x"], s["gamma"], s["beta"], plan["mx"], s["mean"], s["rstd"],
                                plan["ws"], drop=plan["drop"])
        return _mx_out(s) | kept
    if op == "norm_backward":
        sums = {"dgamma": s["dgamma"], "dbeta": s["dbeta"]}
        if f32:
            mq.mqconv_group_norm_backward(plan["norm"], s["dy"], s["x"], s["gamma"], s["beta"], s["mean"], s["rstd"],
                                          s["out"], s["dgamma"], s["dbeta"], plan["ws"], drop=plan["drop"])
            return {"dx": s["out"]} | sums
        mq.mqconv_group_norm_backward_mx(plan["norm"], s["dy"], s["x"], s["gamma"], s["beta"], s["mean"], s["rstd"],
                                         plan["mx"], s["dgamma"], s["dbeta"], plan["ws"], drop=plan["drop"])
        return _mx_out(s) | sums
    if op == "cache_read_mx":
        mq.mqconv_cache_read_mx(plan["cache"], s["from"], plan["mx"])
        return _mx_out(s)
    mq.mqconv_cache_write(plan["cache"], s["new"], s["to"])
    if op == "cache_replay":
        mq.mqconv_cache_read(plan["cache"], s["from"], s["out"])
        return s["out"]
    return {"codes": s["codes"].view(FP8[case["fmt"]]), "scales": s["scales"].view(torch.float8_e8m0fnu)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- work and exact values ----------------------------------------------------------------------
def _mx_bytes(h, w, n, c, fmt, bp):
    ncb = (c + 31) // 32
    return h * w * (n * ncb * 4 * ELEM[fmt][0] + (n + bp - 1) // bp * ncb)


def work(case):
    op, h, w, c = case["op"], case["h"], case["w"], case["c"]
    count = case["read"] if op.startswith("cache") else case["n"]
    e = h * w * count * c
    out = 4 * e if case["out"] == "f32" else _mx_bytes(h, w, count, c, case["out"], case["bp"])
    if op == "dropout":
        return {"bytes": 4 * e * (2 if case["residual"] else 1) + out, "flops": 2 * e}
    if op == "norm":
        return {"bytes": 4 * e + out + 8 * count * case["groups"] + 8 * c, "flops": 12 * e}
    if op == "norm_backward":
        return {"bytes": 8 * e + out + 8 * count * case["groups"] + 16 * c, "flops": 30 * e}
    stored = _mx_bytes(h, w, case["write"], c, case["fmt"], 1)
    new = 4 * h * w * case["write"] * c + stored + 4 * case["write"]
    fetched = _mx_bytes(h, w, case["read"], c, case["fmt"], 1) + 4 * case["read"] + out if case["read"] else 0
    return {"bytes": new + fetched, "flops": 2 * (e + h * w * case["write"] * c)}


def _exact_keep(rows, c, p, seed):
    """Which elements dropout keeps, by numpy's unsigned integers."""
    q = math.floor(p * 65536 + 0.5)
    low = np.uint64(MASK)
    shift = np.uint64(32)
    a = np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], (rows, (c + 7) // 8)).copy()
    b = np.broadcast_to(np.arange((c + 7) // 8, dtype=np.uint64)[None], a.shape).copy()
    d, e = np.ones_like(a), np.zeros_like(a)
    k = [seed & MASK, seed >> 32]
    for _ in range(10):
        u, v = a * np.uint64(0xD2511F53), d * np.uint64(0xCD9E8D57)
        a, b, d, e = (v >> shift) ^ b ^ np.uint64(k[0]), v & low, (u >> shift) ^ e ^ np.uint64(k[1]), u & low
        k = [(k[0] + 0x9E3779B9) & MASK, (k[1] + 0xBB67AE85) & MASK]
    words = np.stack([a, b, d, e], axis=-1).astype("<u4").view("<u2").reshape(rows, -1)
    return torch.from_numpy(words[:, :c] >= q).cuda()


def _exact_dropped(x, p, seed):
    q = math.floor(p * 65536 + 0.5)
    if q == 0:
        return x
    return x * _exact_keep(x.numel() // x.shape[-1], x.shape[-1], p, seed).view(x.shape) * (65536 / (65536 - q))


def _exact_grid(v, fmt):
    """v rounded to the format's nearest value, ties to an even mantissa, saturated."""
    _, _, mb, bias, _, top = ELEM[fmt]
    e = torch.frexp(v)[1] - 1
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e, min=1 - bias) - mb)
    return (torch.round(v / step) * step).clamp(-top, top)


def _exact_mx(y, fmt, bp):
    """Element values over their block's scale, and the scales, of a 64-bit y: the largest binade of a block goes to the
    largest one of the format."""
    h, w, n, c = y.shape
    full = torch.zeros(h * w, -(-n // bp) * bp, -(-c // 32) * 32, dtype=torch.float64, device=y.device)
    full[:, :n, :c] = y.view(h * w, n, c)
    blk = full.unflatten(2, (-1, 32)).unflatten(1, (-1, bp))
    amax = blk.abs().amax(dim=(2, 4))
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 1 - ELEM[fmt][4], -127).clamp(min=-127)
    scale = torch.ldexp(torch.ones_like(amax), e)
    v = _exact_grid(blk / scale[:, :, None, :, None], fmt)
    return {"codes": v.flatten(-2).flatten(1, 2)[:, :n].reshape(h, w, n, -1), "scales": scale.view(h, w, *scale.shape[1:])}


def _exact_values(fmt, packed, scales, c):
    """Values of packed codes [..., bytes] with line scales [..., channel blocks], bit by bit."""
    bits, eb, mb, bias, _, _ = ELEM[fmt]
    raw = (packed[..., None] >> torch.arange(8, device="cuda", dtype=torch.uint8)) & 1
    raw = raw.flatten(-2).unflatten(-1, (-1, bits)).double()  # [..., codes][bits], lowest bit first
    m = (raw[..., :mb] * 2.0 ** torch.arange(mb, device="cuda")).sum(-1)
    e = (raw[..., mb:mb + eb] * 2.0 ** torch.arange(eb, device="cuda")).sum(-1)
    mag = torch.where(e == 0, m * 2.0 ** (1 - bias - mb), (1 + m / 2 ** mb) * 2.0 ** (e - bias))
    v = mag * (1 - 2 * raw[..., -1])
    return (v.unflatten(-1, (-1, 32)) * 2.0 ** (scales.double()[..., None] - 127)).flatten(-2)[..., :c]


def exact(case, seed):
    op, p = case["op"], case.get("p", 0.0)
    key = seed * 0x9E3779B97F4A7C15 & (1 << 64) - 1
    if op.startswith("cache"):
        t = _cache_inputs(case, seed)
        h, w, c, fmt = case["h"], case["w"], case["c"], case["fmt"]
        stored = _exact_mx(t["new"].double(), fmt, 1) if case["write"] else None
        if op == "cache_write":
            codes, scales = t["codes"].view(FP8[fmt]).double(), t["scales"].view(torch.float8_e8m0fnu).double()
            codes[t["to"].long()] = stored["codes"].permute(2, 0, 1, 3)
            scales[t["to"].long()] = stored["scales"].permute(2, 0, 1, 3)
            return {"codes": codes, "scales": scales}
        at = t["from"].long()
        x = torch.empty(h, w, case["read"], c, dtype=torch.float64, device="cuda")
        for k in range(0, case["read"], 16):
            x[:, :, k:k + 16] = _exact_values(fmt, t["codes"][at[k:k + 16]], t["scales"][at[k:k + 16]], c).permute(1, 2, 0, 3)
        if stored is not None:  # the slots that were written just before
            new = (stored["codes"].unflatten(-1, (-1, 32)) * stored["scales"][..., None]).flatten(-2)[..., :c]
            hit = at[:, None] == t["to"].long()[None]
            found = hit.any(1).nonzero().flatten()
            x[:, :, found] = new[:, :, hit[found].int().argmax(1)]
        return x if case["out"] == "f32" else _exact_mx(x, case["out"], case["bp"])
    if op == "dropout":
        g = _generator(seed)
        shape = tuple(case[k] for k in ("h", "w", "n", "c"))
        y = _exact_dropped(_normal(g, *shape).double(), p, key)
        if case["residual"]:
            y += _normal(g, *shape)
        return y if case["out"] == "f32" else _exact_mx(y, case["out"], case["bp"])
    t = {k: v.double() for k, v in _norm_inputs(case, seed).items()}
    h, w, n, c = t["x"].shape
    d = c // case["groups"]
    per_c = lambda v: v.repeat_interleave(d, dim=1)  # noqa: E731  [N][G] -> [N][C]
    if op == "norm":
        xg = t["x"].view(h * w, n, case["groups"], d)
        var, mean = torch.var_mean(xg, dim=(0, 3), correction=0)
        rstd = (var + EPS) ** -0.5
        u = (t["x"] - per_c(mean)) * (per_c(rstd) * t["gamma"]) + t["beta"]
    else:
        mean, rstd = t["mean"], t["rstd"]
        xh = (t["x"] - per_c(mean)) * per_c(rstd)
        u = xh * t["gamma"] + t["beta"]
    cdf = torch.special.ndtr(u) if case["act"] == "gelu" else None
    if op == "norm":
        y = {"none": lambda: u, "relu": lambda: u.clamp(min=0), "silu": lambda: u * torch.sigmoid(u),
             "gelu": lambda: u * cdf}[case["act"]]()
        y = _exact_dropped(y, p, key)
        y = {"y": y} if case["out"] == "f32" else _exact_mx(y, case["out"], case["bp"])
        return y | {"mean": mean, "rstd": rstd}
    sig = torch.sigmoid(u) if case["act"] == "silu" else None
    slope = {"none": lambda: torch.ones_like(u), "relu": lambda: (u > 0).double(),
             "silu": lambda: sig + u * sig * (1 - sig),
             "gelu": lambda: cdf + u * torch.exp(-u * u / 2) * (2 * math.pi) ** -0.5}[case["act"]]()
    g = _exact_dropped(t["dy"], p, key) * slope
    g_sum, gx_sum = g.sum(dim=(0, 1)), (g * xh).sum(dim=(0, 1))  # [N][C]
    fold = lambda v: per_c((v * t["gamma"]).view(n, case["groups"], d).sum(2) / (h * w * d))  # noqa: E731
    dx = per_c(rstd) * (g * t["gamma"] - fold(g_sum) - xh * fold(gx_sum))
    dx = {"dx": dx} if case["out"] == "f32" else _exact_mx(dx, case["out"], case["bp"])
    return dx | {"dgamma": gx_sum.sum(0), "dbeta": g_sum.sum(0)}
