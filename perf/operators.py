"""Timed cases of the operators that surround a routed-expert layer: the residual RMS norm with its 8-bit output, the
scored router, and the quantiser and product of microscaled (MX) numbers.

Where `own` is false, run() computes the operators in elementary torch operations; where it is true, it calls the
library. MX numbers: rows are cut into blocks of 32 columns, each with one power-of-two scale (E8M0, code - 127) and
elements of 4 bits (E2M1, largest 6) or 8 bits (E4M3, largest 448); rows are stored padded to 128 columns.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_MAX = {"e2m1": 6.0, "e4m3": 448.0}
_EPS = 1e-6


# ---- cases -------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode token between two layers: latency
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "t": "f16"},
        # a ragged batch of a wider model
        {"name": "norm_ragged", "op": "norm", "rows": 317, "cols": 7168, "t": "bf16"},
        # a long prefill of the narrower model
        {"name": "norm_prefill", "op": "norm", "rows": 16384, "cols": 4096, "t": "bf16"},
        # one decode token: sigmoid scores, balance bias, 4 of 8 groups
        {"name": "route_token", "op": "route", "tok": 1, "exp": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "t": "f32"},
        # a prefill batch with plain softmax scores, top-6
        {"name": "route_prefill", "op": "route", "tok": 2048, "exp": 256, "k": 6, "score": "softmax", "bias": False,
         "groups": 1, "keep": 1, "t": "f32"},
        # a large batch over the wider model's experts, grouped, 16-bit logits (many ties)
        {"name": "route_large", "op": "route", "tok": 16384, "exp": 384, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "t": "bf16"},
        # a weight matrix into 4 bits, and the numbers that it then stands for
        {"name": "quant_weight", "op": "quant", "rows": 4096, "cols": 7168, "t": "bf16", "fmt": "e2m1", "swiglu": False},
        # between the two products of a shared expert: silu(gate) * up of a prefill batch into 8 bits
        {"name": "swiglu_prefill", "op": "quant", "rows": 4096, "cols": 2048, "t": "f16", "fmt": "e4m3", "swiglu": True},
        # one decode token (8-bit, from the norm) through the gate and up rows of a shared expert
        {"name": "product_token", "op": "gemm", "m": 1, "n": 4096, "k": 4096, "fmt": "e4m3", "raw": False, "t": "f16",
         "add": False},
        # a decode batch quantised to 4 bits and taken through a down matrix, onto the routed experts' sum
        {"name": "product_batch", "op": "gemm", "m": 32, "n": 4096, "k": 2048, "fmt": "e2m1", "raw": True, "t": "f16",
         "add": True},
        # a prefill batch (8-bit, from the norm) through gate and up
        {"name": "product_prefill", "op": "gemm", "m": 2048, "n": 4096, "k": 4096, "fmt": "e4m3", "raw": False, "t": "f16",
         "add": False},
        # a long prefill quantised to 4 bits and taken through a wide matrix
        {"name": "product_large", "op": "gemm", "m": 8192, "n": 8192, "k": 7168, "fmt": "e2m1", "raw": True, "t": "bf16",
         "add": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "route", "quant", "gemm", "gemm"])
    fmt, t = rng.choice(["e2m1", "e4m3"]), rng.choice(["f16", "bf16", "f32"])
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 512, 8192), "t": t}
    if op == "route":
        groups = rng.choice([1, 4, 8])
        each = rng.randint(2, 384 // groups)
        keep = rng.randint(1, groups)
        return {"op": op, "tok": _log(rng, 1, 16384), "exp": groups * each, "k": rng.randint(1, min(8, keep * each)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups, "keep": keep,
                "t": t}
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 4096), "cols": _log(rng, 256, 4096), "t": t, "fmt": fmt,
                "swiglu": rng.random() < 0.5}
    return {"op": op, "m": _log(rng, 1, 4096), "n": _log(rng, 256, 8192), "k": _log(rng, 256, 7168), "fmt": fmt,
            "raw": rng.random() < 0.5, "t": t, "add": rng.random() < 0.5}


def work(case):
    size = {"f16": 2, "bf16": 2, "f32": 4}[case["t"]]
    code = {"e2m1": 0.5 + 1 / 32, "e4m3": 1 + 1 / 32}
    if case["op"] == "norm":   # x and residual in, sum, y and the 8-bit y out
        n = case["rows"] * case["cols"]
        return {"bytes": n * (4 * size + code["e4m3"]) + case["cols"] * size, "flops": 6 * n}
    if case["op"] == "route":
        n = case["tok"] * case["exp"]
        return {"bytes": n * size + 8 * case["tok"] * case["k"] + (4 * case["exp"] if case["bias"] else 0),
                "flops": 4 * n}
    if case["op"] == "quant":   # in 4 bits also the 16-bit numbers that the codes stand for
        n = case["rows"] * case["cols"]
        out = code[case["fmt"]] + (2 if case["fmt"] == "e2m1" else 0)
        return {"bytes": n * ((2 if case["swiglu"] else 1) * size + out), "flops": 4 * n}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": m * k * (size if case["raw"] else code[case["fmt"]]) + n * k * code["e2m1"] +
            m * n * size * (2 if case["add"] else 1), "flops": 2 * m * n * k}


# ---- inputs ------------------------------------------------------------------------------------------------------
def _spiky(gen, rows, cols, dtype, dev):
    """Activations: normal values and, in one column of a thousand, values twenty times as large."""
    x = torch.randn(rows, cols, generator=gen, device=dev)
    hot = torch.randperm(cols, generator=gen, device=dev)[: max(1, cols // 1000)]
    x[:, hot] *= 20.0
    return x.to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case)
    t = _DT[case["t"]]
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _spiky(gen, rows, cols, t, dev)
        s["res"] = _spiky(gen, rows, cols, t, dev)
        s["w"] = (1 + 0.1 * torch.randn(cols, generator=gen, device=dev)).to(t)
        s["sum"], s["y"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        s["codes"], s["scales"] = _buffers(rows, cols, "e4m3", dev)
    elif case["op"] == "route":
        tok, exp = case["tok"], case["exp"]
        s["logits"] = (2 * torch.randn(tok, exp, generator=gen, device=dev)).to(t)
        # a balance bias moves in fixed steps
        s["b"] = 0.001 * torch.randint(-100, 101, (exp,), generator=gen, device=dev).float() if case["bias"] else None
        s["idx"] = torch.empty(tok, case["k"], dtype=torch.int32, device=dev)
        s["wts"] = torch.empty(tok, case["k"], dtype=torch.float32, device=dev)
    elif case["op"] == "quant":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _spiky(gen, rows, cols * (2 if case["swiglu"] else 1), t, dev)
        s["codes"], s["scales"] = _buffers(rows, cols, case["fmt"], dev)
        s["y"] = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev) if case["fmt"] == "e2m1" else None
    else:
        m, n, k = case["m"], case["n"], case["k"]
        x = _spiky(gen, m, k, t, dev)
        if case["raw"]:
            s["x"], s["a"] = x, _buffers(m, k, case["fmt"], dev)
        else:
            s["a"] = _quantize(x.float(), case["fmt"])
        s["w"] = _quantize(torch.randn(n, k, generator=gen, device=dev) * k ** -0.5, "e2m1")
        s["c"] = torch.randn(m, n, generator=gen, device=dev).to(t) if case["add"] else None
        s["y"] = torch.empty(m, n, dtype=t, device=dev)
    return s


def _buffers(rows, cols, fmt, dev):
    g = -(-cols // 128)
    return (torch.empty(rows, g * (64 if fmt == "e2m1" else 128), dtype=torch.uint8, device=dev),
            torch.empty(rows, g * 4, dtype=torch.uint8, device=dev))


# ---- plain forms -------------------------------------------------------------------------------------------------
def _quantize(x, fmt):
    """(codes, scales) of the fp32 rows x, padded to 128 columns. The scale is the smallest power of two that the
    block's largest magnitude divided by it does not pass the format's largest number."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % 128)).reshape(rows, -1, 32)
    m, e = torch.frexp(x.abs().amax(2, keepdim=True))          # amax = m 2^e, m in [1/2, 1)
    e = torch.where(m > _MAX[fmt] / (8 if fmt == "e2m1" else 512), e + 1, e) - (3 if fmt == "e2m1" else 9)
    e = torch.where(m == 0, -127, e.clamp(-127, 127))
    scales = (e + 127).to(torch.uint8).reshape(rows, -1)
    v = torch.ldexp(x, -e)
    if fmt == "e4m3":
        return v.to(torch.float8_e4m3fn).view(torch.uint8).reshape(rows, -1), scales
    a = v.abs()
    # halves up to 2, whole numbers up to 4, even ones above; round() takes ties to even
    r = torch.where(a < 2, torch.round(2 * a), torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4))
    code = (r.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)).reshape(rows, -1, 2)
    return code[..., 0] | (code[..., 1] << 4), scales


def _values(codes, scales, fmt, cols):
    """The fp32 numbers that (codes, scales) stand for, [rows, cols]."""
    rows = codes.shape[0]
    if fmt == "e4m3":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
        v = table[torch.stack((codes & 15, codes >> 4), 2).reshape(rows, -1).int()]
    return torch.ldexp(v.reshape(rows, -1, 32), scales.int()[..., None] - 127).reshape(rows, -1)[:, :cols]


def _route(logits, b, case):
    """(idx, w): scores in 64 bits, the choice by score + bias (without a bias, by the logits themselves, which have
    the scores' order), ties to the lowest index."""
    tok, exp = logits.shape
    l = logits.double()
    s = torch.softmax(l, 1) if case["score"] == "softmax" else 1 / (1 + torch.exp(-l))
    c = s if b is None else s + b.double()
    groups, keep, k = case["groups"], case["keep"], case["k"]
    key = l if b is None else c
    if groups > 1:
        v = torch.sort(c.reshape(tok, groups, -1), 2, descending=True).values[..., :2].sum(2)
        best = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :keep]
        kept = torch.zeros_like(v, dtype=torch.bool).scatter_(1, best, True)
        key = torch.where(kept.repeat_interleave(exp // groups, 1), key, -math.inf)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, idx)
    return idx.int(), (2.5 * w / w.sum(1, keepdim=True)).float()


def _shown(codes, scales, fmt, cols, values):
    """MX numbers as run() returns them: 8-bit ones as they are held (elements and scales), 4-bit ones, which torch
    has no arithmetic for, as the 16-bit numbers that they stand for."""
    if fmt == "e4m3":
        groups = -(-cols // 32)
        return codes.view(torch.float8_e4m3fn)[:, :cols], scales.view(torch.float8_e8m0fnu)[:, :groups]
    return values()


def _plain(s):
    op, t = s["op"], _DT[s["t"]]
    if op == "norm":
        total = (s["x"].float() + s["res"].float()).to(t)
        f = total.float()
        y = f * torch.rsqrt((f * f).mean(1, keepdim=True) + _EPS) * s["w"].float()
        return total, y.to(t), _shown(*_quantize(y, "e4m3"), "e4m3", s["cols"], None)
    if op == "route":
        return _route(s["logits"], s["b"], s)
    if op == "quant":
        x = s["x"].float()
        if s["swiglu"]:
            g, u = x[:, : s["cols"]], x[:, s["cols"]:]
            x = g / (1 + torch.exp(-g)) * u
        mx = _quantize(x, s["fmt"])
        return _shown(*mx, s["fmt"], s["cols"], lambda: _values(*mx, s["fmt"], s["cols"]).to(torch.bfloat16))
    a = _quantize(s["x"].float(), s["fmt"]) if s["raw"] else s["a"]
    y = _values(*a, s["fmt"], s["k"]) @ _values(*s["w"], "e2m1", s["k"]).T
    return (y if s["c"] is None else y + s["c"].float()).to(t)


def _own(s):
    import quantized_expert_gemv_amd as q
    op = s["op"]
    if op == "norm":
        mx = q.MXTensor(s["codes"], s["scales"], s["cols"], q.GALE_MX_E4M3)
        q.add_rms_norm(s["x"], s["w"], residual=s["res"], eps=_EPS, out=s["y"], sum_out=s["sum"], mx_out=mx)
        return s["sum"], s["y"], _shown(mx.codes, mx.scales, "e4m3", s["cols"], None)
    if op == "route":
        return q.route_scored(s["logits"], s["k"], score=s["score"], bias=s["b"], n_groups=s["groups"],
                              keep_groups=s["keep"], group_score="top2", renormalize=True, scale=2.5,
                              out=(s["idx"], s["wts"]))
    fmt = q.GALE_MX_E2M1 if s["fmt"] == "e2m1" else q.GALE_MX_E4M3
    if op == "quant":
        mx = q.MXTensor(s["codes"], s["scales"], s["cols"], fmt)
        (q.mx_swiglu_quantize if s["swiglu"] else q.mx_quantize)(s["x"], fmt, out=mx)
        return _shown(mx.codes, mx.scales, s["fmt"], s["cols"], lambda: q.mx_dequantize(mx, torch.bfloat16, out=s["y"]))
    a = q.MXTensor(s["a"][0], s["a"][1], s["k"], fmt)
    w = q.MXTensor(s["w"][0], s["w"][1], s["k"], q.GALE_MX_E2M1)
    if s["raw"]:
        q.mx_quantize(s["x"], fmt, out=a)
    return q.mx_gemm(a, w, add=s["c"], out=s["y"])


def run(s):
    return _own(s) if own else _plain(s)


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------
def _exact_mx(x, fmt):
    """(elements, scales) of the fp64 rows x by the definition: the nearest of the format's numbers to x / scale."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % 32)).reshape(rows, -1, 32)
    top = x.abs().amax(2, keepdim=True) / _MAX[fmt]
    e = torch.ceil(torch.log2(top)).clamp(-127, 127)
    e = torch.where(torch.exp2(e - 1) >= top, e - 1, e)     # log2 may have rounded across a power of two
    e = torch.where(torch.exp2(e) < top, e + 1, e)
    e = torch.where(top == 0, -127.0, e).clamp(-127, 127)
    v = x / torch.exp2(e)
    low, bits = (0, 1) if fmt == "e2m1" else (-6, 3)        # smallest normal exponent, mantissa bits
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** low))).clamp_min(low) - bits)
    return torch.round(v / step) * step, torch.exp2(e)


def _exact_values(codes, scales, fmt, cols):
    rows = codes.shape[0]
    if fmt == "e4m3":
        c = codes.double()
        sign, e, f = 1 - 2 * torch.floor(c / 128), torch.floor(c / 8) % 16, c % 8
        v = sign * torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.exp2(e - 7))
    else:
        c = torch.stack((codes % 16, codes // 16), 2).reshape(rows, -1).double()
        sign, e, f = 1 - 2 * torch.floor(c / 8), torch.floor(c / 2) % 4, c % 2
        v = sign * torch.where(e == 0, f / 2, (1 + f / 2) * torch.exp2(e - 1))
    return (v.reshape(rows, -1, 32) * torch.exp2(scales.double() - 127)[..., None]).reshape(rows, -1)[:, :cols]


def _exact_shown(x, fmt):
    rows, cols = x.shape
    v, scale = _exact_mx(x, fmt)
    if fmt == "e4m3":
        return v.reshape(rows, -1)[:, :cols], scale[..., 0]
    return (v * scale).reshape(rows, -1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        total = (s["x"].double() + s["res"].double()).to(_DT[case["t"]])    # rounded once: the later layers read this
        f = total.double()
        y = f / torch.sqrt(f.square().mean(1, keepdim=True) + _EPS) * s["w"].double()
        return total.double(), y, _exact_shown(y, "e4m3")
    if op == "route":
        l = s["logits"].double()
        p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.exp(l - l.logsumexp(1, keepdim=True))
        idx, _ = _route(s["logits"], s["b"], s)              # the choice itself is compared as whole numbers
        w = p.gather(1, idx.long())
        return None, w / w.sum(1, keepdim=True) * 2.5
    if op == "quant":
        x = s["x"].double()
        if case["swiglu"]:
            g, u = x.chunk(2, 1)
            x = g * torch.sigmoid(g) * u
        return _exact_shown(x, case["fmt"])
    if case["raw"]:
        v, scale = _exact_mx(s["x"].double(), case["fmt"])
        a = (v * scale).reshape(case["m"], -1)[:, : case["k"]]
    else:
        a = _exact_values(*s["a"], case["fmt"], case["k"])
    y = a @ _exact_values(*s["w"], "e2m1", case["k"]).T
    return y if s["c"] is None else y + s["c"].double()
