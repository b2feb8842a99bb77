"""The feed-forward half of a served layer around the FP8 products, as cases to measure.

Five families, each in its plain form (elementary torch operations in float32, the
router in float64) and through the library's own entry points:

  norm     residual addition, RMS norm and quantization to 8 bits in one call
  gemm     FP8 product with bias, activation (plain or gated) and residual in its epilogue
  route    experts of every token: scores, groups, top-k, and the slots sorted by expert
  experts  the experts' FP8 products over the routed rows
  combine  the weighted sum of every token's routed rows

A case is a dict of plain values; its contents are a function of the seed.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MAX = {"e4m3": 448.0, "e5m2": 57344.0}
CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # the norm of one decoded token: latency
        {"name": "norm_token", "op": "norm", "tokens": 1, "width": 4096, "dtype": "bf16", "residual": True, "mx": False,
         "fmt": "e4m3"},
        # a long prompt's norm in front of the FFN-up product
        {"name": "norm_prefill", "op": "norm", "tokens": 16384, "width": 8192, "dtype": "bf16", "residual": True,
         "mx": False, "fmt": "e4m3"},
        # one token through the gated FFN-up product: the weights' 180 MB once
        {"name": "gemm_token_gated", "op": "gemm", "m": 1, "n": 11008, "k": 8192, "mx": False, "bias": False,
         "act": "silu", "gated": True, "residual": False},
        # the FFN-up product of a prompt, gate and up projection side by side
        {"name": "gemm_prefill_gated", "op": "gemm", "m": 8192, "n": 11008, "k": 8192, "mx": False, "bias": False,
         "act": "silu", "gated": True, "residual": False},
        # block-scaled FFN-down product of a ragged batch onto the residual stream
        {"name": "gemm_down_mx", "op": "gemm", "m": 1777, "n": 4096, "k": 14336, "mx": True, "bias": True,
         "act": "none", "gated": False, "residual": True},
        # one decoded token chooses its experts: latency
        {"name": "route_token", "op": "route", "tokens": 1, "experts": 64, "top_k": 6, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "padded": 0, "dtype": "bf16"},
        # a long prompt, sigmoid scores with a bias for balance, groups of experts, some padded tokens
        {"name": "route_prefill", "op": "route", "tokens": 16384, "experts": 256, "top_k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "padded": 37, "dtype": "f32"},
        # a decode step of 64 requests: few rows for every expert, the weights bound it
        {"name": "experts_decode", "op": "experts", "tokens": 64, "experts": 64, "top_k": 6, "k": 4096, "n": 1408,
         "mx": False, "gated": True, "bias": False, "gather": True, "skew": 0.5},
        # a prompt through many experts of uneven popularity
        {"name": "experts_prefill", "op": "experts", "tokens": 8192, "experts": 128, "top_k": 8, "k": 4096, "n": 1024,
         "mx": False, "gated": True, "bias": False, "gather": True, "skew": 0.5},
        # the second product of the experts, block-scaled, a ragged batch, some experts without a row
        {"name": "experts_down_mx", "op": "experts", "tokens": 1021, "experts": 60, "top_k": 4, "k": 1408, "n": 2048,
         "mx": True, "gated": False, "bias": False, "gather": False, "skew": 2.5},
        # a decode step's routed rows summed
        {"name": "combine_decode", "op": "combine", "tokens": 64, "top_k": 6, "width": 4096, "dtype": "bf16",
         "residual": True},
        # a prompt's
        {"name": "combine_prefill", "op": "combine", "tokens": 8192, "top_k": 8, "width": 4096, "dtype": "bf16",
         "residual": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "gemm", "gemm", "gemm", "route", "experts", "experts", "combine"])
    if op == "norm":
        mx = rng.random() < 0.4
        return {"op": op, "tokens": _log(rng, 1, 8000), "width": 32 * _log(rng, 16, 256),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "residual": rng.random() < 0.7, "mx": mx,
                "fmt": "e4m3" if mx or rng.random() < 0.8 else "e5m2"}
    if op == "gemm":
        gated = rng.random() < 0.5
        return {"op": op, "m": _log(rng, 1, 5000), "n": rng.choice([8, 16, 16, 16]) * _log(rng, 40, 640) + rng.choice([0, 0, 0, 3]),
                "k": 32 * _log(rng, 8, 350), "mx": rng.random() < 0.4, "bias": rng.random() < 0.4,
                "act": rng.choice(["silu", "silu", "gelu_tanh"]) if gated or rng.random() < 0.4 else "none",
                "gated": gated, "residual": not gated and rng.random() < 0.6}
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * rng.choice([8, 16, 32]) if groups > 1 else _log(rng, 8, 400)
        tokens = _log(rng, 1, 12000)
        return {"op": op, "tokens": tokens, "experts": experts, "top_k": rng.choice([1, 2, 4, 6, 8]),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "top_groups": max(1, groups // 2), "padded": rng.choice([0, 0, tokens // 9]),
                "dtype": rng.choice(["bf16", "f32"])}
    if op == "experts":
        experts = _log(rng, 4, 96)
        return {"op": op, "tokens": _log(rng, 1, 5000), "experts": experts, "top_k": min(experts, rng.choice([1, 2, 4, 8])),
                "k": 32 * _log(rng, 16, 128), "n": 16 * _log(rng, 20, 128), "mx": rng.random() < 0.4,
                "gated": rng.random() < 0.5, "bias": rng.random() < 0.3, "gather": rng.random() < 0.6,
                "skew": rng.choice([0.0, 0.5, 1.5])}
    return {"op": op, "tokens": _log(rng, 1, 8000), "top_k": rng.choice([1, 2, 4, 6, 8]), "width": 8 * _log(rng, 32, 512),
            "dtype": rng.choice(["bf16", "bf16", "f32"]), "residual": rng.random() < 0.6}


def work(case):
    c, size = case, {"bf16": 2, "f32": 4}.get(case.get("dtype"), 2)
    if c["op"] == "norm":
        n = c["tokens"] * c["width"]
        moved = n * (size * (3 if c["residual"] else 1) + 1) + c["width"] * 4
        return {"bytes": moved + (n // 32 if c["mx"] else 4 * c["tokens"]), "flops": 8 * n}
    if c["op"] == "gemm":
        rows = c["n"] * (2 if c["gated"] else 1)
        scales = (c["m"] + rows) * (c["k"] // 32 if c["mx"] else 4)
        moved = (c["m"] + rows) * c["k"] + scales + c["m"] * c["n"] * 2 * (2 if c["residual"] else 1) + 4 * rows * c["bias"]
        return {"bytes": moved, "flops": 2 * c["m"] * rows * c["k"]}
    if c["op"] == "route":
        return {"bytes": c["tokens"] * (c["experts"] * size + c["top_k"] * 16) + 4 * c["experts"] * (1 + c["bias"]),
                "flops": 10 * c["tokens"] * c["experts"]}
    if c["op"] == "experts":
        rows, slots = c["n"] * (2 if c["gated"] else 1), c["tokens"] * c["top_k"]
        a_rows = c["tokens"] if c["gather"] else slots
        # an expert that some token chooses: all of them where there are many slots
        used = c["experts"] * (1.0 - (1.0 - 1.0 / c["experts"]) ** slots)
        scale = c["k"] // 32 if c["mx"] else 4
        return {"bytes": (a_rows + used * rows) * (c["k"] + scale) + slots * (2 * c["n"] + 4) + 4 * rows * used * c["bias"],
                "flops": 2 * slots * rows * c["k"]}
    n = c["tokens"] * c["width"]
    return {"bytes": n * size * (c["top_k"] + 1 + c["residual"]) + c["tokens"] * c["top_k"] * 8,
            "flops": 2 * n * c["top_k"]}


# ------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _operand(g, rows, k, mx, size):
    """E4M3 codes [rows, k] of normal values and their scales, as a quantizer leaves them; size: of the values."""
    codes = torch.empty(rows, k, dtype=torch.float8_e4m3fn, device="cuda")
    step = max(1, (1 << 28) // k)
    for at in range(0, rows, step):
        x = torch.randn(min(step, rows - at), k, generator=g, device="cuda")
        codes[at:at + step] = (x * 100.0).clamp_(-448.0, 448.0)
    if not mx:
        return codes, size / 100.0 * (0.7 + 0.6 * torch.rand(rows, generator=g, device="cuda"))
    power = round(math.log2(size / 100.0)) + 127
    return codes, torch.randint(power - 1, power + 2, (rows, k // 32), generator=g, device="cuda").to(torch.uint8)


def _routing(g, tokens, experts, top_k, skew):
    """Expert starts [E + 1] and slot-to-token rows of tokens that choose among experts of uneven popularity."""
    logits = torch.randn(tokens, experts, generator=g, device="cuda") + skew * torch.randn(experts, generator=g, device="cuda")
    ids = logits.topk(top_k, 1).indices.flatten()
    chosen, order = ids.sort(stable=True)
    start = torch.searchsorted(chosen, torch.arange(experts + 1, device="cuda"))
    return start.to(torch.int32), (order // top_k).to(torch.int32), order


def prepare(case, seed):
    c, g = case, _generator(seed)
    if c["op"] == "norm":
        dt, shape = DTYPES[c["dtype"]], (c["tokens"], c["width"])
        channel = torch.exp(0.5 * torch.randn(c["width"], generator=g, device="cuda"))     # some channels run large
        return {"op": "norm", "x": (_normal(g, *shape) * channel).to(dt),
                "residual": (_normal(g, *shape, scale=2.0) * channel).to(dt) if c["residual"] else None,
                "weight": 1.0 + _normal(g, c["width"], scale=0.2), "eps": 1e-6, "mx": c["mx"], "fmt": c["fmt"]}
    if c["op"] == "gemm":
        rows = c["n"] * (2 if c["gated"] else 1)
        A, sa = _operand(g, c["m"], c["k"], c["mx"], 1.0)
        B, sb = _operand(g, rows, c["k"], c["mx"], c["k"] ** -0.5)
        return {"op": "gemm", "m": c["m"], "n": c["n"], "k": c["k"], "mx": c["mx"], "A": A, "B": B, "sa": sa, "sb": sb,
                "bias": _normal(g, rows, scale=0.5) if c["bias"] else None, "act": c["act"], "gated": c["gated"],
                "residual": _normal(g, c["m"], c["n"], dtype=torch.bfloat16) if c["residual"] else None}
    if c["op"] == "route":
        T, E = c["tokens"], c["experts"]
        logits = 2.0 * torch.randn(T, E, generator=g, device="cuda")
        if c["padded"]:
            logits[T - c["padded"]:] = -math.inf          # tokens that fill the batch up go nowhere
        return {"op": "route", "logits": logits.to(DTYPES[c["dtype"]]), "top_k": c["top_k"], "score": c["score"],
                "bias": _normal(g, E, scale=0.05) if c["bias"] else None, "groups": c["groups"],
                "top_groups": c["top_groups"], "scale": 2.5}
    if c["op"] == "experts":
        start, rows, _ = _routing(g, c["tokens"], c["experts"], c["top_k"], c["skew"])
        n = c["n"] * (2 if c["gated"] else 1)
        A, sa = _operand(g, c["tokens"] if c["gather"] else rows.shape[0], c["k"], c["mx"], 1.0)
        B, sb = _operand(g, c["experts"] * n, c["k"], c["mx"], c["k"] ** -0.5)
        return {"op": "experts", "A": A, "sa": sa, "B": B.unflatten(0, (c["experts"], n)),
                "sb": sb.unflatten(0, (c["experts"], n)), "start": start, "rows": rows if c["gather"] else None,
                "mx": c["mx"], "bias": _normal(g, c["experts"], n, scale=0.5) if c["bias"] else None, "gated": c["gated"],
                "act": "silu" if c["gated"] else "none", "most": int((start[1:] - start[:-1]).max())}
    T, k, dt = c["tokens"], c["top_k"], DTYPES[c["dtype"]]
    _, _, order = _routing(g, T, 64, k, 0.5)
    slots = torch.empty_like(order)
    slots[order] = torch.arange(T * k, device="cuda")
    weights = torch.rand(T, k, generator=g, device="cuda") + 0.05
    return {"op": "combine", "y": _normal(g, T * k, c["width"], dtype=dt), "slots": slots.view(T, k).to(torch.int32),
            "weights": weights / weights.sum(1, keepdim=True),
            "residual": _normal(g, T, c["width"], dtype=dt) if c["residual"] else None}


# ------------------------------------------------------------- the plain forms

def _values(codes, scale, mx):
    """float32 values of E4M3 codes [.., k] with a scale a row, or a UE8M0 code for every 32 elements."""
    x = codes.float()
    if not mx:
        return x * scale[..., None]
    power = torch.ldexp(torch.ones((), device=x.device), scale.int() - 127)
    return (x.unflatten(-1, (-1, 32)) * power[..., None]).flatten(-2)


def _activate(z, act, gated):
    """act(z), or act of the first half of z's columns times the second half."""
    z, up = z.chunk(2, -1) if gated else (z, None)
    if act == "silu":
        z = z / (1.0 + torch.exp(-z))
    elif act == "gelu_tanh":
        u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
        z = z / (1.0 + torch.exp(-2.0 * u))
    return z * up if gated else z


def _plain_norm(s):
    x = s["x"]
    if s["residual"] is not None:
        x = (x.float() + s["residual"].float()).to(x.dtype)
    f = x.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    if s["mx"]:
        blocks = y.unflatten(-1, (-1, 32))
        amax = blocks.abs().amax(-1, keepdim=True)
        mantissa, exponent = torch.frexp(amax)                  # 448 = 0.875 * 2^9
        e = torch.where(amax > 0, exponent - 9 + (mantissa > 0.875).int(), -127).clamp(-127, 127)
        q = torch.ldexp(blocks, -e).flatten(-2).to(torch.float8_e4m3fn)
        scale = (e.squeeze(-1) + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        most = MAX[s["fmt"]]
        scale = y.abs().amax(-1) / most
        q = torch.where(scale[:, None] > 0, y / scale[:, None], 0.0).clamp(-most, most).to(CODES[s["fmt"]])
    return (q, scale) if s["residual"] is None else (q, scale, x)


def _plain_route(s):
    logits = s["logits"].double()
    T, E = logits.shape
    k = s["top_k"]
    there = logits > -math.inf
    if s["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-logits))
    else:
        top = logits.amax(1, keepdim=True)
        p = torch.exp(logits - torch.where(top > -math.inf, top, 0.0))
        p = p / p.sum(1, keepdim=True).clamp_min(1e-300)
    choice = logits if s["bias"] is None else p + s["bias"].double()
    if s["groups"] > 1:
        value = p if s["bias"] is None else choice
        value = torch.where(there, value, -math.inf).unflatten(1, (s["groups"], -1))
        best = value.sort(2, descending=True).values[:, :, :2].sum(2)
        rank = best.sort(stable=True, dim=1, descending=True).indices[:, :s["top_groups"]]
        kept = (rank[:, :, None] == torch.arange(s["groups"], device=p.device)).any(1)
        there = there & kept.repeat_interleave(E // s["groups"], 1)
    order = torch.where(there, choice, -math.inf).sort(stable=True, dim=1, descending=True).indices[:, :k]
    fine = there.gather(1, order)
    ids = torch.where(fine, order, -1)
    weight = torch.where(fine, p.gather(1, order), 0.0)
    total = weight.sum(1, keepdim=True)
    weight = torch.where(total > 0, weight / torch.where(total > 0, total, 1.0), 0.0) * s["scale"]
    by = torch.where(fine, order, E).flatten()
    chosen, slot = by.sort(stable=True)
    start = torch.searchsorted(chosen, torch.arange(E + 1, device=p.device))
    rows = torch.where(chosen < E, slot // k, -1)
    back = torch.empty_like(slot)
    back[slot] = torch.arange(T * k, device=p.device)
    slots = torch.where(fine, back.view(T, k), -1)
    i32 = torch.int32
    return ids.to(i32), weight.float(), start.to(i32), rows.to(i32), slots.to(i32)


def _plain(s):
    if s["op"] == "norm":
        return _plain_norm(s)
    if s["op"] == "gemm":
        if s["mx"]:
            z = torch.matmul(_values(s["A"], s["sa"], True), _values(s["B"], s["sb"], True).T)
        else:
            z = torch.matmul(s["A"].float(), s["B"].float().T) * s["sa"][:, None] * s["sb"]
        if s["bias"] is not None:
            z = z + s["bias"]
        v = _activate(z, s["act"], s["gated"])
        return (v if s["residual"] is None else v + s["residual"].float()).to(torch.bfloat16)
    if s["op"] == "route":
        return _plain_route(s)
    if s["op"] == "experts":
        start, E = s["start"].long(), s["B"].shape[0]
        rows = s["rows"]
        S = s["A"].shape[0] if rows is None else rows.shape[0]
        at = torch.arange(S, device="cuda")
        e = torch.searchsorted(start[1:].contiguous(), at, right=True)
        place = at - start[e]
        x = _values(s["A"], s["sa"], s["mx"])
        padded = torch.zeros(E, s["most"], x.shape[1], device="cuda")
        padded[e, place] = x if rows is None else x[rows.long()]
        z = torch.matmul(padded, _values(s["B"], s["sb"], s["mx"]).transpose(1, 2))[e, place]
        if s["bias"] is not None:
            z = z + s["bias"][e]
        return _activate(z, s["act"], s["gated"]).to(torch.bfloat16)
    out = (s["y"].float()[s["slots"].long()] * s["weights"][..., None]).sum(1)
    return (out if s["residual"] is None else out + s["residual"].float()).to(s["y"].dtype)


# --------------------------------------------------------- the library's calls

def run(state):
    s = state
    if not own:
        return _plain(s)
    import fp8_scaled_gemm_amd as fp8g
    if s["op"] == "norm":
        fmt = fp8g.FMT_E4M3 if s["fmt"] == "e4m3" else fp8g.FMT_E5M2
        r = fp8g.add_rms_norm_quantize(s["x"], s["weight"], residual=s["residual"], eps=s["eps"], mx=s["mx"], fmt=fmt)
        scale = r.scale.view(torch.float8_e8m0fnu) if s["mx"] else r.scale        # the powers that the codes stand for
        return (r.q, scale) if s["residual"] is None else (r.q, scale, r.sum)
    if s["op"] == "gemm":
        call = fp8g.mxfp8_gemm_fused if s["mx"] else fp8g.fp8_gemm_fused
        return call(s["m"], s["n"], s["k"], s["A"], s["B"], s["sa"], s["sb"], bias=s["bias"], act=s["act"],
                    gated=s["gated"], residual=s["residual"])
    if s["op"] == "route":
        r = fp8g.moe_route(s["logits"], s["top_k"], bias=s["bias"], score=s["score"], groups=s["groups"],
                           top_groups=s["top_groups"], scale=s["scale"])
        return r.ids, r.weights, r.expert_start, r.rows, r.slots
    if s["op"] == "experts":
        call = fp8g.mxfp8_moe_gemm if s["mx"] else fp8g.fp8_moe_gemm
        return call(s["A"], s["B"], s["sa"], s["sb"], s["start"], rows=s["rows"], bias=s["bias"], act=s["act"],
                    gated=s["gated"])
    return fp8g.moe_combine(s["y"], s["slots"], s["weights"], residual=s["residual"])


# ---------------------------------------------------- the definitions in 64 bits

def _nearest(x, mantissa, low, most):
    """float64 x to the nearest value with `mantissa` fraction bits, exponents from `low`, ties to even, up to `most`."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -300)))
    e = torch.where(2.0 ** e > x.abs(), e - 1, torch.where(2.0 ** (e + 1) <= x.abs(), e + 1, e)).clamp_min(low)
    step = 2.0 ** (e - mantissa)
    return (torch.round(x / step) * step).clamp(-most, most)        # torch.round takes ties to even


def _exact_norm(s, case):
    x = s["x"].double()
    if s["residual"] is not None:
        # the sum is the residual stream of the layers behind: its rounding is part of the definition
        x = (x + s["residual"].double()).to(s["x"].dtype).double()
    y = x / ((x * x).sum(1, keepdim=True) / case["width"] + s["eps"]).sqrt() * s["weight"].double()
    if case["mx"]:
        blocks = y.reshape(case["tokens"], -1, 32)
        amax = blocks.abs().amax(2, keepdim=True)
        e = torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448.0)).clamp(-127, 127)
        e = torch.where((e > -127) & (amax <= 448.0 * 2.0 ** (e - 1)), e - 1, e)        # log2's own rounding
        e = torch.where(amax > 448.0 * 2.0 ** e, e + 1, e)
        return (_nearest(blocks / 2.0 ** e, 3, -6, 448.0).reshape(x.shape), (2.0 ** e).squeeze(2),
                None if s["residual"] is None else x)
    scale = y.abs().amax(1) / MAX[case["fmt"]]
    bits = {"e4m3": (3, -6), "e5m2": (2, -14)}[case["fmt"]]
    q = _nearest(y / scale[:, None].clamp_min(1e-300), *bits, MAX[case["fmt"]])
    return q, scale, None if s["residual"] is None else x


def _exact_rows(codes, scale, mx):
    if mx:
        scale = (2.0 ** (scale.double() - 127.0)).repeat_interleave(32, -1)
    return codes.float().double() * (scale if mx else scale.double()[..., None])


def _exact_act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def _exact_product(a, B, sb, bias, case):
    """float64 rows a against the codes B [n', k], a block of output columns at a time."""
    n, out = case["n"], []
    for at in range(0, n, 4096):
        part = []
        for base in ((0, n) if case["gated"] else (0,)):
            cut = slice(base + at, base + min(at + 4096, n))
            z = a @ _exact_rows(B[cut], sb[cut], case["mx"]).T
            part.append(z if bias is None else z + bias[cut].double())
        z = _exact_act(part[0], case["act"])
        out.append(z * part[1] if case["gated"] else z)
    return torch.cat(out, 1)


def _exact_route(s, case):
    """Every token's experts from numpy's float64, token by token where groups matter."""
    import numpy as np
    logits = s["logits"].double().cpu().numpy()
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if case["score"] == "sigmoid":
            p = 1.0 / (1.0 + np.exp(-logits))
        else:
            m = logits.max(1, keepdims=True)
            p = np.exp(logits - np.where(np.isfinite(m), m, 0.0))
            p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    value = p if s["bias"] is None else p + s["bias"].double().cpu().numpy()
    key = logits if s["bias"] is None else value
    there = np.isfinite(logits)
    if case["groups"] > 1:
        G, width = case["groups"], E // case["groups"]
        best = np.sort(np.where(there, value, -np.inf).reshape(T, G, width), 2)[:, :, -2:].sum(2)
        place = np.argsort(np.argsort(-best, 1, kind="stable"), 1, kind="stable")
        there = there & np.repeat(place < case["top_groups"], width, 1)
    ids = np.argsort(-np.where(there, key, -np.inf), 1, kind="stable")[:, :k]
    fine = np.take_along_axis(there, ids, 1)
    w = np.where(fine, np.take_along_axis(p, ids, 1), 0.0)
    total = w.sum(1, keepdims=True)
    w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0) * s["scale"]
    flat = np.where(fine, ids, E).reshape(-1)
    order = np.argsort(flat, kind="stable")
    start = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E + 1)[:E])])
    rows = np.where(flat[order] < E, order // k, -1)
    slots = np.empty(T * k, np.int64)
    slots[order] = np.arange(T * k)
    slots = np.where(fine, slots.reshape(T, k), -1)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32))    # noqa: E731
    return i32(np.where(fine, ids, -1)), torch.from_numpy(w), i32(start), i32(rows), i32(slots)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        out = _exact_norm(s, case)
        return out[:2] if s["residual"] is None else out
    if s["op"] == "gemm":
        a = _exact_rows(s["A"], s["sa"], case["mx"])
        v = _exact_product(a, s["B"], s["sb"], s["bias"], case)
        return v if s["residual"] is None else v + s["residual"].double()
    if s["op"] == "route":
        return _exact_route(s, case)
    if s["op"] == "experts":
        cuts, out = s["start"].tolist(), []
        part = dict(case, act="silu" if case["gated"] else "none")
        for e, (a, b) in enumerate(zip(cuts, cuts[1:])):
            if b > a:
                at = torch.arange(a, b, device="cuda") if s["rows"] is None else s["rows"][a:b].long()
                out.append(_exact_product(_exact_rows(s["A"][at], s["sa"][at], case["mx"]), s["B"][e], s["sb"][e],
                                          None if s["bias"] is None else s["bias"][e], part))
        return torch.cat(out)
    out = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda")
    for j in range(case["top_k"]):
        out += s["weights"][:, j, None].double() * s["y"][s["slots"][:, j].long()].double()
    return out if s["residual"] is None else out + s["residual"].double()
