"""The attention block's operators around the FP8 projections, as cases to measure.

Four families, each in its plain form (elementary torch operations in float32)
and through the library's own entry points:

  qk       per-head RMS norm of queries and keys with the position rotation
  cache    rows appended to a paged MXFP4 key/value cache and read back
  attention  attention over that cache, decode and chunked prefill
  lora     low-rank adapters of many requests added to a shared projection

A case is a dict of plain values; its lengths are a function of the case, its
contents of the seed.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one token of one request: the latency of a decode step's smallest launch
        {"name": "qk_token", "op": "qk", "tokens": 1, "q_heads": 32, "k_heads": 8, "dim": 128, "rotary": 128,
         "axes": 1, "interleaved": False, "dtype": "bf16"},
        # float32 projections, rotation of part of the head in neighbouring pairs, an odd number of rows
        {"name": "qk_partial_f32", "op": "qk", "tokens": 1021, "q_heads": 16, "k_heads": 16, "dim": 64, "rotary": 32,
         "axes": 1, "interleaved": True, "dtype": "f32"},
        # prefill of image and text tokens: positions in time, height and width
        {"name": "qk_prefill_axes", "op": "qk", "tokens": 8192, "q_heads": 64, "k_heads": 8, "dim": 128, "rotary": 128,
         "axes": 3, "interleaved": False, "dtype": "bf16"},
        # a decode step of 128 requests: every row to a page of its own
        {"name": "cache_decode", "op": "cache", "tokens": 128, "heads": 8, "dk": 128, "dv": 128, "page": 16,
         "requests": 128, "dtype": "bf16"},
        # prefill of MLA key rows (128 + 64 elements) with their values
        {"name": "cache_prefill_mla", "op": "cache", "tokens": 16384, "heads": 16, "dk": 192, "dv": 128, "page": 64,
         "requests": 3, "dtype": "bf16"},
        # one request, one token: the latency of a decode step
        {"name": "attn_token", "op": "attention", "batch": 1, "q_len": 1, "kv_len": 2048, "q_heads": 32, "kv_heads": 8,
         "dk": 128, "dv": 128, "page": 16, "causal": True, "window": 0, "ragged": False},
        # a decode step of 64 requests with long contexts of different lengths
        {"name": "attn_decode", "op": "attention", "batch": 64, "q_len": 1, "kv_len": 16384, "q_heads": 64,
         "kv_heads": 8, "dk": 128, "dv": 128, "page": 16, "causal": True, "window": 0, "ragged": True},
        # five speculated tokens of each request, MLA heads, a sliding window
        {"name": "attn_verify_mla", "op": "attention", "batch": 13, "q_len": 5, "kv_len": 4099, "q_heads": 16,
         "kv_heads": 16, "dk": 192, "dv": 128, "page": 32, "causal": True, "window": 2048, "ragged": True},
        # chunks of three prompts, each behind a context that the cache already holds
        {"name": "attn_prefill", "op": "attention", "batch": 3, "q_len": 4096, "kv_len": 8192, "q_heads": 32,
         "kv_heads": 8, "dk": 128, "dv": 128, "page": 16, "causal": True, "window": 0, "ragged": True},
        # a decode step of 64 requests, each with its own adapter
        {"name": "lora_decode", "op": "lora", "tokens": 64, "segments": 64, "adapters": 64, "k": 4096, "n": 4096,
         "rank": 16, "dtype": "bf16"},
        # prefill of seven requests over four adapters
        {"name": "lora_prefill", "op": "lora", "tokens": 8192, "segments": 7, "adapters": 4, "k": 8192, "n": 2048,
         "rank": 64, "dtype": "bf16"},
        # a mixed step on a float32 projection of odd width
        {"name": "lora_mixed_f32", "op": "lora", "tokens": 777, "segments": 37, "adapters": 12, "k": 4096, "n": 1001,
         "rank": 8, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["qk", "cache", "attention", "attention", "lora", "lora"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "qk":
        dim = rng.choice([64, 128, 192, 256])
        k_heads = rng.choice([1, 2, 5, 8])
        return {"op": op, "tokens": _log(rng, 1, 4096), "q_heads": k_heads * rng.choice([1, 3, 4, 8]),
                "k_heads": k_heads, "dim": dim, "rotary": rng.choice([32, 64, dim]), "axes": rng.choice([1, 1, 3]),
                "interleaved": rng.random() < 0.5, "dtype": dtype}
    if op == "cache":
        dk = rng.choice([64, 128, 192])
        tokens = _log(rng, 1, 12000)
        return {"op": op, "tokens": tokens, "heads": rng.choice([1, 3, 8, 16]), "dk": dk, "dv": min(dk, 128),
                "page": rng.choice([16, 32, 64, 256]), "requests": min(tokens, _log(rng, 1, 64)), "dtype": dtype}
    if op == "attention":
        dk = rng.choice([64, 128, 128, 192])
        kv_heads = rng.choice([1, 2, 5, 8])
        group = rng.choice([1, 3, 4, 8])
        c = {"op": op, "q_heads": kv_heads * group, "kv_heads": kv_heads, "dk": dk, "dv": min(dk, 128),
             "page": rng.choice([16, 32, 64, 256]), "causal": rng.random() < 0.8, "ragged": rng.random() < 0.7}
        if rng.random() < 0.5:     # decode and verification
            c.update(batch=_log(rng, 1, 48), q_len=rng.choice([1, 1, 2, 7]), kv_len=_log(rng, 1, 16000))
        else:                      # prefill, or cross attention where it is not causal
            c.update(batch=_log(rng, 1, 3), q_len=_log(rng, 16, 3500), kv_len=_log(rng, 16, 8000))
        c["window"] = rng.choice([0, 0, 1 + c["kv_len"] // 3]) if c["causal"] else 0
        return c
    tokens = _log(rng, 1, 6000)
    adapters = _log(rng, 1, 64 if tokens < 500 else 8)
    return {"op": op, "tokens": tokens, "segments": min(tokens, _log(rng, 1, 100)), "adapters": adapters,
            "k": rng.choice([1024, 2048, 4096, 8192]), "n": rng.choice([1001, 1024, 2048, 4096]),
            "rank": rng.choice([8, 16, 32, 64, 128]), "dtype": dtype}


# ------------------------------------------------------- lengths of a case

def _spread(count, top, ragged):
    """`count` lengths up to `top`: all equal, or spread over [top / 4, top]."""
    if not ragged:
        return [top] * count
    return [max(1, int(top * (1.0 - 0.75 * ((i * 0.6180339887) % 1.0)))) for i in range(count)]


def _cuts(total, parts):
    """Starts of `parts` uneven runs that cover [0, total), total included."""
    weights = [1.0 + 3.0 * ((i * 0.6180339887) % 1.0) for i in range(parts)]
    cuts, run = [0], 0.0
    for i, w in enumerate(weights):
        run += w
        # at least one token for each run that is left
        at = int(total * run / sum(weights))
        cuts.append(min(max(at, cuts[-1] + 1), total - (parts - 1 - i)))
    cuts[-1] = total
    return cuts


def _attention_lengths(case):
    kv = _spread(case["batch"], case["kv_len"], case["ragged"])
    q = _spread(case["batch"], case["q_len"], case["ragged"] and case["q_len"] > 16)
    return q, kv


def _pairs(case):
    """Visible (query, key) pairs, and visible keys, over the batch."""
    pairs = keys = 0
    for n, length in zip(*_attention_lengths(case)):
        if not case["causal"]:
            pairs, keys = pairs + n * length, keys + length
            continue
        window = case["window"] or length + n
        first = length - n                       # position of the first query
        for p in (range(first, length) if n < 64 else ()):
            pairs += max(0, p + 1) - max(0, p + 1 - window)
        if n >= 64:
            # sums over p + 1 = first + 1 .. length of max(p + 1, 0), less the same behind the window
            tri = lambda a, b: sum((x * (x + 1) // 2) * s for x, s in ((max(b, 0), 1), (max(a - 1, 0), -1)))  # noqa: E731
            pairs += tri(first + 1, length) - tri(first + 1 - window, length - window)
        keys += length - max(0, first + 1 - window)
    return pairs, keys


def _adapters(case):
    """Adapter of each segment; every seventh has none."""
    return [-1 if i % 7 == 6 else (i * 5 + 1) % case["adapters"] for i in range(case["segments"])]


def work(case):
    size = {"bf16": 2, "f32": 4}.get(case.get("dtype"), 2)
    if case["op"] == "qk":
        n = case["tokens"] * (case["q_heads"] + case["k_heads"])
        table = case["tokens"] * (case["rotary"] * 4 + case["axes"] * 4)
        return {"bytes": 2 * n * case["dim"] * size + table, "flops": n * (4 * case["dim"] + 3 * case["rotary"])}
    if case["op"] == "cache":
        n = case["tokens"] * case["heads"] * (case["dk"] + case["dv"])
        # the rows in, their codes out, the codes in, the rows out in bf16
        return {"bytes": n * (size + 2) + 2 * n * 17 // 32 + case["tokens"] * 16, "flops": 6 * n}
    if case["op"] == "attention":
        pairs, keys = _pairs(case)
        rows = sum(_attention_lengths(case)[0]) * case["q_heads"]
        width = case["dk"] + case["dv"]
        return {"bytes": keys * case["kv_heads"] * width * 17 // 32 + rows * (2 * width + 4),
                "flops": 2 * pairs * case["q_heads"] * width}
    cuts, of = _cuts(case["tokens"], case["segments"]), _adapters(case)
    served = sum(b - a for a, b, w in zip(cuts, cuts[1:], of) if w >= 0)
    k, n, rank = case["k"], case["n"], case["rank"]
    used = len({w for w in of if w >= 0})
    return {"bytes": served * k * 2 + case["tokens"] * n * 2 * size + used * rank * (k + n) * 2,
            "flops": 2 * served * rank * (k + n) + 2 * case["tokens"] * n}


# ------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _filled(g, pages, heads, page, dim):
    """A cache's codes and scales, holding normal rows whose channels differ in size."""
    codes = torch.empty(pages, heads, page, dim // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, heads, dim // 32, page, dtype=torch.uint8, device="cuda")
    channel = torch.exp(0.5 * torch.randn(heads, 1, dim, generator=g, device="cuda"))
    step = max(1, (1 << 24) // (heads * page * dim))
    for at in range(0, pages, step):
        count = min(step, pages - at)
        code, scale = _quantize(torch.randn(count, heads, page, dim, generator=g, device="cuda") * channel)
        codes[at:at + count] = code
        scales[at:at + count] = scale.transpose(2, 3)
    return codes, scales


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "qk":
        T, dt = case["tokens"], DTYPES[case["dtype"]]
        rows = (case["q_heads"] + 2 * case["k_heads"]) * case["dim"]
        projected = _normal(g, T, rows, dtype=dt)          # q, k and v side by side, as one projection leaves them
        half = case["rotary"] // 2
        span = 4096 + T
        angle = torch.arange(span, device="cuda").double()[:, None] * \
            10000.0 ** (-torch.arange(half, device="cuda").double() / half)
        if case["axes"] == 1:
            start = int(torch.randint(0, 4096, (1,), generator=g, device="cuda"))
            positions = torch.arange(start, start + T, device="cuda").to(torch.int32)
            axis = None
        else:
            positions = torch.randint(0, span, (case["axes"], T), generator=g, device="cuda").to(torch.int32)
            axis = (torch.arange(half, device="cuda") * case["axes"] // half).to(torch.int32)
        split = [case["q_heads"] * case["dim"], case["k_heads"] * case["dim"]]
        return {"op": "qk", "q": projected[:, :split[0]].unflatten(1, (case["q_heads"], case["dim"])),
                "k": projected[:, split[0]:sum(split)].unflatten(1, (case["k_heads"], case["dim"])),
                "q_weight": 1.0 + _normal(g, case["dim"], scale=0.2), "k_weight": 1.0 + _normal(g, case["dim"], scale=0.2),
                "positions": positions, "axis": axis, "interleaved": case["interleaved"], "eps": 1e-6,
                "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()}
    if case["op"] == "cache":
        T, H, page, dt = case["tokens"], case["heads"], case["page"], DTYPES[case["dtype"]]
        cuts = _cuts(T, case["requests"])
        need = sum((b - a + page - 1) // page + 1 for a, b in zip(cuts, cuts[1:]))
        pages = need + need // 4 + 1
        order = torch.randperm(pages, generator=g, device="cuda")
        # each request's run starts somewhere in its first page and goes on over pages in no order
        lengths = _ints([b - a for a, b in zip(cuts, cuts[1:])], torch.int64)
        starts = _ints(cuts[:-1], torch.int64)
        first = torch.randint(0, page, (len(cuts) - 1,), generator=g, device="cuda")
        base = torch.cumsum((lengths + page - 1) // page + 1, 0) - ((lengths + page - 1) // page + 1)
        owner = torch.repeat_interleave(torch.arange(len(cuts) - 1, device="cuda"), lengths)
        at = torch.arange(T, device="cuda") - starts[owner] + first[owner]
        slots = order[base[owner] + at // page] * page + at % page
        return {"op": "cache", "cache": (*_filled(g, pages, H, page, case["dk"]), *_filled(g, pages, H, page, case["dv"])),
                "k": _normal(g, T, H, case["dk"], dtype=dt), "v": _normal(g, T, H, case["dv"], dtype=dt), "slots": slots}
    if case["op"] == "attention":
        q, kv = _attention_lengths(case)
        page = case["page"]
        width = (max(kv) + page - 1) // page
        counts = [(n + page - 1) // page for n in kv]
        pages = sum(counts) + 8
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(len(kv), width, dtype=torch.int32)
        order_host, at = order.cpu(), 0
        for i, n in enumerate(counts):
            table[i, :n] = order_host[at:at + n]
            at += n
        starts = [0]
        for n in q:
            starts.append(starts[-1] + n)
        H = case["kv_heads"]
        return {"op": "attention", "q": _normal(g, starts[-1], case["q_heads"], case["dk"], dtype=torch.bfloat16),
                "cache": (*_filled(g, pages, H, page, case["dk"]), *_filled(g, pages, H, page, case["dv"])),
                "table": table.cuda(), "q_start": _ints(starts), "kv_len": _ints(kv), "q_most": max(q),
                "scale": case["dk"] ** -0.5, "causal": case["causal"], "window": case["window"]}
    T, dt = case["tokens"], DTYPES[case["dtype"]]
    k, n, r, N = case["k"], case["n"], case["rank"], case["adapters"]
    return {"op": "lora", "base": _normal(g, T, n, dtype=dt), "x": _normal(g, T, k, dtype=torch.bfloat16),
            "A": _normal(g, N, r, k, dtype=torch.bfloat16, scale=k ** -0.5),
            "B": _normal(g, N, n, r, dtype=torch.bfloat16, scale=r ** -0.5),
            "scale": 0.5 + torch.rand(N, generator=g, device="cuda"),
            "seg_start": _ints(_cuts(T, case["segments"])), "seg_adapter": _ints(_adapters(case))}


# ------------------------------------------------------------- the plain forms

def _quantize(x):
    """E2M1 codes (two a byte) and UE8M0 scale codes of float32 x, 32 elements of the last axis a scale."""
    blocks = x.unflatten(-1, (-1, 32))
    amax = blocks.abs().amax(-1, keepdim=True)
    mantissa, exponent = torch.frexp(amax)
    e = torch.where(amax > 0, exponent - 3 + (mantissa > 0.75).int(), -127).clamp(-127, 127)
    y = torch.ldexp(blocks.abs(), -e)
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = (code | (torch.signbit(blocks).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


def _values(codes, scales):
    """Float32 values of codes [..., d / 2] with scale codes [..., d / 32]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    x = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    power = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    return (x.unflatten(-1, (-1, 32)) * power[..., None]).flatten(-2)


def _rotate(x, weight, s):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight
    half = s["cos_sin"].shape[1] // 2
    p = s["positions"].long()
    if s["axis"] is None:
        c, n = s["cos_sin"][p][:, None].split(half, -1)
    else:
        p = p[s["axis"].long()].T                                        # [T, half]
        i = torch.arange(half, device=x.device)
        c, n = s["cos_sin"][p, i][:, None], s["cos_sin"][p, half + i][:, None]
    if s["interleaved"]:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([turned, y[..., 2 * half:]], -1)


def _append(x, slots, codes, scales):
    """Write rows x to the cache's slots, and read them back."""
    at, row = slots // codes.shape[2], slots % codes.shape[2]
    codes[at, :, row], scales[at, :, :, row] = _quantize(x.float())
    return _values(codes[at, :, row], scales[at, :, :, row]).to(torch.bfloat16)


def _plain(s):
    if s["op"] == "qk":
        return (_rotate(s["q"], s["q_weight"], s).to(s["q"].dtype), _rotate(s["k"], s["k_weight"], s).to(s["k"].dtype))
    if s["op"] == "cache":
        return _append(s["k"], s["slots"], *s["cache"][:2]), _append(s["v"], s["slots"], *s["cache"][2:])
    if s["op"] == "attention":
        q, B, most = s["q"].float(), s["kv_len"].shape[0], s["q_most"]
        gather = lambda codes, scales: _values(codes[s["table"].long()],                             # noqa: E731
                                               scales[s["table"].long()].transpose(3, 4)).permute(0, 2, 1, 3, 4).flatten(2, 3)
        k, v = gather(*s["cache"][:2]), gather(*s["cache"][2:])          # [B, Hk, L, d]
        starts, lengths = s["q_start"].long(), s["kv_len"].long()
        i = torch.arange(most, device=q.device)
        inside = i[None] < (starts[1:] - starts[:-1])[:, None]           # [B, most]
        index = torch.where(inside, starts[:-1, None] + i, 0)
        Hk = k.shape[1]
        rows = q[index].permute(0, 2, 1, 3).unflatten(1, (Hk, -1)).flatten(2, 3)     # [B, Hk, G * most, dk]
        score = torch.matmul(rows, k.transpose(2, 3)).mul_(s["scale"]).unflatten(2, (-1, most))
        j = torch.arange(k.shape[2], device=q.device)
        p = (lengths - (starts[1:] - starts[:-1]))[:, None] + i          # positions of the queries
        seen = (j < lengths[:, None])[:, None] & inside[..., None]
        if s["causal"]:
            seen = seen & (j <= p[..., None])
            if s["window"]:
                seen = seen & (j > p[..., None] - s["window"])
        seen = seen[:, None, None]
        score.masked_fill_(~seen, -math.inf)
        top = score.amax(-1, keepdim=True)
        weight = torch.exp_(score.sub_(torch.where(top.isinf(), 0.0, top)))
        total = weight.sum(-1, keepdim=True)
        lse = (top + total.log()).squeeze(-1)
        out = torch.matmul(weight.flatten(2, 3), v).unflatten(2, (-1, most)) / torch.where(total > 0, total, 1.0)
        out = out.flatten(1, 2).transpose(1, 2)[inside].to(s["q"].dtype)
        return out, lse.flatten(1, 2).transpose(1, 2)[inside]
    T, N = s["base"].shape[0], s["A"].shape[0]
    segment = torch.searchsorted(s["seg_start"][1:].contiguous(), torch.arange(T, device="cuda", dtype=torch.int32), right=True)
    adapter = s["seg_adapter"][segment].long()
    chosen = (adapter[:, None] == torch.arange(N, device="cuda")).float() * s["scale"]      # [T, N]
    low = torch.matmul(s["x"].float(), s["A"].float().flatten(0, 1).T).unflatten(1, (N, -1)) * chosen[..., None]
    delta = torch.matmul(low.flatten(1), s["B"].float().transpose(1, 2).flatten(0, 1))
    return (s["base"].float() + delta).to(s["base"].dtype)


# --------------------------------------------------------- the library's calls

def run(state):
    s = state
    if not own:
        return _plain(s)
    import fp8_scaled_gemm_amd as fp8g
    if s["op"] == "qk":
        return fp8g.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["cos_sin"],
                                 axis=s["axis"], eps=s["eps"], interleaved=s["interleaved"])
    if s["op"] == "cache":
        cache = fp8g.KV4Cache(*s["cache"])
        fp8g.kv4_append(cache, s["k"], s["v"], s["slots"])
        return fp8g.kv4_gather(cache, s["slots"])
    if s["op"] == "attention":
        return fp8g.kv4_attention(s["q"], fp8g.KV4Cache(*s["cache"]), s["table"], s["q_start"], s["kv_len"],
                                  scale=s["scale"], causal=s["causal"], window=s["window"], return_lse=True)
    return fp8g.lora_add(s["base"], s["x"], s["A"], s["B"], s["scale"], s["seg_start"], s["seg_adapter"])


# ---------------------------------------------------- the definitions in 64 bits

def _exact_values(codes, scales):
    """Codes [..., d / 2], scale codes [..., d / 32] -> float64, from the bit fields of E2M1 and UE8M0."""
    nibble = torch.stack([codes.long() % 16, codes.long() // 16], -1).reshape(*codes.shape[:-1], -1)
    field, fraction = nibble % 8 // 2, (nibble % 2).double()
    size = torch.where(field == 0, 0.5 * fraction, (1.0 + 0.5 * fraction) * 2.0 ** (field - 1).double())
    return (1.0 - 2.0 * (nibble // 8).double()) * size * \
        (2.0 ** (scales.double() - 127.0)).repeat_interleave(32, -1)


def _exact_rounded(x):
    """The MXFP4 values that stand for x: the nearest one, ties to the even code."""
    x = x.double()
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    amax = blocks.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax.clamp_min(2.0 ** -140) / 6.0)).clamp(-127, 127)
    e = torch.where((e > -127) & (amax <= 6.0 * 2.0 ** (e - 1)), e - 1, e)       # log2's own rounding, either way
    e = torch.where(amax > 6.0 * 2.0 ** e, e + 1, e).clamp(-127, 127)
    y = blocks / 2.0 ** e
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    best = torch.zeros_like(y)
    for code in (1, 3, 5, 7, 0, 2, 4, 6):          # even codes last: they win a tie
        near = grid[code] - y.abs()
        best = torch.where(near.abs() <= (best - y.abs()).abs(), grid[code], best)
    return (torch.where(y < 0, -best, best) * 2.0 ** e).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "qk":
        out = []
        half = case["rotary"] // 2
        i = torch.arange(half, device="cuda")
        which = torch.zeros_like(i) if s["axis"] is None else s["axis"].long()
        place = s["positions"].long().reshape(-1, case["tokens"])[which]           # [half, T]
        c = s["cos_sin"].double()[place, i[:, None]].T[:, None]
        n = s["cos_sin"].double()[place, half + i[:, None]].T[:, None]
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            x = x.double()
            y = x / (x.pow(2).sum(-1, keepdim=True) / case["dim"] + s["eps"]).sqrt() * w.double()
            z = y.clone()
            z[..., first] = y[..., first] * c - y[..., second] * n
            z[..., second] = y[..., second] * c + y[..., first] * n
            out.append(z)
        return tuple(out)
    if s["op"] == "cache":
        return _exact_rounded(s["k"]), _exact_rounded(s["v"])
    if s["op"] == "attention":
        H, G = case["kv_heads"], case["q_heads"] // case["kv_heads"]
        out, lse = [], []
        at = 0
        for b, (n, length) in enumerate(zip(*_attention_lengths(case))):
            ids = s["table"][b, :(length + case["page"] - 1) // case["page"]].long()
            q = s["q"][at:at + n].double()
            at += n
            j = torch.arange(length, device="cuda")
            p = length - n + torch.arange(n, device="cuda")[:, None]
            seen = torch.ones(n, length, dtype=torch.bool, device="cuda")
            if case["causal"]:
                seen = j <= p
                if case["window"]:
                    seen = seen & (j > p - case["window"])
            heads, logs = [], []
            for h in range(H):
                rows = [_exact_values(codes[ids, h], scales[ids, h].transpose(1, 2)).reshape(-1, codes.shape[-1] * 2)[:length]
                        for codes, scales in (s["cache"][:2], s["cache"][2:])]
                for r in range(G):
                    score = (q[:, h * G + r] @ rows[0].T * s["scale"]).masked_fill(~seen, -math.inf)
                    log = torch.logsumexp(score, 1)
                    share = torch.where(seen, torch.exp(score - log[:, None]), 0.0)
                    heads.append(share @ rows[1])
                    logs.append(log)
            out.append(torch.stack(heads, 1))
            lse.append(torch.stack(logs, 1))
        return torch.cat(out), torch.cat(lse)
    out = s["base"].double()
    cuts = _cuts(case["tokens"], case["segments"])
    for a, b, w in zip(cuts, cuts[1:], _adapters(case)):
        if w >= 0:
            out[a:b] += s["scale"][w].double() * ((s["x"][a:b].double() @ s["A"][w].double().T) @ s["B"][w].double().T)
    return out
