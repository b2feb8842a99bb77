"""CPU definitions of the attention block's operators (include/fp8g_block.h),
in float64: low-rank adapters, head norm with rotation, MXFP4 rows, attention.

Plain loops and numpy, written from the formulas; the library never uses it.
Each returns the exact value and, where a bound needs it, the sum of magnitudes
that rounding errors scale with.
"""

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mxfp4_quantize(x):
    """Codes (one an element, 0..15) and UE8M0 scale codes of x [..., D], by the
    definition: the smallest e with amax <= 6 * 2^e, the nearest E2M1 value of x
    * 2^-e, ties to the even code."""
    x = np.asarray(x, np.float64)
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(blocks).max(-1)
    e = np.full(amax.shape, -127, np.int64)
    for c in range(-127, 127):                 # raise e while 6 * 2^e is too small
        e = np.where(amax > 6.0 * 2.0 ** c, c + 1, e)
    y = np.abs(blocks) / (2.0 ** e.astype(np.float64))[..., None]
    dist = np.abs(y[..., None] - E2M1)
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])   # even codes first: argmin takes the first of equals
    code = order[np.argmin(dist[..., order], -1)]
    code = code + 8 * np.signbit(blocks)
    return code.reshape(x.shape).astype(np.uint8), (e + 127).astype(np.uint8)


def mxfp4_values(codes, scales):
    """Float64 values of codes [..., D] (one an element) with scale codes [..., D / 32]."""
    mag = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return mag * np.repeat(2.0 ** (scales.astype(np.float64) - 127.0), 32, -1)


def pack(codes):
    """One code an element -> two a byte, element 2i in the low nibble."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(b):
    out = np.empty(b.shape[:-1] + (2 * b.shape[-1],), np.uint8)
    out[..., 0::2], out[..., 1::2] = b & 15, b >> 4
    return out


def lora_add(base, x, A, B, scale, seg_start, seg_adapter):
    """(out, sum |scale| |B| |A x|, sum |scale| |B| |A| |x|)."""
    out = np.array(base, np.float64)
    low, full = np.zeros_like(out), np.zeros_like(out)
    for s, a in enumerate(seg_adapter):
        t0, t1 = max(0, seg_start[s]), min(len(out), seg_start[s + 1])
        if 0 <= a < len(A) and t1 > t0:
            h = x[t0:t1] @ A[a].T
            out[t0:t1] += scale[a] * (h @ B[a].T)
            low[t0:t1] = abs(scale[a]) * (np.abs(h) @ np.abs(B[a]).T)
            full[t0:t1] = abs(scale[a]) * ((np.abs(x[t0:t1]) @ np.abs(A[a]).T) @ np.abs(B[a]).T)
    return out, low, full


def qk_norm_rope(x, weight, positions, axis, cos_sin, eps, interleaved):
    """(out, sum of the magnitudes of each output's terms) for x [T, H, D];
    positions [axes, T], axis [rotary / 2]."""
    x = np.asarray(x, np.float64)
    T, H, D = x.shape
    half = cos_sin.shape[1] // 2
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if weight is None else weight)
    out, mag = y.copy(), np.abs(y)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        p = positions[axis[i]]
        c, s = cos_sin[p, i][:, None], cos_sin[p, half + i][:, None]
        out[:, :, a] = y[:, :, a] * c - y[:, :, b] * s
        out[:, :, b] = y[:, :, b] * c + y[:, :, a] * s
        mag[:, :, a] = np.abs(y[:, :, a] * c) + np.abs(y[:, :, b] * s)
        mag[:, :, b] = np.abs(y[:, :, b] * c) + np.abs(y[:, :, a] * s)
    return out, mag


def attention(q, k, v, q_start, kv_len, scale, causal, window):
    """q [Tq, Hq, dk]; k[b], v[b] [kv_len, Hkv, d] values of sequence b.  Returns
    (out, lse, sum p |v|, bound on |error of a score| per unit roundoff), NaN in
    rows of no sequence."""
    Tq, Hq, dk = q.shape
    dv = v[0].shape[2] if v else dk
    out = np.full((Tq, Hq, dv), np.nan)
    weight = np.zeros((Tq, Hq, dv))
    lse = np.full((Tq, Hq), np.nan)
    spread = np.zeros((Tq, Hq))
    for b in range(len(kv_len)):
        q0, n, L = q_start[b], q_start[b + 1] - q_start[b], kv_len[b]
        group = Hq // k[b].shape[1]
        for i in range(n):
            p = L - n + i
            j = np.arange(L)
            seen = np.ones(L, bool)
            if causal:
                seen = (j <= p) & ((j > p - window) if window else True)
            out[q0 + i], lse[q0 + i] = 0.0, -np.inf
            if not seen.any():
                continue
            for h in range(Hq):
                kk, vv = k[b][seen, h // group], v[b][seen, h // group]
                s = scale * (kk @ q[q0 + i, h])
                m = s.max()
                w = np.exp(s - m)
                out[q0 + i, h] = w @ vv / w.sum()
                weight[q0 + i, h] = w @ np.abs(vv) / w.sum()
                lse[q0 + i, h] = m + np.log(w.sum())
                spread[q0 + i, h] = (abs(scale) * (np.abs(kk) @ np.abs(q[q0 + i, h]))).max()
    return out, lse, weight, spread
