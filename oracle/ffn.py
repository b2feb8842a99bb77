"""The feed-forward half's operators in float64 -- oracle, test infrastructure.

Plain restatements of the definitions in include/fp8g_ffn.h, with the error
bounds that the GPU results are held to.
"""

import numpy as np

from . import gemm

EPS32 = 2.0 ** -24        # half a step of float32, relative


def rms_norm(s, weight, eps):
    """y = s / sqrt(mean s^2 + eps) * weight over the last axis, float64."""
    s = np.asarray(s, np.float64)
    y = s / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    return y if weight is None else y * np.asarray(weight, np.float64)


def activate(z, act):
    if act == "silu":
        p = z
    elif act == "gelu_tanh":
        p = 2.0 * np.sqrt(2.0 / np.pi) * (z + 0.044715 * z ** 3)
    else:
        return z, np.zeros_like(z)
    with np.errstate(over="ignore"):
        v = z / (1.0 + np.exp(-p))
    return v, (4 + np.abs(p)) * 2.0 ** -22 * np.abs(v)


SLOPE = 1.13              # the activations' largest derivative: silu 1.0998, gelu 1.1290


def fused(A, B, sa, sb, mx, bias, act, gated, residual, T):
    """(D, bound): the exact result and how far an fp32 computation with the
    matrix core's truncation term T may be from it, before the last rounding."""
    if mx:
        z, W = gemm.mxfp8_gemm(A, B, sa, sb), gemm.mxfp8_gemm_weight(A, B, sa, sb)
    else:
        z, W = gemm.gemm_scaled(A, B, sa, sb), gemm.gemm_scaled_weight(A, B, sa, sb)
    tol = gemm.REL_TOL * W + T
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    tol = tol + EPS32 * np.abs(z) * 3          # the two scales' products and the bias
    n = B.shape[0] // 2 if gated else B.shape[0]
    v, own = activate(z[:, :n], act)
    tol_v = (SLOPE if act not in (None, "none") else 1.0) * tol[:, :n] + own
    if gated:
        up, tol_u = z[:, n:], tol[:, n:]
        tol_v = tol_v * (np.abs(up) + tol_u) + np.abs(v) * tol_u + EPS32 * np.abs(v * up)
        v = v * up
    if residual is not None:
        v = v + np.asarray(residual, np.float64)
        tol_v = tol_v + EPS32 * np.abs(v)
    return v, tol_v


def route(logits, top_k, bias=None, score="softmax", groups=1, top_groups=1, group_top=2, renormalize=True, scale=1.0):
    """Token by token, expert by expert: (ids, weights, expert_start, rows, slots)."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    ids, weights = np.full((T, top_k), -1, np.int32), np.zeros((T, top_k))
    for t in range(T):
        there = [e for e in range(E) if logits[t, e] > -np.inf]      # NaN: not there
        p = np.zeros(E)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                p[there] = 1.0 / (1.0 + np.exp(-logits[t, there]))
        elif there:
            m = max(logits[t, there])
            d = np.array([0.0 if logits[t, e] == m else logits[t, e] - m for e in there])
            p[there] = np.exp(d) / np.exp(d).sum()
        value = p if bias is None else p + np.asarray(bias, np.float64)
        there = [e for e in there if value[e] > -np.inf]
        if groups > 1:
            width = E // groups
            best = []
            for q in range(groups):
                mine = sorted((value[e] for e in there if e // width == q), reverse=True)
                best.append(sum(mine[:group_top]) if len(mine) >= group_top else -np.inf)
            kept = sorted(range(groups), key=lambda q: (-best[q], q))[:top_groups]
            there = [e for e in there if e // width in kept]
        key = logits[t] if bias is None else value
        chosen = sorted(there, key=lambda e: (-key[e], e))[:top_k]
        w = p[chosen]
        if renormalize:
            w = w / w.sum() if len(chosen) and w.sum() > 0 else np.zeros(len(chosen))
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = w * scale
    start, rows, slots = [0], [], np.full((T, top_k), -1, np.int32)
    for e in range(E):
        for t in range(T):
            for j in np.flatnonzero(ids[t] == e):
                slots[t, j] = len(rows)
                rows.append(t)
        start.append(len(rows))
    rows += [-1] * (T * top_k - len(rows))
    return ids, weights, np.array(start, np.int32), np.array(rows, np.int32), slots


def combine(y, slots, weights, residual):
    """(out, sum of the terms' magnitudes), float64."""
    y, weights = np.asarray(y, np.float64), np.asarray(weights, np.float64)
    T, k = slots.shape
    out = np.zeros((T, y.shape[1])) if residual is None else np.array(residual, np.float64)
    size = np.abs(out)
    for t in range(T):
        for j in range(k):
            if 0 <= slots[t, j] < len(y):
                out[t] += weights[t, j] * y[slots[t, j]]
                size[t] += np.abs(weights[t, j] * y[slots[t, j]])
    return out, size
