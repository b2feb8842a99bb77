"""Seeded inputs and bounds for the tests of the feed-forward half's operators."""

import numpy as np
import torch

from block_util import half_ulp, rng
from gpu_util import alignment
from oracle import e4m3, ffn


def operand(r, rows, k, mx, wide=False):
    """E4M3 codes [rows, k] of normal values (wide: of very different sizes) and their scales."""
    x = r.standard_normal((rows, k)) * 60.0
    if wide:
        x *= np.exp(1.5 * r.standard_normal((rows, k)))
    codes = e4m3.encode(np.clip(x, -448, 448).astype(np.float32))
    if mx:
        return codes, r.integers(116, 124, (rows, k // 32)).astype(np.uint8)
    return codes, (0.01 * np.exp(0.5 * r.standard_normal(rows))).astype(np.float32)


def want(A, B, sa, sb, mx, bias, act, gated, residual):
    """The exact result and its bound before the last rounding (oracle.ffn.fused)."""
    if A.shape[0] == 0 or B.shape[0] == 0:
        n = B.shape[0] // 2 if gated else B.shape[0]
        return np.zeros((A.shape[0], n)), np.zeros((A.shape[0], n))
    T = alignment(A, B, None if mx else sa, None if mx else sb, sa if mx else None, sb if mx else None) if A.shape[1] \
        else np.zeros((A.shape[0], B.shape[0]))
    return ffn.fused(A, B, sa, sb, mx, bias, act, gated, residual, T)


def rounded(exact, tol, dtype):
    """The bound with the rounding to dtype: half a step of what is rounded."""
    return tol + half_ulp(dtype) * (np.abs(exact) + tol)


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


__all__ = ["operand", "want", "rounded", "dev", "rng", "half_ulp"]
