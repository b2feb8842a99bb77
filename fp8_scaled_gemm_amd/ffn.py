"""The feed-forward half's operators around the FP8 products (binding of
``include/fp8g_ffn.h``, where each one is defined).

Like the rest of the package this only checks tensors, allocates outputs and
workspaces with torch, and queues the library's kernels on torch's current
stream; that part is compiled (csrc/ffn_binding.cpp), and the functions here are
its public signatures.
"""

import collections

import torch

from . import FMT_E4M3, load
from .block import _block, _bytes, _done

__all__ = ["NormQuant", "add_rms_norm_quantize", "fp8_gemm_fused", "mxfp8_gemm_fused", "gemm_fused_workspace", "MoeRoute", "moe_route",
           "moe_route_workspace", "fp8_moe_gemm", "mxfp8_moe_gemm", "moe_gemm_workspace", "moe_combine"]

_ACTS = {None: 0, "none": 0, "silu": 1, "gelu_tanh": 2}
_SCORES = {"softmax": 0, "sigmoid": 1}


def _choice(table, value, name):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError("%s must be one of %s, got %r" % (name, ", ".join(repr(k) for k in table), value)) from None


def _is_f32(D, out_dtype):
    """Whether the output is float32 (else bfloat16): out_dtype, or D's type."""
    dtype = out_dtype if out_dtype is not None else torch.bfloat16 if D is None else D.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32, got %s" % dtype)
    return dtype is torch.float32


class NormQuant(collections.namedtuple("NormQuant", "q scale sum norm")):
    """Codes q [R, C] and their scale (float32 [R], or UE8M0 codes [R, C / 32]);
    sum (x + residual) and norm where they were asked for, else None."""

    __slots__ = ()


def add_rms_norm_quantize(x, weight=None, residual=None, eps=1e-6, mx=False, fmt=FMT_E4M3, sum=None, norm=None, q=None,
                          scale=None, return_norm=False):
    """RMS norm of x [R, C] (bfloat16 or float32, any stride between rows), plus
    residual where given, times weight [C] float32, quantized to FP8: one scale a
    row (fmt FMT_E4M3 or FMT_E5M2), or with mx one UE8M0 code for 32 elements.

    Returns NormQuant(q, scale, sum, norm).  sum, the new residual stream, is
    there with a residual (it may be written over x or residual: sum=residual),
    norm, the normed rows in x's type, with return_norm or a norm tensor.
    """
    return NormQuant(*_done(_block().norm_quantize(x, weight, residual, eps, mx, fmt, sum, norm, q, scale, return_norm),
                            "add_rms_norm_quantize"))


def fp8_gemm_fused(m, n, k, A, B, scale_a, scale_b, bias=None, act=None, gated=False, residual=None, D=None,
                   out_dtype=None, workspace=None):
    """D [m, n] = act(z) + residual with z = scale_a * scale_b * (A [m, k] @ B [n, k]^T) + bias (E4M3 operands);
    gated: B [2 n, k] holds the gate and then the up projection, and D =
    act(z_gate) * z_up + residual.

    act: None, "silu" or "gelu_tanh"; bias float32 [n or 2 n]; residual of D's
    type, bfloat16 or float32, and may be D itself.  workspace: a device tensor
    to use instead of a fresh one (gemm_fused_workspace gives its bytes).
    """
    return _done(_block().gemm_fused(m, n, k, A, B, scale_a, scale_b, False, bias, _choice(_ACTS, act, "act"), gated, residual,
                                     D, _is_f32(D, out_dtype), workspace), "fp8_gemm_fused")


def mxfp8_gemm_fused(m, n, k, A, B, scale_a, scale_b, bias=None, act=None, gated=False, residual=None, D=None,
                     out_dtype=None, workspace=None):
    """fp8_gemm_fused with a UE8M0 code (uint8) for every 32 elements of k in
    scale_a [m, k / 32] and scale_b [n or 2 n, k / 32]."""
    return _done(_block().gemm_fused(m, n, k, A, B, scale_a, scale_b, True, bias, _choice(_ACTS, act, "act"), gated, residual,
                                     D, _is_f32(D, out_dtype), workspace), "mxfp8_gemm_fused")


def gemm_fused_workspace(m, n, k, gated=False, mx=False):
    """Bytes of workspace that fp8_gemm_fused (mx: mxfp8_gemm_fused) needs for these sizes."""
    return _bytes(load().gemm_fused_workspace(m, n, k, gated, mx), "gemm_fused_workspace")


class MoeRoute(collections.namedtuple("MoeRoute", "ids weights expert_start rows slots")):
    """Experts ids [T, k] of every token (-1: none) and their weights [T, k]; the
    routed rows sorted by expert: expert e has the slots expert_start[e] ..
    expert_start[e + 1] - 1, rows[slot] is a slot's token and slots[t, j] the
    slot of token t's j-th expert (-1: none).

    The five are parts of one allocation, which stays as long as one of them is
    kept, and which torch.save writes whole: clone() what outlives the step."""

    __slots__ = ()


def moe_route_workspace(tokens, experts, top_k):
    """Bytes of workspace that moe_route needs for these sizes."""
    return _bytes(load().moe_route_workspace(tokens, experts, top_k), "moe_route_workspace")


def moe_route(logits, top_k, bias=None, score="softmax", groups=1, top_groups=1, group_top=None, renormalize=True, scale=1.0,
              workspace=None):
    """The top_k experts of every token of logits [T, E] (bfloat16 or float32),
    by score "softmax" or "sigmoid" plus bias [E] float32 (for the choice only),
    among the top_groups of `groups` groups of experts with the largest sum of
    their group_top best (1 or 2; None: 2, or 1 where groups is 1).  Weights are
    the scores, divided by their sum with renormalize, times scale.  Experts with a
    logit or bias of -inf are not available.

    Returns MoeRoute(ids, weights, expert_start, rows, slots).  workspace: a
    device tensor to use instead of a fresh one (moe_route_workspace bytes).
    """
    if group_top is None:
        group_top = 1 if groups == 1 else 2
    return MoeRoute(*_done(_block().moe_route(logits, top_k, bias, _choice(_SCORES, score, "score"), groups, top_groups, group_top,
                                              renormalize, scale, workspace), "moe_route"))


def moe_gemm_workspace(slots, n, k, experts, gathered=True, gated=False, mx=False):
    """Bytes of workspace that fp8_moe_gemm (mx: mxfp8_moe_gemm) needs for these
    sizes; gathered: with rows."""
    return _bytes(load().moe_gemm_workspace(slots, n, k, experts, gathered, gated, mx), "moe_gemm_workspace")


def fp8_moe_gemm(A, B, scale_a, scale_b, expert_start, rows=None, bias=None, act=None, gated=False, D=None, out_dtype=None,
                 workspace=None):
    """The experts' products over routed rows: D [S, n], row s of expert e
    (expert_start[e] <= s < expert_start[e + 1], int32 [E + 1]) from A's row
    rows[s] (int32 [S]; None: s) and B[e], as fp8_gemm_fused computes it.

    A [Ra, k] and B [E, n or 2 n, k] E4M3; scale_a [Ra], scale_b and bias
    [E, n or 2 n] float32.  Rows of no expert are not written.  workspace: a
    device tensor to use instead of a fresh one (moe_gemm_workspace bytes).
    """
    return _done(_block().moe_gemm(A, B, scale_a, scale_b, False, expert_start, rows, bias, _choice(_ACTS, act, "act"), gated, D,
                                   _is_f32(D, out_dtype), workspace), "fp8_moe_gemm")


def mxfp8_moe_gemm(A, B, scale_a, scale_b, expert_start, rows=None, bias=None, act=None, gated=False, D=None, out_dtype=None,
                   workspace=None):
    """fp8_moe_gemm with UE8M0 codes scale_a [Ra, k / 32] and scale_b [E, n or 2 n, k / 32] (uint8)."""
    return _done(_block().moe_gemm(A, B, scale_a, scale_b, True, expert_start, rows, bias, _choice(_ACTS, act, "act"), gated, D,
                                   _is_f32(D, out_dtype), workspace), "mxfp8_moe_gemm")


def moe_combine(y, slots, weights, residual=None, out=None):
    """out [T, H] = residual + sum_j weights[t, j] * y[slots[t, j]] (y [S, H]
    bfloat16 or float32; slots int32 [T, k], negative: nothing; weights float32
    [T, k]).  out may be residual itself."""
    return _done(_block().moe_combine(y, slots, weights, residual, out), "moe_combine")
