"""The attention block's operators around the FP8 projections (binding of
``include/fp8g_block.h``, where each one is defined).

Like the rest of the package this only checks tensors, allocates outputs and
workspaces with torch, and queues the library's kernels on torch's current
stream.  A decode step calls these once a layer, so that part is compiled
(csrc/block_binding.cpp); the functions here are its public signatures.
"""

import collections

import torch

from . import Fp8gError, _check, load

__all__ = ["lora_add", "lora_add_workspace", "qk_norm_rope", "KV4Cache", "kv4_cache", "kv4_append", "kv4_gather",
           "kv4_attention", "kv4_attention_workspace"]

_UNSUPPORTED = 6      # FP8G_ERR_UNSUPPORTED

_native = None


def _block():
    """The compiled binding (csrc/block_binding.cpp), loaded with the library."""
    global _native
    if _native is None:
        load()
        try:
            from . import _block as native
        except ImportError as e:
            raise RuntimeError("the binding _block is not built; run `python -m fp8_scaled_gemm_amd.build` (%s)" % e)
        _native = native
    return _native


def _done(result, where):
    """A result of the binding, or its status as an error."""
    if type(result) is int:
        _check(result, where)
    return result


def _bytes(need, where):
    """A workspace's size, or the refusal of its sizes as an error."""
    if need < 0:
        raise Fp8gError(_UNSUPPORTED, where)
    return need


def lora_add_workspace(tokens, n, k, rank, adapters, segments):
    """Bytes of workspace that lora_add needs for these sizes (0: none)."""
    return _bytes(load().lora_add_workspace(tokens, n, k, rank, adapters, segments), "lora_add_workspace")


def lora_add(base, x, A, B, scale, seg_start, seg_adapter, out=None, workspace=None):
    """base [T, n] + scale[a] * (x [T, k] @ A[a] [rank, k]^T) @ B[a] [n, rank]^T with
    the adapter a = seg_adapter[s] of the token's segment seg_start[s] <= t <
    seg_start[s + 1]; a negative adapter leaves base.

    base and out are bfloat16 or float32 (out may be base); x, A [N, rank, k]
    and B [N, n, rank] bfloat16; scale [N] float32; seg_start [S + 1] and
    seg_adapter [S] int32.  workspace: a device tensor to use instead of a
    fresh one from torch's allocator (lora_add_workspace gives its bytes).
    """
    return _done(_block().lora_add(base, x, A, B, scale, seg_start, seg_adapter, out, workspace), "lora_add")


def qk_norm_rope(q, k, q_weight, k_weight, positions, cos_sin, axis=None, eps=1e-6, interleaved=False, q_out=None,
                 k_out=None):
    """RMS norm of every head of q [T, Hq, D] and k [T, Hk, D] (over D, times
    q_weight / k_weight [D] float32 or None), then the rotation by the
    positions' rows of cos_sin [P, rotary_dim] float32 (cosines, then sines).

    q and k are bfloat16 or float32 and may be slices of one projection (any
    stride between tokens).  positions: int32 [T], or [axes, T] with axis
    [rotary_dim / 2] int32, the axis that turns each pair.  Pairs are (i, i +
    rotary_dim / 2), or (2i, 2i + 1) if interleaved.  q_out and k_out may be q
    and k themselves.  Returns (q_out, k_out).
    """
    return _done(_block().qk_norm_rope(q, k, q_weight, k_weight, positions, cos_sin, axis, eps, interleaved, q_out, k_out),
                 "qk_norm_rope")


class KV4Cache(collections.namedtuple("KV4Cache", "k k_scale v v_scale")):
    """A paged MXFP4 key/value cache: E2M1 codes k [pages, heads, page_size, dk
    / 2] and v [.., dv / 2], UE8M0 scale codes k_scale [pages, heads, dk / 32,
    page_size] and v_scale [.., dv / 32, page_size], all uint8."""

    __slots__ = ()


def kv4_cache(pages, heads, page_size, dk, dv, device="cuda"):
    """A cache of zeros for key rows of dk and value rows of dv elements
    ((64, 64), (128, 128) or (192, 128)); page_size a multiple of 16."""
    def empty(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device=device)
    return KV4Cache(empty(pages, heads, page_size, dk // 2), empty(pages, heads, dk // 32, page_size),
                    empty(pages, heads, page_size, dv // 2), empty(pages, heads, dv // 32, page_size))


def kv4_append(cache, k, v, slots):
    """Quantize key rows k [T, heads, dk] and value rows v [T, heads, dv]
    (bfloat16 or float32, any stride between tokens) to MXFP4 and write row t
    to slot slots[t] = page * page_size + row (int64; negative: skipped)."""
    _done(_block().kv4_append(*cache, k, v, slots), "kv4_append")


def kv4_gather(cache, slots, k_out=None, v_out=None, dtype=torch.bfloat16):
    """The values of the rows at slots (int64 [T]; zeros where negative) as
    (k [T, heads, dk], v [T, heads, dv]) of dtype bfloat16 or float32."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("dtype must be bfloat16 or float32, got %s" % dtype)
    return _done(_block().kv4_gather(*cache, slots, k_out, v_out, dtype is torch.float32), "kv4_gather")


def kv4_attention_workspace(queries, q_heads, kv_heads, dk, dv, batch, max_pages, page_size, window=0):
    """Bytes of workspace that kv4_attention needs for these sizes (0: none; at
    most 69 MB, whatever max_pages is)."""
    return _bytes(load().kv4_attention_workspace(queries, q_heads, kv_heads, dk, dv, batch, max_pages, page_size, window),
                  "kv4_attention_workspace")


def kv4_attention(q, cache, page_table, q_start, kv_len, scale=None, causal=True, window=0, out=None, lse=None,
                  return_lse=False, workspace=None):
    """Attention of q [Tq, Hq, dk] (bfloat16, any stride between queries) over a
    KV4Cache.  Sequence b has the queries q_start[b] .. q_start[b + 1] - 1
    (int32 [B + 1]), the last of its kv_len[b] (int32 [B]) positions, and the
    pages page_table[b] (int32 [B, max_pages]).  causal: a query sees no key
    behind its own position, and with window > 0 only the last `window` keys up
    to it.  scale defaults to dk ** -0.5.

    Returns out [Tq, Hq, dv] bfloat16, or (out, lse [Tq, Hq] float32) if
    return_lse or an lse tensor is given; a query that sees no key has out 0 and
    lse -inf.  workspace: a device tensor to use instead of a fresh one from
    torch's allocator (kv4_attention_workspace gives its bytes).
    """
    return _done(_block().kv4_attention(q, *cache, page_table, q_start, kv_len, scale, causal, window, out, lse, return_lse,
                                        workspace), "kv4_attention")
