"""The attention block's operators around the FP8 projections (binding of
``include/fp8g_block.h``, where each one is defined).

Like the rest of the package this only checks tensors, allocates outputs and
workspaces with torch, and queues the library's kernels on torch's current
stream.  A decode step calls these once a layer, so the checks are written to
cost little: plain attribute compares, no tensor operations.
"""

import collections

import torch

from . import OUT_BF16, OUT_F32, _check, load

__all__ = ["lora_add", "qk_norm_rope", "KV4Cache", "kv4_cache", "kv4_append", "kv4_gather", "kv4_attention"]

_BF16, _F32, _I32, _I64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
_CODES = {_BF16: OUT_BF16, _F32: OUT_F32}     # fp8g_out_t
_IN_CODES = {_F32: 0, _BF16: 1}               # fp8g_in_t


def _need(t, name, dtype, shape, device, dense=True):
    """t: a tensor on `device` (index) of that dtype and shape, contiguous unless dense is False."""
    if t.get_device() != device:
        if not t.is_cuda:
            raise ValueError("%s must be a device tensor" % name)
        # the kernels run on the current device and take raw pointers
        raise ValueError("%s is on %s but the current device is cuda:%d (call under torch.cuda.device(%s))"
                         % (name, t.device, device, t.device))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if dense and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _rows(t, name):
    """Elements between the tokens of t [T, H, D], whose rows of one token must be dense."""
    T, H, D = t.shape
    stride = t.stride()
    if H and D and ((D > 1 and stride[2] != 1) or (H > 1 and stride[1] != D)):
        raise ValueError("%s must be dense within a token (stride of the token axis is free), got strides %s"
                         % (name, stride))
    return stride[0] if T > 1 else H * D


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


def _workspace(given, need, device):
    """(pointer, bytes) of the caller's workspace, or of one from torch's allocator for this call, and its owner."""
    if given is None:
        if need == 0:
            return None, 0, None
        given = torch.empty(need, dtype=_U8, device="cuda:%d" % device)
    return given.data_ptr(), given.numel() * given.element_size(), given


def lora_add(base, x, A, B, scale, seg_start, seg_adapter, out=None, workspace=None):
    """base [T, n] + scale[a] * (x [T, k] @ A[a] [rank, k]^T) @ B[a] [n, rank]^T with
    the adapter a = seg_adapter[s] of the token's segment seg_start[s] <= t <
    seg_start[s + 1]; a negative adapter leaves base.

    base and out are bfloat16 or float32 (out may be base); x, A [N, rank, k]
    and B [N, n, rank] bfloat16; scale [N] float32; seg_start [S + 1] and
    seg_adapter [S] int32.  workspace: a device tensor to use instead of a
    fresh one from torch's allocator (lora_add_workspace gives its bytes).
    """
    dev = torch.cuda.current_device()
    if x.dim() != 2 or base.dim() != 2 or A.dim() != 3:
        raise ValueError("base and x must be 2-D, A and B 3-D")
    T, k = x.shape
    n = base.shape[1]
    N, rank, _ = A.shape
    S = seg_adapter.numel()
    code = _CODES.get(base.dtype)
    if code is None:
        raise TypeError("base must be bfloat16 or float32, got %s" % base.dtype)
    _need(base, "base", base.dtype, (T, n), dev)
    _need(x, "x", _BF16, (T, k), dev)
    _need(A, "A", _BF16, (N, rank, k), dev)
    _need(B, "B", _BF16, (N, n, rank), dev)
    _need(scale, "scale", _F32, (N,), dev)
    _need(seg_start, "seg_start", _I32, (S + 1,), dev)
    _need(seg_adapter, "seg_adapter", _I32, (S,), dev)
    if out is None:
        out = torch.empty_like(base)
    else:
        _need(out, "out", base.dtype, (T, n), dev)
    lib = load()
    ws, size, _owner = _workspace(workspace, max(0, lib.lora_add_workspace(T, n, k, rank, N, S)), dev)
    _check(lib.lora_add(base.data_ptr(), x.data_ptr(), A.data_ptr(), B.data_ptr(), scale.data_ptr(),
                        seg_start.data_ptr(), seg_adapter.data_ptr(), T, n, k, rank, N, S, code, out.data_ptr(),
                        ws, size, _stream(dev)), "lora_add")
    return out


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
    dev = torch.cuda.current_device()
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    T, Hq, D = q.shape
    Hk = k.shape[1]
    dt = q.dtype
    code = _CODES.get(dt)
    if code is None:
        raise TypeError("q must be bfloat16 or float32, got %s" % dt)
    _need(q, "q", dt, (T, Hq, D), dev, False)
    _need(k, "k", dt, (T, Hk, D), dev, False)
    if q_weight is not None:
        _need(q_weight, "q_weight", _F32, (D,), dev)
    if k_weight is not None:
        _need(k_weight, "k_weight", _F32, (D,), dev)
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    _need(positions, "positions", _I32, (T,) if positions.dim() == 1 else (axes, T), dev)
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [max_position, rotary_dim]")
    P, rotary = cos_sin.shape
    _need(cos_sin, "cos_sin", _F32, (P, rotary), dev)
    if axis is not None:
        _need(axis, "axis", _I32, (rotary // 2,), dev)
    elif axes > 1:
        raise ValueError("positions of several axes need axis, the axis of each pair")
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
    else:
        _need(q_out, "q_out", dt, (T, Hq, D), dev, False)
    if k_out is None:
        k_out = torch.empty((T, Hk, D), dtype=dt, device=q.device)
    else:
        _need(k_out, "k_out", dt, (T, Hk, D), dev, False)
    _check(load().qk_norm_rope(q.data_ptr(), _rows(q, "q"), k.data_ptr(), _rows(k, "k"), code, T, Hq, Hk, D,
                               None if q_weight is None else q_weight.data_ptr(),
                               None if k_weight is None else k_weight.data_ptr(), eps, positions.data_ptr(), axes,
                               None if axis is None else axis.data_ptr(), cos_sin.data_ptr(), P, rotary,
                               1 if interleaved else 0, q_out.data_ptr(), _rows(q_out, "q_out"), k_out.data_ptr(),
                               _rows(k_out, "k_out"), _stream(dev)), "qk_norm_rope")
    return q_out, k_out


class KV4Cache(collections.namedtuple("KV4Cache", "k k_scale v v_scale")):
    """A paged MXFP4 key/value cache: E2M1 codes k [pages, heads, page_size, dk
    / 2] and v [.., dv / 2], UE8M0 scale codes k_scale [pages, heads, dk / 32,
    page_size] and v_scale [.., dv / 32, page_size], all uint8."""

    __slots__ = ()


def kv4_cache(pages, heads, page_size, dk, dv, device="cuda"):
    """A cache of zeros for key rows of dk and value rows of dv elements
    ((64, 64), (128, 128) or (192, 128)); page_size a multiple of 16."""
    def empty(*shape):
        return torch.zeros(shape, dtype=_U8, device=device)
    return KV4Cache(empty(pages, heads, page_size, dk // 2), empty(pages, heads, dk // 32, page_size),
                    empty(pages, heads, page_size, dv // 2), empty(pages, heads, dv // 32, page_size))


def _sizes(cache, dev):
    """(pages, heads, page_size, dk, dv) of a cache, checked."""
    k, ks, v, vs = cache
    if k.dim() != 4 or v.dim() != 4:
        raise ValueError("the cache's codes must be [pages, heads, page_size, dim / 2]")
    pages, heads, page_size, dk = k.shape
    dv = v.shape[3]
    _need(k, "cache.k", _U8, (pages, heads, page_size, dk), dev)
    _need(ks, "cache.k_scale", _U8, (pages, heads, dk // 16, page_size), dev)
    _need(v, "cache.v", _U8, (pages, heads, page_size, dv), dev)
    _need(vs, "cache.v_scale", _U8, (pages, heads, dv // 16, page_size), dev)
    return pages, heads, page_size, 2 * dk, 2 * dv


def kv4_append(cache, k, v, slots):
    """Quantize key rows k [T, heads, dk] and value rows v [T, heads, dv]
    (bfloat16 or float32, any stride between tokens) to MXFP4 and write row t
    to slot slots[t] = page * page_size + row (int64; negative: skipped)."""
    dev = torch.cuda.current_device()
    pages, heads, page_size, dk, dv = _sizes(cache, dev)
    if k.dim() != 3:
        raise ValueError("k and v must be [tokens, heads, dim]")
    T, dt = k.shape[0], k.dtype
    code = _IN_CODES.get(dt)
    if code is None:
        raise TypeError("k must be bfloat16 or float32, got %s" % dt)
    _need(k, "k", dt, (T, heads, dk), dev, False)
    _need(v, "v", dt, (T, heads, dv), dev, False)
    _need(slots, "slots", _I64, (T,), dev)
    _check(load().kv4_append(k.data_ptr(), _rows(k, "k"), v.data_ptr(), _rows(v, "v"), code, T, heads, dk, dv,
                             slots.data_ptr(), pages, page_size, cache[0].data_ptr(), cache[1].data_ptr(),
                             cache[2].data_ptr(), cache[3].data_ptr(), _stream(dev)), "kv4_append")


def kv4_gather(cache, slots, k_out=None, v_out=None, dtype=_BF16):
    """The values of the rows at slots (int64 [T]; zeros where negative) as
    (k [T, heads, dk], v [T, heads, dv]) of dtype bfloat16 or float32."""
    dev = torch.cuda.current_device()
    pages, heads, page_size, dk, dv = _sizes(cache, dev)
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("dtype must be bfloat16 or float32, got %s" % dtype)
    T = slots.shape[0]
    _need(slots, "slots", _I64, (T,), dev)
    if k_out is None:
        k_out = torch.empty((T, heads, dk), dtype=dtype, device=slots.device)
    else:
        _need(k_out, "k_out", dtype, (T, heads, dk), dev)
    if v_out is None:
        v_out = torch.empty((T, heads, dv), dtype=dtype, device=slots.device)
    else:
        _need(v_out, "v_out", dtype, (T, heads, dv), dev)
    _check(load().kv4_gather(cache[0].data_ptr(), cache[1].data_ptr(), cache[2].data_ptr(), cache[3].data_ptr(), pages,
                             page_size, heads, dk, dv, slots.data_ptr(), T, code, k_out.data_ptr(), v_out.data_ptr(),
                             _stream(dev)), "kv4_gather")
    return k_out, v_out


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
    dev = torch.cuda.current_device()
    pages, heads, page_size, dk, dv = _sizes(cache, dev)
    if q.dim() != 3:
        raise ValueError("q must be [queries, q_heads, dk]")
    Tq, Hq, _ = q.shape
    B = kv_len.numel()
    if page_table.dim() != 2:
        raise ValueError("page_table must be [batch, max_pages]")
    max_pages = page_table.shape[1]
    _need(q, "q", _BF16, (Tq, Hq, dk), dev, False)
    _need(page_table, "page_table", _I32, (B, max_pages), dev)
    _need(q_start, "q_start", _I32, (B + 1,), dev)
    _need(kv_len, "kv_len", _I32, (B,), dev)
    if out is None:
        out = torch.empty((Tq, Hq, dv), dtype=_BF16, device=q.device)
    else:
        _need(out, "out", _BF16, (Tq, Hq, dv), dev)
    if lse is not None:
        _need(lse, "lse", _F32, (Tq, Hq), dev)
    elif return_lse:
        lse = torch.empty((Tq, Hq), dtype=_F32, device=q.device)
    lib = load()
    need = lib.kv4_attention_workspace(Tq, Hq, heads, dk, dv, B, max_pages, page_size, window)
    ws, size, _owner = _workspace(workspace, max(0, need), dev)
    _check(lib.kv4_attention(q.data_ptr(), _rows(q, "q"), Tq, Hq, cache[0].data_ptr(), cache[1].data_ptr(),
                             cache[2].data_ptr(), cache[3].data_ptr(), pages, page_size, heads, dk, dv,
                             page_table.data_ptr(), B, max_pages, q_start.data_ptr(), kv_len.data_ptr(),
                             dk ** -0.5 if scale is None else scale, 1 if causal else 0, window, out.data_ptr(),
                             None if lse is None else lse.data_ptr(), ws, size, _stream(dev)), "kv4_attention")
    return out if lse is None else (out, lse)
