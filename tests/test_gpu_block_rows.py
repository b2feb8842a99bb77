"""kv4_append / kv4_gather (bit-exact), qk_norm_rope and lora_add against the
float64 definitions."""

import numpy as np
import pytest
import torch

from block_util import F32_HALF, close, half_ulp, host, rng, typed
from gpu_util import say
from oracle import block

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ the cache

def rows(r, T, H, D, dtype):
    x = r.standard_normal((T, H, D)) * np.exp(3 * r.standard_normal((T, H, 1)))
    if T > 2:
        x[0] = 0.0
        x[1, :, 1::2] = -0.0
        x[2, 0, :32] = 0.0
    edge = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]) * 2.0 ** r.integers(-20, 20)
    if T > 3:
        x[3, 0, :8], x[3, 0, 8:32] = edge, 0.1 * edge[0]          # ties
        x[3, 0, 16:24] = np.nextafter(edge.astype(np.float32), 0)
    if T > 5:
        x[4] = 1e-38 * r.standard_normal((H, D))                    # e at its lower end
        x[5] = 1.5e38 * np.sign(r.standard_normal((H, D)))          # and near its upper
    return typed(x, dtype)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("T,H,page", [(1, 1, 16), (7, 3, 16), (600, 1, 48), (33, 8, 64)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_append_and_gather(gpu_lib, dk, dv, T, H, page, dtype):
    r = rng(T, H, dk, page)
    pages = T // page + 3
    slots = r.permutation(pages * page)[:T].astype(np.int64)
    skip = r.random(T) < 0.2
    slots[skip] = r.choice([-1, -(1 << 40), pages * page, 1 << 40], skip.sum())
    k64, k = rows(r, T, H, dk, dtype)
    v64, v = rows(r, T, H, dv, dtype)
    say("kv4_append", dk, dv, T, H, page, dtype)
    pad = torch.zeros(T, 16, dtype=dtype)                           # token strides of their own
    k_dev = torch.cat([k.flatten(1), pad], 1).cuda()[:, :H * dk].unflatten(1, (H, dk))
    cache = gpu_lib.KV4Cache(*[torch.randint(0, 256, t.shape, dtype=torch.uint8, device="cuda")
                               for t in gpu_lib.kv4_cache(pages, H, page, dk, dv)])
    want = [t.cpu().numpy().copy() for t in cache]
    gpu_lib.kv4_append(cache, k_dev, v.cuda(), torch.from_numpy(slots).cuda())
    torch.cuda.synchronize()
    values = []
    for x, c, s, dim in ((k64, 0, 1, dk), (v64, 2, 3, dv)):
        codes, scales = block.mxfp4_quantize(x)
        for t in range(T):
            if 0 <= slots[t] < pages * page:
                at, row = divmod(int(slots[t]), page)
                want[c][at, :, row], want[s][at, :, :, row] = block.pack(codes[t]), scales[t]
        value = block.mxfp4_values(codes, scales)
        value[(slots < 0) | (slots >= pages * page)] = 0.0
        values.append(value)
    for got, w, name in zip(cache, want, gpu_lib.KV4Cache._fields):
        assert np.array_equal(got.cpu().numpy(), w), name           # untouched bytes too
    for dt in (BF, F):
        for got, w in zip(gpu_lib.kv4_gather(cache, torch.from_numpy(slots).cuda(), dtype=dt), values):
            assert got.dtype == dt and np.array_equal(host(got), w)


@pytest.mark.parametrize("T,H,dk,dv", [(1030, 2, 128, 128), (2049, 1, 192, 128), (1500, 3, 64, 64)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_append_many_rows(gpu_lib, T, H, dk, dv, dtype):
    test_append_and_gather(gpu_lib, dk, dv, T, H, 32, dtype)


def test_append_past_32_bit_offsets(gpu_lib):
    H, dk, page = 8, 128, 64
    pages = (1 << 32) // (H * page * dk // 2) + 4
    cache = gpu_lib.KV4Cache(*[torch.empty(t.shape, dtype=torch.uint8, device="cuda")
                               for t in (torch.empty(pages, H, page, dk // 2, device="meta"),
                                         torch.empty(pages, H, dk // 32, page, device="meta")) * 2])
    k64, k = rows(rng(5), 9, H, dk, BF)
    slots = (torch.arange(9) * 25 + (pages - 4) * page).cuda()
    gpu_lib.kv4_append(cache, k.cuda(), k.cuda(), slots)
    got = gpu_lib.kv4_gather(cache, slots)
    want = block.mxfp4_values(*block.mxfp4_quantize(k64))
    assert np.array_equal(host(got[0]), want) and np.array_equal(host(got[1]), want)


# ------------------------------------------------------------ norm and rotation

@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,Hq,Hk,D,rotary,axes,interleaved", [
    (1, 32, 8, 128, 128, 1, False), (5, 3, 1, 64, 32, 1, True), (37, 4, 4, 128, 64, 3, False),
    (3, 1, 1, 192, 192, 1, False), (300, 2, 1, 256, 256, 2, True), (9, 7, 2, 80, 16, 4, False),
    (2, 40, 0, 128, 128, 1, False), (2, 0, 5, 64, 64, 1, True), (2100, 10, 2, 64, 64, 1, False), (11, 1, 1, 8 * 11, 80, 2, True)])
@pytest.mark.parametrize("weights", [True, False])
def test_qk_norm_rope(gpu_lib, dtype, T, Hq, Hk, D, rotary, axes, interleaved, weights):
    r = rng(T, Hq, D, rotary)
    P = 500
    angle = r.uniform(-4, 4, (P, rotary // 2))
    table64, table = typed(np.concatenate([np.cos(angle), np.sin(angle)], 1), F)
    positions = r.integers(0, P, (axes, T)).astype(np.int32)
    axis = r.integers(0, axes, rotary // 2).astype(np.int32)
    x64, x = typed(r.standard_normal((T, (Hq + 2 * Hk) * D)) * np.exp(2 * r.standard_normal((T, 1))), dtype)
    x64[0] = 0.0
    x[0] = 0.0                                                       # a row of zeros
    w64, w = typed(1 + 0.3 * r.standard_normal((2, D)), F)
    say("qk_norm_rope", T, Hq, Hk, D, rotary, axes, interleaved, dtype, weights)
    dev = x.cuda()
    q = dev[:, :Hq * D].unflatten(1, (Hq, D)) if Hq else dev.new_empty(T, 0, D)
    k = dev[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)) if Hk else dev.new_empty(T, 0, D)
    pos = torch.from_numpy(positions).cuda()
    args = dict(eps=1e-5, interleaved=interleaved, axis=None if axes == 1 else torch.from_numpy(axis).cuda())
    wq, wk = (w[0].cuda(), w[1].cuda()) if weights else (None, None)
    got = gpu_lib.qk_norm_rope(q, k, wq, wk, pos[0] if axes == 1 else pos, table.cuda(), **args)
    eps = float(np.float32(1e-5))
    for g, part, wt in ((got[0], x64[:, :Hq * D].reshape(T, Hq, D), w64[0]),
                        (got[1], x64[:, Hq * D:(Hq + Hk) * D].reshape(T, Hk, D), w64[1])):
        if part.size == 0:
            continue
        want, mag = block.qk_norm_rope(part, wt if weights else None, positions, axis * (axes > 1), table64, eps, interleaved)
        # the sum of D squares, its root and reciprocal, and five products and sums a term, in float32
        tol = half_ulp(dtype) * np.abs(want) * 1.01 + (D / 2 + 12) * F32_HALF * mag
        close(host(g), want, tol, "qk_norm_rope")
    # in place, in the projection's own rows, the rest untouched
    before = dev.clone()
    gpu_lib.qk_norm_rope(q, k, wq, wk, pos[0] if axes == 1 else pos, table.cuda(), q_out=q, k_out=k, **args)
    assert torch.equal(q, got[0]) and torch.equal(k, got[1])
    assert torch.equal(dev[:, (Hq + Hk) * D:], before[:, (Hq + Hk) * D:])


def test_qk_positions_are_clamped(gpu_lib):
    q = torch.randn(4, 2, 64, device="cuda")
    angle = torch.rand(10, 32, device="cuda")
    table = torch.cat([angle.cos(), angle.sin()], 1)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    a = gpu_lib.qk_norm_rope(q, q, None, None, ints(-1 << 31, -1, 10, (1 << 31) - 1), table)
    b = gpu_lib.qk_norm_rope(q, q, None, None, ints(0, 0, 9, 9), table)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# -------------------------------------------------------------------- adapters

def lora_case(seed, T, n, k, rank, N, cuts, adapters, dtype):
    r = rng(seed, T, n, k, rank)
    base64, base = typed(r.standard_normal((T, n)), dtype)
    x64, x = typed(r.standard_normal((T, k)), BF)
    A64, A = typed(r.standard_normal((N, rank, k)) * max(k, 1) ** -0.5, BF)
    B64, B = typed(r.standard_normal((N, n, rank)), BF)
    s64, s = typed(r.uniform(0.5, 2, N), F)
    return (base64, x64, A64, B64, s64, cuts, adapters), [t.cuda() for t in (base, x, A, B, s)] + [
        torch.tensor(cuts, dtype=torch.int32).cuda(), torch.tensor(adapters, dtype=torch.int32).cuda()]


def lora_check(got, ref, k, rank, dtype):
    want, low, full = block.lora_add(*ref)
    # h in pieces of 16 (bf16) or 24 (float32) significant bits, k products and
    # rank * pieces products summed in float32, three roundings at the end
    tol = half_ulp(dtype) * np.abs(want) * 1.01 + (2.0 ** -16 if dtype == BF else 2.0 ** -22) * low + \
        (k + 3 * rank + 8) * F32_HALF * full + 2 * F32_HALF * np.abs(ref[0])
    close(host(got), want, tol, "lora_add")


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("rank", [8, 16, 24, 40, 64, 128, 200, 256])
@pytest.mark.parametrize("T,n,k", [(1, 64, 32), (37, 1001, 264), (130, 96, 1032)])
def test_lora(gpu_lib, dtype, rank, T, n, k):
    cuts = sorted({0, T // 5, T // 2, T - 1, T})
    adapters = [(2 * i + 1) % 3 if i != 1 else -1 for i in range(len(cuts) - 1)]
    ref, args = lora_case(1, T, n, k, rank, 3, cuts, adapters, dtype)
    say("lora_add", dtype, rank, T, n, k)
    got = gpu_lib.lora_add(*args)
    lora_check(got, ref, k, rank, dtype)
    torch.cuda.synchronize()
    again = gpu_lib.lora_add(*args)
    assert torch.equal(got, again)
    base = args[0]
    gpu_lib.lora_add(*args, out=base)                       # in place
    assert torch.equal(base, got)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("cuts,adapters", [
    ([0, 0, 0, 5, 5, 40], [0, 1, 2, 0, 1]),                 # empty segments
    ([3, 20, 30], [1, 2]),                                  # tokens of no segment in front and behind
    ([0, 16, 32, 40], [5, -3, 2]),                          # adapters that do not exist
    (list(range(41)), [i % 3 for i in range(40)]),          # a segment a token
    ([0], []),                                              # no segment
    ([-9, 7, 90], [1, 0])])                                 # starts outside
def test_lora_segments(gpu_lib, dtype, cuts, adapters):
    ref, args = lora_case(2, 40, 200, 520, 16, 3, cuts, adapters, dtype)
    lora_check(gpu_lib.lora_add(*args), ref, 520, 16, dtype)
    lora_check(gpu_lib.lora_add(*args, out=args[0]), ref, 520, 16, dtype)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T", [70, 1100])
def test_lora_long_segments(gpu_lib, dtype, T):
    ref, args = lora_case(3, T, 520, 2056, 64, 2, [0, T - 33, T], [1, 0], dtype)
    lora_check(gpu_lib.lora_add(*args), ref, 2056, 64, dtype)


# Long segments at ranks that end inside a unit of 32 or 64, empty segments and
# tokens of no segment between them, an odd number of columns.
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("rank", [8, 24, 40, 64, 72, 200, 256])
@pytest.mark.parametrize("T,n,k", [(530, 129, 72), (777, 1001, 8)])
def test_lora_long_segments_ranks(gpu_lib, dtype, rank, T, n, k):
    ref, args = lora_case(8, T, n, k, rank, 3, [5, 200, 200, T - 65, T - 1], [2, 1, -1, 0], dtype)
    say("lora_add", dtype, rank, T, n, k)
    got = gpu_lib.lora_add(*args)
    lora_check(got, ref, k, rank, dtype)
    base = args[0]
    gpu_lib.lora_add(*args, out=base)
    assert torch.equal(base, got)


@pytest.mark.parametrize("k,rank,N", [(0, 16, 2), (32, 0, 2), (32, 16, 0)])
def test_lora_nothing_to_add(gpu_lib, k, rank, N):
    ref, args = lora_case(4, 20, 100, k, rank, N, [0, 20], [0], BF)
    assert torch.equal(gpu_lib.lora_add(*args), args[0])
    gpu_lib.lora_add(*args, out=args[0])


def test_lora_keeps_what_other_adapters_hold_out(gpu_lib):
    # NaN in an adapter that no token uses, and infinities in x of tokens without one
    ref, args = lora_case(5, 64, 128, 256, 16, 3, [0, 20, 40, 64], [0, -1, 2], BF)
    args[2][1], args[3][1], args[1][20:40] = float("nan"), float("nan"), float("inf")
    ref[1][20:40] = 0
    lora_check(gpu_lib.lora_add(*args), ref, 256, 16, BF)


def test_binding_refuses(gpu_lib):
    """Wrong types, shapes, devices and layouts are errors of Python's own kinds;
    what the library refuses keeps its status."""
    _, args = lora_case(7, 8, 64, 64, 16, 2, [0, 8], [1], BF)
    base, x, A, B, scale, start, adapter = args

    def bad(kind, **change):
        names = dict(base=base, x=x, A=A, B=B, scale=scale, seg_start=start, seg_adapter=adapter)
        with pytest.raises(kind):
            gpu_lib.lora_add(**{**names, **change})

    bad(TypeError, x=x.float())
    bad(TypeError, base=base.half())
    bad(TypeError, A=None)
    bad(TypeError, seg_start=start.long())
    bad(ValueError, x=x.cpu())
    bad(ValueError, x=x[:, :32])
    bad(ValueError, B=B.transpose(1, 2))
    bad(ValueError, A=A.transpose(1, 2).contiguous().transpose(1, 2))
    bad(ValueError, out=base[:4])
    bad(ValueError, x=x[0])
    with pytest.raises(gpu_lib.Fp8gError) as e:
        gpu_lib.lora_add(*args, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 6
    with pytest.raises(gpu_lib.Fp8gError):
        gpu_lib.lora_add(base, x[:, :60].contiguous(), A[:, :, :60].contiguous(), B, scale, start, adapter)
    cache = gpu_lib.kv4_cache(4, 2, 16, 128, 128)
    rows_ = torch.zeros(3, 2, 128, device="cuda", dtype=BF)
    slots = torch.arange(3, device="cuda")
    for change in ({"k": rows_[:, :1]}, {"v": rows_.transpose(1, 2).contiguous().transpose(1, 2)}, {"slots": slots[:2]}):
        with pytest.raises(ValueError):
            gpu_lib.kv4_append(**{**dict(cache=cache, k=rows_, v=rows_, slots=slots), **change})
    with pytest.raises(TypeError):
        gpu_lib.kv4_append(cache, rows_, rows_, slots.int())
    with pytest.raises(TypeError):
        gpu_lib.kv4_gather(cache, slots, dtype=torch.float16)
    with pytest.raises(ValueError):
        gpu_lib.kv4_gather(gpu_lib.KV4Cache(*cache[:3], cache.v_scale[:, :, :2]), slots)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    q, table = torch.zeros(1, 4, 128, device="cuda", dtype=BF), torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(gpu_lib.Fp8gError) as e:
        gpu_lib.kv4_attention(q, cache, table, ints(0, 1), ints(5), causal=False, window=3)
    assert e.value.status == 2
    with pytest.raises(TypeError):
        gpu_lib.kv4_attention(q.float(), cache, table, ints(0, 1), ints(5))
    with pytest.raises(ValueError):
        gpu_lib.kv4_attention(q, cache, table, ints(0, 1, 1), ints(5))
    angle = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError):
        gpu_lib.qk_norm_rope(q, q, None, None, torch.zeros(3, 1, dtype=torch.int32, device="cuda"), angle)
    with pytest.raises(TypeError):
        gpu_lib.qk_norm_rope(q, q, None, None, torch.zeros(1, dtype=torch.int64, device="cuda"), angle)
    # a call after the refusals works
    assert torch.equal(gpu_lib.lora_add(*args), gpu_lib.lora_add(*args))


def test_block_step_in_a_graph(gpu_lib):
    """The operators of one decode step together, captured and replayed."""
    T, H, Hk, D, n = 6, 8, 2, 128, 12 * 128
    ref, args = lora_case(6, T, n, 512, 16, 4, list(range(T + 1)), [0, 1, -1, 3, 2, 2], BF)
    cache = gpu_lib.kv4_cache(12, Hk, 16, D, D)
    angle = torch.rand(100, 64, device="cuda")
    table = torch.cat([angle.cos(), angle.sin()], 1)
    pages = torch.arange(12, dtype=torch.int32, device="cuda").view(T, 2)
    starts = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    length = torch.zeros(T, dtype=torch.int32, device="cuda")
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")

    def step():
        qkv = gpu_lib.lora_add(*args)
        q, k = qkv[:, :H * D].unflatten(1, (H, D)), qkv[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D))
        v = qkv[:, (H + Hk) * D:].unflatten(1, (Hk, D))
        q, k = gpu_lib.qk_norm_rope(q, k, None, None, length, table)
        gpu_lib.kv4_append(cache, k, v, slots)
        return gpu_lib.kv4_attention(q, cache, pages, starts, length + 1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for at in (0, 1, 17, 5):
        args[1].normal_()
        length.fill_(at)
        slots.copy_(pages[:, at // 16].long() * 16 + at % 16)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step()), at
