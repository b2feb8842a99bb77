"""The attention block's operators at sizes whose loops go round several times:
steps of keys and their prefetch, maxima that grow while the sums run, rows of a
workgroup in flight, batches of k, strips of columns."""

import numpy as np
import pytest
import torch

import test_gpu_block_rows as rows
from block_util import BF16_HALF, F32_HALF, bf16, close, half_ulp, host, rng, typed
from gpu_util import say
from oracle import block

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


# ------------------------------------------------------------------- attention

class SharedPages:
    """A paged cache of one long run of keys, of which every sequence holds the
    first part.  Keys drift along one direction, so that the scores of a query
    rise or fall by some times its size from the first key to the last."""

    def __init__(self, lengths, heads, dk, dv, page, seed, drift):
        r = rng(seed, 78)
        n, counts = max(lengths), [(m + page - 1) // page for m in lengths]
        pages = max(counts) + 3
        order = r.permutation(pages)[:max(counts)]
        self.table = r.choice([-7, 1 << 30, -(1 << 31), 0], size=(len(lengths), max(counts) + 1)).astype(np.int32)
        for b, c in enumerate(counts):
            self.table[b, :c] = order[:c]
        place = (order[np.arange(n) // page], np.arange(n) % page)
        self.arrays, self.values = [], []
        for dim in (dk, dv):
            x = r.standard_normal((n, heads, dim))
            if not self.values:
                x += drift * (np.arange(n) / n)[:, None, None] * np.sign(r.standard_normal((heads, dim)))
            codes, scales = block.mxfp4_quantize(x.astype(np.float32))
            for part, shape in ((block.pack(codes), (pages, heads, page, dim // 2)), (scales, (pages, heads, dim // 32, page))):
                array = np.full(shape, 255, np.uint8)
                if shape[2] == page and part is not scales:
                    array[place[0], :, place[1]] = part
                else:
                    array[place[0], :, :, place[1]] = part
                self.arrays.append(array)
            self.values.append(block.mxfp4_values(codes, scales))

    def device(self, fp8g):
        return fp8g.KV4Cache(*[torch.from_numpy(a).cuda() for a in self.arrays])


def reference(q, k, v, length, scale, causal, window):
    """oracle.block.attention for one sequence's queries [n, Hq, dk], a head at a time."""
    n, Hq, _ = q.shape
    out, weight = np.zeros((n, Hq, v.shape[2])), np.zeros((n, Hq, v.shape[2]))
    lse, spread = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    p, j = length - n + np.arange(n)[:, None], np.arange(length)
    seen = np.ones((n, length), bool)
    if causal:
        seen = (j <= p) & ((j > p - window) if window else True)
    some = seen.any(1)
    for h in range(Hq):
        kk, vv = k[:length, h * k.shape[1] // Hq], v[:length, h * k.shape[1] // Hq]
        s = np.where(seen, scale * (q[:, h] @ kk.T), -np.inf)
        m = np.where(some, s.max(1), 0.0)
        w = np.exp(s - m[:, None])
        total = np.where(some, w.sum(1), 1.0)
        out[:, h], weight[:, h] = w @ vv / total[:, None], w @ np.abs(vv) / total[:, None]
        lse[some, h] = (m + np.log(total))[some]
        spread[:, h] = np.where(seen, abs(scale) * (np.abs(q[:, h]) @ np.abs(kk).T), 0.0).max(1)
    return out, lse, weight, spread


def check_attention(fp8g, q_lens, kv_lens, q_heads, kv_heads, dk, dv, causal, window, splits, drift, page=16):
    """splits: the chunks of a row that the sizes have to lead to."""
    cache = SharedPages(kv_lens, kv_heads, dk, dv, page, dk + len(q_lens), drift)
    q_start = np.concatenate([[0], np.cumsum(q_lens)])
    Tq, scale = int(q_start[-1]), dk ** -0.5
    q64, q = bf16(rng(dk, 5).standard_normal((Tq, q_heads, dk)))
    need = fp8g.kv4_attention_workspace(Tq, q_heads, kv_heads, dk, dv, len(q_lens), cache.table.shape[1], page, window)
    assert need == (Tq * q_heads * splits * (dv + 2) * 4 if splits > 1 else 0)
    say("kv4_attention", len(q_lens), Tq, max(kv_lens), q_heads, kv_heads, dk, dv, causal, window, drift)
    out, lse = fp8g.kv4_attention(q.cuda(), cache.device(fp8g), torch.from_numpy(cache.table).cuda(),
                                  torch.from_numpy(q_start.astype(np.int32)).cuda(),
                                  torch.tensor(kv_lens, dtype=torch.int32).cuda(), causal=causal, window=window, return_lse=True)
    got, got_lse = host(out), host(lse)
    for b, length in enumerate(kv_lens):
        mine = slice(int(q_start[b]), int(q_start[b + 1]))
        want, want_lse, weight, spread = reference(q64[mine], *cache.values, length, scale, causal, window)
        # as in test_gpu_block_attention.py
        delta = (dk + 8) * F32_HALF * spread
        tol = BF16_HALF * np.abs(want) + (BF16_HALF + 2 * np.expm1(delta) + (length + 16) * F32_HALF)[..., None] * weight * 1.01
        tol = tol + 2.0 ** -126 * length * np.abs(cache.values[1]).max()
        close(got[mine], want, tol, "out of sequence %d" % b)
        close(got_lse[mine], want_lse, delta + (length + 16) * F32_HALF + 4 * F32_HALF * np.abs(want_lse), "lse of sequence %d" % b)


DIMS = [(64, 64), (128, 128), (192, 128)]


def test_reference_is_the_oracle():
    r = rng(8)
    q, k, v = r.standard_normal((5, 6, 64)), r.standard_normal((40, 3, 64)), r.standard_normal((40, 3, 64))
    for causal, window in ((True, 0), (False, 0), (True, 7)):
        for a, b in zip(reference(q, k, v, 40, 0.3, causal, window), block.attention(q, [k], [v], [0, 5], [40], 0.3, causal, window)):
            assert np.allclose(a, b, rtol=1e-12, atol=1e-12)


# 16 rows a block: a wave takes a step of 64 keys in 256 of its chunk
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("drift", [0, 6, 40])
@pytest.mark.parametrize("q_len,batch,splits,window", [(1, 64, 1, 0), (3, 64, 1, 900), (2, 32, 2, 0)])
def test_few_rows_many_steps(gpu_lib, dk, dv, drift, q_len, batch, splits, window):
    # 64 sequences x 8 key heads fill the chip without splits; chunks of up to 1800 keys, or of 1024
    kv_lens = [700 + (i * 467) % 1101 for i in range(batch - 1)] + [1800]
    check_attention(gpu_lib, [q_len] * batch, kv_lens, 16, 8, dk, dv, True, window, splits, drift)


# 256 rows a block, 64 keys a step, two steps a round of the loop
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("drift", [0, 6, 40])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 300), (False, 0)])
def test_many_rows_many_steps(gpu_lib, dk, dv, drift, causal, window):
    # 8 sequences x 64 key heads: 5 to 12 steps, odd and even
    check_attention(gpu_lib, [256] * 8, [330, 384, 385, 449, 500, 640, 700, 705], 64, 64, dk, dv, causal, window, 1, drift)


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("causal", [True, False])
def test_many_rows_many_steps_of_chunks(gpu_lib, dk, dv, causal):
    # 256 blocks: two chunks of 512 keys and less
    check_attention(gpu_lib, [256, 250, 256, 240], [1024, 900, 770, 300], 64, 64, dk, dv, causal, 0, 2, 10)


# ------------------------------------------------------------ norm and rotation

@pytest.mark.parametrize("T,Hq,Hk,D,rotary,axes,interleaved,dtype,passes", [
    (2731, 90, 6, 128, 128, 3, False, BF, 12), (3001, 80, 8, 64, 64, 1, True, F, 11), (1101, 55, 5, 256, 192, 1, False, F, 15),
    (2801, 93, 3, 80, 48, 2, True, BF, 12), (4003, 63, 2, 64, 32, 1, False, BF, 4)])
def test_norm_many_rows_of_a_workgroup(gpu_lib, T, Hq, Hk, D, rotary, axes, interleaved, dtype, passes):
    """More rows than 2048 workgroups take at once: each goes round `passes` times, four in flight."""
    lanes = next(n for n in (8, 16, 32, 64) if 16 * n >= D * (2 if dtype == BF else 4))
    slots, heads = 256 // lanes, Hq + Hk
    all_passes = -(-T * heads // slots)
    tokens = min(-(-min(16, all_passes // 2048) * slots // heads), 16384 // (16 * D))
    assert all_passes > 2048 and tokens * heads // slots >= passes
    r = rng(T, D)
    angle = r.uniform(-4, 4, (700, rotary // 2))
    table64, table = typed(np.concatenate([np.cos(angle), np.sin(angle)], 1), F)
    positions, axis = r.integers(0, 700, (axes, T)).astype(np.int32), r.integers(0, axes, rotary // 2).astype(np.int32)
    x64, x = typed(r.standard_normal((T, heads * D)) * np.exp(2 * r.standard_normal((T, 1))), dtype)
    w64, w = typed(1 + 0.3 * r.standard_normal((2, D)), F)
    say("qk_norm_rope", T, Hq, Hk, D, rotary, axes, interleaved, dtype)
    dev = x.cuda()
    q, k = dev[:, :Hq * D].unflatten(1, (Hq, D)), dev[:, Hq * D:].unflatten(1, (Hk, D))
    pos = torch.from_numpy(positions).cuda()
    args = (w[0].cuda(), w[1].cuda(), pos[0] if axes == 1 else pos, table.cuda())
    more = dict(eps=1e-5, interleaved=interleaved, axis=None if axes == 1 else torch.from_numpy(axis).cuda())
    got = gpu_lib.qk_norm_rope(q, k, *args, **more)
    for g, part, wt in ((got[0], x64[:, :Hq * D].reshape(T, Hq, D), w64[0]), (got[1], x64[:, Hq * D:].reshape(T, Hk, D), w64[1])):
        want, mag = block.qk_norm_rope(part, wt, positions, axis * (axes > 1), table64, float(np.float32(1e-5)), interleaved)
        # as in test_gpu_block_rows.py
        close(host(g), want, half_ulp(dtype) * np.abs(want) * 1.01 + (D / 2 + 12) * F32_HALF * mag, "qk_norm_rope")
    gpu_lib.qk_norm_rope(q, k, *args, q_out=q, k_out=k, **more)
    assert torch.equal(q, got[0]) and torch.equal(k, got[1])


# -------------------------------------------------------------------- adapters

@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("rank", [8, 24, 64, 200])
def test_adapters_of_many_short_segments(gpu_lib, dtype, rank):
    # 600 blocks of one token: k in one part of 41 units of 64 and 24 more, 3 or 4 strips of 256 columns
    T, n, k = 600, 3001, 2648
    ref, args = rows.lora_case(12, T, n, k, rank, 3, list(range(T + 1)), [(5 * i) % 4 - 1 for i in range(T)], dtype)
    assert gpu_lib.lora_add_workspace(T, n, k, rank, 3, T) == T * rank * 4
    say("lora_add", T, n, k, rank, dtype)
    got = gpu_lib.lora_add(*args)
    rows.lora_check(got, ref, k, rank, dtype)
    gpu_lib.lora_add(*args, out=args[0])
    assert torch.equal(args[0], got)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("rank", [16, 64, 136])
def test_adapters_of_long_segments(gpu_lib, dtype, rank):
    # 64 blocks of 64 tokens and more: parts of k of 9 units, 3 strips of 128 columns
    T, n, k = 4096, 4001, 4616
    ref, args = rows.lora_case(13, T, n, k, rank, 3, [0, 1000, 1003, 2600, T], [2, 0, -1, 1], dtype)
    assert gpu_lib.lora_add_workspace(T, n, k, rank, 3, 4) == (8 if rank <= 64 else 2) * T * rank * 4
    say("lora_add", T, n, k, rank, dtype)
    got = gpu_lib.lora_add(*args)
    rows.lora_check(got, ref, k, rank, dtype)
    gpu_lib.lora_add(*args, out=args[0])
    assert torch.equal(args[0], got)
