"""NaN and infinity in the attention block's inputs: they reach the rows that
depend on them and no others."""

import numpy as np
import pytest
import torch

from block_util import BF16_HALF, F32_HALF, Paged, bf16, close, half_ulp, host, rng, typed
from gpu_util import say
from oracle import block

pytestmark = pytest.mark.gpu

# (queries and keys of each sequence, whether the keys of a row are cut into chunks
# that are joined), for the blocks of 16 rows and for those of 256
SHAPES = [([3, 2], [200, 30], False), ([1, 2, 1], [900, 5, 2000], True),
          ([200], [200], False), ([100, 90], [500, 1200], True)]


def attention(fp8g, q_lens, kv_lens, split, spoil, dk=128, dv=128, q_heads=8, kv_heads=2, scale=None, causal=True):
    """Runs with q and the cache as spoil(q, paged) leaves them.  Returns out and lse
    with what clean inputs give: (values, bounds) of both."""
    paged = Paged(kv_lens, kv_heads, dk, dv, 16, 31)
    q_start = np.concatenate([[0], np.cumsum(q_lens)])
    Tq = int(q_start[-1])
    q64, q = bf16(rng(32).standard_normal((Tq, q_heads, dk)))
    need = fp8g.load().kv4_attention_workspace(Tq, q_heads, kv_heads, dk, dv, len(kv_lens), paged.max_pages, 16, 0)
    assert (need > 0) == split
    used = dk ** -0.5 if scale is None or scale != scale else scale
    want, want_lse, weight, spread = block.attention(q64, paged.k, paged.v, q_start, kv_lens, used, causal, 0)
    spoil(q, paged)
    say("kv4_attention", q_lens, kv_lens, dk, dv, "not finite")
    out, lse = fp8g.kv4_attention(q.cuda(), paged.device(fp8g), torch.from_numpy(paged.table).cuda(),
                                  torch.from_numpy(q_start.astype(np.int32)).cuda(),
                                  torch.tensor(kv_lens, dtype=torch.int32).cuda(), scale=scale, causal=causal, return_lse=True)
    # as in test_gpu_block_attention.py
    delta, keys = (dk + 8) * F32_HALF * spread, max(kv_lens)
    tol = BF16_HALF * np.abs(want) + (BF16_HALF + 2 * np.expm1(delta) + (keys + 16) * F32_HALF)[..., None] * weight * 1.01
    tol_lse = delta + (keys + 16) * F32_HALF + 4 * F32_HALF * np.abs(want_lse)
    return host(out), host(lse), (want, tol), (want_lse, tol_lse)


def check(got, lse, out_ref, lse_ref, spoiled):
    """spoiled [Tq, Hq]: rows that have to be NaN; all others are as they were."""
    assert np.isnan(got[spoiled]).all() and np.isnan(lse[spoiled]).all(), "a row that depends on it"
    close(got[~spoiled], out_ref[0][~spoiled], out_ref[1][~spoiled], "out")
    sees = ~spoiled & ~np.isinf(lse_ref[0])
    close(lse[sees], lse_ref[0][sees], lse_ref[1][sees], "lse")
    empty = ~spoiled & np.isinf(lse_ref[0])
    assert (got[empty] == 0).all() and (lse[empty] == -np.inf).all()


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("q_lens,kv_lens,split", SHAPES)
def test_query(gpu_lib, q_lens, kv_lens, split, value, dk, dv):
    rows = [(0, 1), (sum(q_lens) - 1, 6)]           # the second also of a sequence with other lengths

    def spoil(q, paged):
        for t, h in rows:
            q[t, h, 5] = value
    out = attention(gpu_lib, q_lens, kv_lens, split, spoil, dk, dv, causal=False)
    spoiled = np.zeros(out[1].shape, bool)
    spoiled[tuple(zip(*rows))] = True
    check(*out, spoiled)


@pytest.mark.parametrize("q_lens,kv_lens", [([3, 1], [900, 40]), ([200, 100], [1500, 300])])
def test_keys(gpu_lib, q_lens, kv_lens):
    # the first 256 keys of one key head of sequence 0: whole chunks of nothing but NaN
    def spoil(q, paged):
        for j in range(256):
            paged.arrays[1][paged.table[0, j // 16], 1, :, j % 16] = 255
    out = attention(gpu_lib, q_lens, kv_lens, True, spoil)
    spoiled = np.zeros(out[1].shape, bool)
    spoiled[:q_lens[0], 4:] = True
    check(*out, spoiled)


@pytest.mark.parametrize("q_lens,kv_lens", [([40, 3], [12, 100]), ([300, 40], [120, 90])])
def test_rows_without_keys_stay_zero(gpu_lib, q_lens, kv_lens):
    # rows in front of the first key, beside rows of the same block that see NaN keys and values
    def spoil(q, paged):
        for j in range(kv_lens[0]):
            for i in (1, 3):
                paged.arrays[i][paged.table[0, j // 16], 0, :, j % 16] = 255
    out = attention(gpu_lib, q_lens, kv_lens, False, spoil)
    spoiled = np.zeros(out[1].shape, bool)
    spoiled[q_lens[0] - kv_lens[0]:q_lens[0], :4] = True
    check(*out, spoiled)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,kv_lens,split", SHAPES + [([300, 40], [120, 90], False), ([40, 3, 1], [12, 900, 0], True)])
def test_scale(gpu_lib, q_lens, kv_lens, split, causal):
    out = attention(gpu_lib, q_lens, kv_lens, split, lambda q, paged: None, scale=float("nan"), causal=causal)
    check(*out, ~np.isinf(out[3][0]))           # all but rows that see no key


# short segments and long ones (those at rank 64), two pieces of h and three
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,rank", [(40, 16), (600, 64)])
def test_adapter_sums_at_the_end_of_float32(gpu_lib, dtype, T, rank):
    r = rng(T, rank)
    n, k, N = 200, 256, 2
    base64, base = typed(r.standard_normal((T, n)), dtype)
    x64, x = bf16(r.standard_normal((T, k)))
    A64, A = bf16(r.standard_normal((N, rank, k)) * k ** -0.5)
    B64, B = bf16(0.25 * np.sign(r.standard_normal((N, n, rank))))
    # columns 7 and 8 of x count in rank 3 of adapter 0 only
    for a in (A64, A):
        a[0, :, 7:9] = 0.0
        a[0, 3, 7], a[0, 3, 8] = 255 / 128, 0.75
    over, most, nan = 5, 11, 13
    for t, pair in ((over, (3e38, 3e38)), (most, (2.0 ** 127, 2.0 ** 120)), (nan, (float("nan"), 0.0))):
        x[t, 7], x[t, 8] = pair
        x64[t, 7:9] = x[t, 7:9].double().numpy()
    # most: h = 255.75 * 2^120, above every bf16 number and below 2^128
    cuts, adapters = [0, 20, T], [0, 1]
    say("lora_add", T, rank, dtype, "not finite")
    got = host(gpu_lib.lora_add(base.cuda(), x.cuda(), A.cuda(), B.cuda(), torch.ones(N, device="cuda"),
                                torch.tensor(cuts, dtype=torch.int32).cuda(), torch.tensor(adapters, dtype=torch.int32).cuda()))
    assert np.isnan(got[nan]).all()
    # 1.2e39 in float32
    assert np.array_equal(got[over], np.inf * np.sign(B64[0, :, 3]))
    rest = np.ones(T, bool)
    rest[[over, nan]] = False
    x64[~rest] = 0.0
    want, low, full = block.lora_add(base64, x64, A64, B64, np.ones(N), cuts, adapters)
    # as in test_gpu_block_rows.py
    tol = half_ulp(dtype) * np.abs(want) * 1.01 + (2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -22) * low + \
        (k + 3 * rank + 8) * F32_HALF * full + 2 * F32_HALF * np.abs(base64)
    close(got[rest], want[rest], tol[rest], "lora_add")
