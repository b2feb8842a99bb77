"""kv4_attention against the float64 definition: head layouts, lengths from
nothing to many steps, masks that leave rows empty, pages that end inside a
step, memory of no sequence full of NaN scales and wild table entries."""

import numpy as np
import pytest
import torch

from block_util import BF16_HALF, F32_HALF, Paged, bf16, close, host, rng
from gpu_util import say
from oracle import block

pytestmark = pytest.mark.gpu


def check(fp8g, q_lens, kv_lens, q_heads, kv_heads, dk, dv, page, causal, window, seed, scale=None, pad=(0, 0),
          q_pad=0, channel=1.0, stream=None):
    paged = Paged(kv_lens, kv_heads, dk, dv, page, seed, channel=channel)
    q_start = pad[0] + np.concatenate([[0], np.cumsum(q_lens)])
    Tq = int(q_start[-1]) + pad[1]
    q64, qt = bf16(rng(seed, 1).standard_normal((Tq, q_heads * dk + q_pad)))
    q64 = q64[:, :q_heads * dk].reshape(Tq, q_heads, dk)
    q = qt.cuda()[:, :q_heads * dk].unflatten(1, (q_heads, dk))
    scale = dk ** -0.5 if scale is None else scale
    say("kv4_attention", q_lens, kv_lens, q_heads, kv_heads, dk, dv, page, causal, window, seed)
    out = torch.full((Tq, q_heads, dv), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Tq, q_heads), 7.0, device="cuda")
    args = (q, paged.device(fp8g), torch.from_numpy(paged.table).cuda(),
            torch.from_numpy(q_start.astype(np.int32)).cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda())
    fp8g.kv4_attention(*args, scale=scale, causal=causal, window=window, out=out, lse=lse)
    torch.cuda.synchronize()
    want, want_lse, weight, spread = block.attention(q64, paged.k, paged.v, q_start, kv_lens, scale, causal, window)
    got, got_lse = host(out), host(lse)
    nowhere = np.isnan(want_lse)
    assert (got[nowhere] == 7.0).all() and (got_lse[nowhere] == 7.0).all(), "rows of no sequence were written"
    got, got_lse, want, want_lse, weight, spread = (a[~nowhere] for a in (got, got_lse, want, want_lse, weight, spread))
    empty = np.isinf(want_lse)
    assert (got[empty] == 0).all() and (got_lse[empty] == -np.inf).all(), "rows that see no key"
    # a score is a sum of dk products in float32 (dk roundings of at most the sum
    # of magnitudes), then two multiplications and a subtraction in units of log 2
    delta = (dk + 8) * F32_HALF * spread
    keys = max(list(kv_lens) + [1])
    # softmax weights: two roundings to bf16 cover the weight and the result;
    # scores move numerator and denominator, sums of `keys` terms
    tol = BF16_HALF * np.abs(want) + (BF16_HALF + 2 * np.expm1(delta) + (keys + 16) * F32_HALF)[..., None] * weight * 1.01
    # a weight below 2^-126 of the largest is no float32 number, nor is its share a bf16 result
    tol = tol + 2.0 ** -126 * keys * max([np.abs(v).max() for v in paged.v if v.size] + [0.0])
    close(got, want, tol, "out")
    close(got_lse[~empty], want_lse[~empty], (delta + (keys + 16) * F32_HALF + 4 * F32_HALF * np.abs(want_lse))[~empty], "lse")


DIMS = [(64, 64), (128, 128), (192, 128)]


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("kv", [1, 15, 16, 17, 63, 64, 65, 255, 256, 257, 700])
def test_one_query_each(gpu_lib, dk, dv, kv):
    check(gpu_lib, [1, 1, 1], [kv, 1, max(1, kv - 3)], 8, 2, dk, dv, 16, True, 0, kv + dk)


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (3, 3), (5, 1), (16, 2), (24, 1), (40, 2), (12, 4)])
@pytest.mark.parametrize("q_len", [1, 3])
def test_head_layouts(gpu_lib, q_heads, kv_heads, q_len):
    check(gpu_lib, [q_len, q_len], [130, 77], q_heads, kv_heads, 128, 128, 32, True, 0, q_heads * 10 + q_len)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_ragged_batch_with_empty_sequences(gpu_lib, causal, dk, dv):
    # no queries, no keys, fewer keys than queries (rows that see nothing), many queries
    check(gpu_lib, [1, 0, 5, 40, 3, 0, 33], [300, 20, 0, 12, 3, 0, 129], 4, 2, dk, dv, 16, causal, 0, 5)


@pytest.mark.parametrize("window", [1, 7, 64, 100, 1000])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_window(gpu_lib, window, dk, dv):
    check(gpu_lib, [1, 9, 70], [513, 400, 70], 6, 3, dk, dv, 16, True, window, window)


@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_page_sizes(gpu_lib, page):
    check(gpu_lib, [2, 1], [333, 97], 8, 4, 128, 128, page, True, 0, page)


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 90)])
@pytest.mark.parametrize("q_heads,kv_heads", [(4, 1), (3, 3)])
def test_prefill(gpu_lib, dk, dv, causal, window, q_heads, kv_heads):
    check(gpu_lib, [200, 131, 64], [200, 400, 70], q_heads, kv_heads, dk, dv, 16, causal, window, dk + q_heads)


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 33)])
@pytest.mark.parametrize("q_lens,kv_lens,q_heads,kv_heads", [
    ([200], [200], 2, 2),                       # one chunk of keys
    ([400, 260], [700, 260], 2, 2),             # several
    ([300, 0, 90], [120, 5, 90], 3, 1),         # rows in front of the first key
    ([17, 130], [0, 513], 40, 2)])              # a sequence without keys
def test_prefill_blocks(gpu_lib, dk, dv, causal, window, q_lens, kv_lens, q_heads, kv_heads):
    check(gpu_lib, q_lens, kv_lens, q_heads, kv_heads, dk, dv, 32, causal, window, dk + len(q_lens))


def test_long_context_is_split(gpu_lib):
    check(gpu_lib, [1], [5000], 4, 1, 128, 128, 16, True, 0, 1)
    check(gpu_lib, [2, 1, 1], [4100, 40, 0], 4, 2, 64, 64, 64, True, 0, 2)
    check(gpu_lib, [2, 1, 1], [4100, 40, 0], 4, 2, 192, 128, 64, True, 3000, 2)


def test_rows_of_no_sequence_and_strides(gpu_lib):
    check(gpu_lib, [3, 2], [50, 300], 4, 2, 128, 128, 16, True, 0, 3, pad=(5, 4), q_pad=64)
    check(gpu_lib, [70, 100], [90, 300], 4, 2, 128, 128, 16, True, 0, 3, pad=(5, 4), q_pad=64)


@pytest.mark.parametrize("q_len", [1, 80])
def test_large_scores(gpu_lib, q_len):
    # one key takes nearly all the weight, far channels
    check(gpu_lib, [q_len], [300], 4, 2, 128, 128, 16, True, 0, 4, scale=3.0, channel=2.0)


@pytest.mark.parametrize("q_len", [1, 100])
def test_scale_zero_and_negative(gpu_lib, q_len):
    check(gpu_lib, [q_len], [300], 4, 2, 64, 64, 16, False, 0, 4, scale=0.0)
    check(gpu_lib, [q_len], [300], 4, 2, 64, 64, 16, True, 0, 4, scale=-0.2)


def _setup(fp8g, q_lens, kv_lens, Hq=8, Hkv=2, dk=128, dv=128, page=16, seed=9):
    paged = Paged(kv_lens, Hkv, dk, dv, page, seed)
    q_start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = bf16(rng(seed).standard_normal((int(q_start[-1]), Hq, dk)))[1].cuda()
    return [q, paged.device(fp8g), torch.from_numpy(paged.table).cuda(), torch.from_numpy(q_start).cuda(),
            torch.tensor(kv_lens, dtype=torch.int32).cuda()]


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [900, 5, 2000]), ([100, 37], [500, 1200])])
def test_same_bits_every_time_on_any_stream(gpu_lib, q_lens, kv_lens):
    args = _setup(gpu_lib, q_lens, kv_lens)
    want, want_lse = gpu_lib.kv4_attention(*args, return_lse=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, lse = gpu_lib.kv4_attention(*args, return_lse=True)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [60, 9, 1]])
def test_graph_replays(gpu_lib, q_lens):
    args = _setup(gpu_lib, q_lens, [900, 70, 2000])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gpu_lib.kv4_attention(*args, return_lse=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = gpu_lib.kv4_attention(*args, return_lse=True)
    for step in range(4):
        args[0].copy_(torch.randn_like(args[0].float()))
        args[4].copy_(torch.tensor([900 - 100 * step, 70 - step, 2000 - 7 * step], dtype=torch.int32))
        graph.replay()
        want, want_lse = gpu_lib.kv4_attention(*args, return_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse), step


@pytest.mark.parametrize("q_len", [1, 50])
def test_pages_past_32_bit_offsets(gpu_lib, q_len):
    # codes of 4.3 GB and more in front of the pages in use
    Hkv, dk, page, L = 8, 128, 64, 500
    paged = Paged([L], Hkv, dk, dk, page, 21)
    far = (1 << 32) // (Hkv * page * dk // 2) + 5
    cache = []
    for a in paged.arrays:
        t = torch.empty((far + paged.pages,) + a.shape[1:], dtype=torch.uint8, device="cuda")
        t[far:] = torch.from_numpy(a).cuda()
        cache.append(t)
    near = gpu_lib.KV4Cache(*[t[far:].clone() for t in cache])
    q = bf16(rng(4).standard_normal((q_len, 16, dk)))[1].cuda()
    table = torch.from_numpy(np.maximum(np.minimum(paged.table, paged.pages - 1), 0)).cuda()
    start, length = torch.tensor([0, q_len], dtype=torch.int32).cuda(), torch.tensor([L], dtype=torch.int32).cuda()
    want = gpu_lib.kv4_attention(q, near, table, start, length)
    got = gpu_lib.kv4_attention(q, gpu_lib.KV4Cache(*cache), table + far, start, length)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_no_pages(gpu_lib):
    cache = gpu_lib.kv4_cache(0, 2, 16, 128, 128)
    q = torch.randn(3, 4, 128, device="cuda").bfloat16()
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    out, lse = gpu_lib.kv4_attention(q, cache, torch.zeros(1, 4, dtype=torch.int32, device="cuda"), ints(0, 3), ints(40),
                                     return_lse=True)
    assert (out == 0).all() and torch.isinf(lse).all()
    out = gpu_lib.kv4_attention(q[:0], cache, torch.zeros(1, 4, dtype=torch.int32, device="cuda"), ints(0, 0), ints(40))
    assert out.shape == (0, 4, 128)


def test_wild_lengths_stay_in_bounds(gpu_lib):
    # lengths beyond the table and starts beyond the queries are cut
    args = _setup(gpu_lib, [2, 2], [32, 32])
    args[2] = args[2][:, :2].contiguous()
    want = gpu_lib.kv4_attention(*args, causal=False)
    args[4] = torch.tensor([1 << 30, 100], dtype=torch.int32).cuda()
    args[3] = torch.tensor([-5, 2, 1 << 30], dtype=torch.int32).cuda()
    got = gpu_lib.kv4_attention(*args, causal=False)
    assert torch.equal(got, want)
