"""Sizes and arguments at the edge of what the attention block's operators take."""

import numpy as np
import pytest
import torch

import test_gpu_block_attention as attention
import test_gpu_block_rows as rows
from block_util import rng
from gpu_util import say

pytestmark = pytest.mark.gpu


def test_many_more_segments_than_tokens(gpu_lib):
    # block numbers for 8192 segments times the columns' parts would be 2^32 threads
    T, S, n, k, rank = 2, 8192, 1 << 19, 64, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    base = torch.randn(T, n, generator=g, device="cuda")
    x, A, B = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((T, k), (1, rank, k), (1, n, rank)))
    start = torch.from_numpy(np.sort(rng(2).integers(0, 2, S + 1)).astype(np.int32)).cuda()
    start[0], start[-1] = 0, T
    say("lora_add", T, S, n)
    got = gpu_lib.lora_add(base, x, A, B, torch.ones(1, device="cuda"), start, torch.zeros(S, dtype=torch.int32, device="cuda"))
    want = base.double() + (x.double() @ A[0].double().T) @ B[0].double().T
    low = (x.double() @ A[0].double().T).abs() @ B[0].double().abs().T
    full = (x.double().abs() @ A[0].double().abs().T) @ B[0].double().abs().T
    # as in test_gpu_block_rows.py
    tol = 2.0 ** -24 * want.abs() * 1.01 + 2.0 ** -22 * low + (k + 3 * rank + 8) * 2.0 ** -24 * full + 2.0 ** -23 * base.abs()
    assert ((got.double() - want).abs() <= tol).all()


def guarded(need):
    """A workspace of exactly `need` bytes inside a larger allocation, and a check that the rest is untouched."""
    room = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")

    def check():
        assert (room[:4096] == 0xA5).all() and (room[4096 + need:] == 0xA5).all()
    return room[4096:4096 + need], check


@pytest.mark.parametrize("T,rank", [(40, 16), (600, 64)])
def test_own_workspace_of_the_adapters(gpu_lib, T, rank):
    ref, args = rows.lora_case(11, T, 200, 520, rank, 3, [0, 20, T], [2, 1], torch.bfloat16)
    workspace, check = guarded(gpu_lib.lora_add_workspace(T, 200, 520, rank, 3, 2))
    got = gpu_lib.lora_add(*args, workspace=workspace)
    check()
    rows.lora_check(got, ref, 520, rank, torch.bfloat16)
    assert torch.equal(got, gpu_lib.lora_add(*args))
    with pytest.raises(gpu_lib.Fp8gError):
        gpu_lib.lora_add(*args, workspace=workspace[:-1])


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [900, 5, 2000]), ([100, 37], [500, 1200])])
def test_own_workspace_of_attention(gpu_lib, q_lens, kv_lens):
    args = attention._setup(gpu_lib, q_lens, kv_lens)
    need = gpu_lib.kv4_attention_workspace(sum(q_lens), 8, 2, 128, 128, len(kv_lens), args[2].shape[1], 16)
    assert need > 0
    workspace, check = guarded(need)
    out, lse = gpu_lib.kv4_attention(*args, return_lse=True, workspace=workspace)
    check()
    want, want_lse = gpu_lib.kv4_attention(*args, return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    with pytest.raises(gpu_lib.Fp8gError):
        gpu_lib.kv4_attention(*args, workspace=workspace[:-1])


class NoTruth:
    def __bool__(self):
        raise ZeroDivisionError


def test_flags_without_a_truth_value(gpu_lib):
    """An argument's own error comes back, and nothing has been written."""
    args = attention._setup(gpu_lib, [1, 2], [40, 30])
    out = torch.full((3, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    for flag in ("causal", "return_lse"):
        with pytest.raises(ZeroDivisionError):
            gpu_lib.kv4_attention(*args, out=out, **{flag: NoTruth()})
    q = torch.ones(3, 2, 64, device="cuda")
    q_out = torch.full_like(q, 7.0)
    with pytest.raises(ZeroDivisionError):
        gpu_lib.qk_norm_rope(q, q, None, None, torch.zeros(3, dtype=torch.int32, device="cuda"),
                             torch.zeros(4, 64, device="cuda"), interleaved=NoTruth(), q_out=q_out)
    torch.cuda.synchronize()
    assert (out == 7.0).all() and (q_out == 7.0).all()


def test_host_tensors_are_refused(gpu_lib):
    """Every tensor of every operator, one at a time."""
    _, lora = rows.lora_case(7, 8, 64, 64, 16, 2, [0, 8], [1], torch.bfloat16)
    cache = gpu_lib.kv4_cache(4, 2, 16, 128, 128)
    row = torch.zeros(3, 2, 128, device="cuda", dtype=torch.bfloat16)
    slots = torch.arange(3, device="cuda")
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    weight, angle = torch.ones(128, device="cuda"), torch.zeros(4, 128, device="cuda")
    calls = [(gpu_lib.lora_add, lora),
             (gpu_lib.qk_norm_rope, [row, row, weight, weight, ints(0, 1, 2), angle]),
             (lambda *a: gpu_lib.kv4_append(gpu_lib.KV4Cache(*a[:4]), *a[4:]), [*cache, row, row, slots]),
             (lambda *a: gpu_lib.kv4_gather(gpu_lib.KV4Cache(*a[:4]), *a[4:]), [*cache, slots]),
             (lambda *a: gpu_lib.kv4_attention(a[0], gpu_lib.KV4Cache(*a[1:5]), *a[5:]),
              [row, *cache, torch.zeros(1, 2, dtype=torch.int32, device="cuda"), ints(0, 3), ints(5)])]
    for call, args in calls:
        call(*args)
        for i, arg in enumerate(args):
            with pytest.raises(ValueError):
                call(*args[:i], arg.cpu(), *args[i + 1:])
    torch.cuda.synchronize()
