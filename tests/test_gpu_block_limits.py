"""Sizes and arguments at the edge of what the attention block's operators take."""

import numpy as np
import pytest
import torch

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
