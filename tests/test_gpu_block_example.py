"""The example's attention block: prompts, single tokens and a mix of both over
one cache, against float64 attention on the rows that the cache gives back."""

import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def load_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_attention_block(gpu_lib):
    example = load_example()
    block = example.AttentionBlock(hidden=512, q_heads=8, kv_heads=2, dim=64, pages=64, page_size=16, max_position=400)
    lengths, adapters = [0, 0, 0], [3, -1, 1]
    table = [[(7 * (20 * b + i)) % 61 for i in range(20)] for b in range(3)]      # pages in no order
    assert len({p for row in table for p in row}) == 60
    for new in ([70, 5, 200], [1, 1, 1], [1, 40, 1], [1, 0, 1]):
        step = example.plan(block, lengths, new, adapters, table)
        x = torch.randn(sum(new), block.hidden, device="cuda", generator=torch.Generator(device="cuda").manual_seed(sum(new))).bfloat16()
        q, k, v = block.qkv(x, step)
        out = block.attend(q, k, v, step)
        lengths = [a + b for a, b in zip(lengths, new)]
        at = 0
        for b, n in enumerate(new):
            slots = torch.tensor([table[b][p // 16] * 16 + p % 16 for p in range(lengths[b])], device="cuda")
            keys, values = (t.double().repeat_interleave(4, 1) for t in gpu_lib.kv4_gather(block.cache, slots))
            score = torch.einsum("qhd,khd->hqk", q[at:at + n].double(), keys) / math.sqrt(64)
            late = torch.arange(lengths[b], device="cuda") > torch.arange(lengths[b] - n, lengths[b], device="cuda")[:, None]
            want = torch.einsum("hqk,khd->qhd", score.masked_fill(late, -math.inf).softmax(-1), values)
            if n:
                # weights and result rounded to bf16: at most 2^-8 of the row's size each
                got = out[at:at + n].double()
                assert (got - want).norm() <= 2 * 2.0 ** -8 * want.norm(), (new, b)
            at += n
        y = block(x, step)
        assert y.shape == x.shape and torch.isfinite(y).all()
        assert torch.equal(y, block(x, step))
