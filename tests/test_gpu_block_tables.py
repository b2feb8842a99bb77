"""kv4_attention with page tables far wider than the contexts: the keys are cut
by the lengths, and what is left empty changes nothing."""

import numpy as np
import pytest
import torch

import block_util
import test_gpu_block_attention as attention
from block_util import rng

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[1 << 12, 1 << 17, 1 << 20])
def wide_tables(request, monkeypatch):
    """Tables of that many keys, full of entries that are no page behind a sequence's own."""
    class Wide(block_util.Paged):
        def __init__(self, *args, **kwargs):
            super().__init__(*args, **kwargs)
            more = max(0, request.param // self.page - self.max_pages)
            wild = rng(3).choice([-7, 1 << 30, -(1 << 31), 0], size=(len(self.table), more)).astype(np.int32)
            self.table = np.concatenate([self.table, wild], 1)
            self.max_pages += more
    monkeypatch.setattr(attention, "Paged", Wide)


@pytest.mark.parametrize("dk,dv", attention.DIMS)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 300)])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [2000, 1, 257]), ([5, 0, 2], [1030, 20, 0]),
                                            ([200, 130], [513, 1800]), ([300, 90], [120, 700])])
def test_wide_tables(gpu_lib, wide_tables, q_lens, kv_lens, causal, window, dk, dv):
    attention.check(gpu_lib, q_lens, kv_lens, 8, 2, dk, dv, 16, causal, window, dk + len(q_lens))


def test_many_chunks(gpu_lib, wide_tables):
    # one key head: more chunks than the lanes that join a row
    attention.check(gpu_lib, [1], [9000], 3, 1, 64, 64, 16, True, 0, 6)
    attention.check(gpu_lib, [1, 1], [9000, 40], 2, 1, 128, 128, 16, True, 0, 6)


def test_same_bits_from_every_run(gpu_lib, wide_tables):
    args = attention._setup(gpu_lib, [1, 1, 1], [900, 5, 2000])
    want, want_lse = gpu_lib.kv4_attention(*args, return_lse=True)
    for _ in range(3):
        out, lse = gpu_lib.kv4_attention(*args, return_lse=True)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
