"""Limits of the attention block's operators on the CPU: what a call may take in
memory and in launch size.  Pointers are never dereferenced."""

import itertools

import pytest

import fp8_scaled_gemm_amd as fp8g


@pytest.fixture(scope="module")
def lib():
    return fp8g.load()


def test_attention_workspace_does_not_follow_the_table(lib):
    """The page table is as wide as the longest context a server allows, in a
    captured graph always: the workspace must not grow with it."""
    for queries, batch, (heads, group), (dk, dv), window in itertools.product(
            (1, 64, 700, 8192, 100000), (1, 3, 64, 1000), ((1, 1), (8, 1), (8, 8), (2, 16)),
            ((64, 64), (128, 128), (192, 128)), (0, 4096)):
        for keys in (16, 8192, 1 << 17, 1 << 20, 1 << 30):
            need = lib.kv4_attention_workspace(queries, heads * group, heads, dk, dv, batch, keys // 16, 16, window)
            assert 0 <= need <= 69_000_000, (queries, batch, heads, group, dk, keys, window)
    # a prompt that fills the chip needs none
    for keys in (8192, 1 << 17, 1 << 20):
        assert lib.kv4_attention_workspace(8192, 64, 8, 128, 128, 1, keys // 16, 16, 0) == 0
