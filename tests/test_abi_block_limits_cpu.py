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


OK, UNSUPPORTED = 0, 6


def pointer(i):
    return 0x100000 + i * (1 << 42)


def test_launches_of_2_to_the_32_threads_are_refused(lib):
    """The runtime takes fewer than 2^32 threads along a dimension; the header
    promises a status for what the library does not do, before any HIP call."""
    p = [pointer(i) for i in range(12)]
    # 2^20 sequences of 16 key heads, a workgroup of 256 threads each at least
    assert lib.kv4_attention_workspace(1 << 20, 16, 16, 64, 64, 1 << 20, 1, 16, 0) == -1
    assert lib.kv4_attention(p[0], 16 * 64, 1 << 20, 16, p[1], p[2], p[3], p[4], 9, 16, 16, 64, 64, p[5], 1 << 20, 1, p[6],
                             p[7], 0.1, 1, 0, p[8], p[9], p[10], 1 << 40, None) == UNSUPPORTED
    assert lib.kv4_attention_workspace(1 << 19, 16, 16, 64, 64, 1 << 19, 1, 16, 0) >= 0
    # 16 tokens a workgroup
    for tokens, heads in ((1 << 28, 1), (1 << 24, 4096)):
        assert lib.kv4_append(p[0], heads * 64, p[1], heads * 64, 1, tokens, heads, 64, 64, p[2], 5, 16, p[3], p[4], p[5],
                              p[6], None) == UNSUPPORTED
        assert lib.kv4_gather(p[3], p[4], p[5], p[6], 5, 16, heads, 64, 64, p[2], tokens, 0, p[0], p[1], None) == UNSUPPORTED
    # 4 tokens a workgroup
    assert lib.qk_norm_rope(p[0], 256, p[1], 0, 0, 1 << 27, 1, 0, 256, p[2], p[3], 1e-6, p[4], 1, None, p[5], 100, 128, 0,
                            p[6], 256, p[7], 0, None) == UNSUPPORTED
    # 64 tokens and 64 ranks a workgroup
    assert lib.lora_add_workspace((1 << 28) - 1, 8, 8, 256, 1, 1) == -1
    assert lib.lora_add(p[0], p[1], p[2], p[3], p[4], p[5], p[6], (1 << 28) - 1, 8, 8, 256, 1, 1, 0, p[7], p[8], 1 << 50,
                        None) == UNSUPPORTED


def test_workspace_sizes_from_python(lib):
    assert fp8g.lora_add_workspace(8, 64, 64, 16, 2, 3) == lib.lora_add_workspace(8, 64, 64, 16, 2, 3) > 0
    assert fp8g.lora_add_workspace(0, 64, 64, 16, 2, 3) == 0
    assert fp8g.kv4_attention_workspace(4, 8, 2, 128, 128, 3, 40, 16) == \
        lib.kv4_attention_workspace(4, 8, 2, 128, 128, 3, 40, 16, 0) > 0
    for refused in (lambda: fp8g.lora_add_workspace(8, 64, 64, 12, 2, 3),
                    lambda: fp8g.kv4_attention_workspace(4, 8, 3, 128, 128, 3, 40, 16)):
        with pytest.raises(fp8g.Fp8gError) as e:
            refused()
        assert e.value.status == UNSUPPORTED
