"""Limits of the feed-forward half's operators that the host checks before any HIP
call.  Pointers are integers that are never dereferenced, and calls that would
pass every check are not made."""

import pytest

import fp8_scaled_gemm_amd as fp8g
from test_abi_ffn_cpu import UNSUPPORTED, moe, route

M = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return fp8g.load()


@pytest.mark.parametrize("mx", [False, True])
def test_experts_of_too_many_workgroups(lib, mx):
    """A workgroup of 256 threads for every 16 or 32 columns of an expert, two above 16 rows: 2^24 of them are too many."""
    for gated, cols in ((1, 16), (0, 32)):
        for S, shares in ((8, 1), (17, 2)):
            n = cols * ((1 << 24) // (1024 * shares))
            assert lib.moe_gemm_workspace(S, n - cols, 32, 1024, 1, gated, mx) == 0
            for wide in (n - cols + 1, n, 2 * M // (2 if gated else 1) - 16):
                assert lib.moe_gemm_workspace(S, wide, 32, 1024, 1, gated, mx) == -1
                assert moe(lib, mx, S=S, n=wide, k=32, E=1024, gated=gated, Ra=S) == UNSUPPORTED
    assert lib.moe_gemm_workspace(8, M, 32, 3, 1, 1, mx) == 0


def test_route_of_too_many_runs(lib):
    """A workgroup of 1024 threads for 64 tokens: 2^22 of them are too many."""
    assert lib.moe_route_workspace((1 << 28) - 64, 8, 1) == (1 << 22) * 8 * 4
    for T in ((1 << 28) - 63, (1 << 28) - 1):
        assert lib.moe_route_workspace(T, 8, 1) == -1
        assert route(lib, T=T, E=8, k=1, groups=1, top=1, each=1) == UNSUPPORTED
