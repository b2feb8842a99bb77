"""fp8_gemm_fused / mxfp8_gemm_fused and the experts' products against the
float64 definitions, element by element within the derived bound."""

import numpy as np
import pytest
import torch

from block_util import close, host, rng, typed
from ffn_util import dev, operand, rounded, want
from gpu_util import say

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
KINDS = [("none", False), ("silu", False), ("gelu_tanh", False), ("none", True), ("silu", True), ("gelu_tanh", True)]


def call_of(gpu_lib, mx):
    return gpu_lib.mxfp8_gemm_fused if mx else gpu_lib.fp8_gemm_fused


def case(gpu_lib, m, n, k, mx, act, gated, bias, residual, dtype, wide=False):
    r = rng(m, n, k, mx, gated)
    rows = 2 * n if gated else n
    A, sa = operand(r, m, k, mx, wide)
    B, sb = operand(r, rows, k, mx, wide)
    b = r.standard_normal(rows).astype(np.float32) if bias else None
    res64, res = typed(r.standard_normal((m, n)), dtype) if residual else (None, None)
    say("fused", m, n, k, mx, act, gated, bias, residual, dtype)
    exact, tol = want(A, B, sa, sb, mx, b, act, gated, res64)
    D = call_of(gpu_lib, mx)(m, n, k, dev(A), dev(B), dev(sa), dev(sb), bias=dev(b), act=act, gated=gated,
                             residual=None if res is None else res.cuda(), out_dtype=dtype)
    assert D.dtype == dtype and D.shape == (m, n)
    close(host(D), exact, rounded(exact, tol, dtype), "D")
    if residual:
        here = res.cuda()
        again = call_of(gpu_lib, mx)(m, n, k, dev(A), dev(B), dev(sa), dev(sb), bias=dev(b), act=act, gated=gated,
                                     residual=here, D=here)
        assert again.data_ptr() == here.data_ptr() and torch.equal(again, D)


@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (1, 128, 512), (3, 40, 96), (16, 64, 2048), (17, 33, 160), (65, 130, 1056),
                                   (130, 272, 384), (300, 520, 128), (257, 384, 800)])
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("act,gated", KINDS)
def test_fused(gpu_lib, m, n, k, mx, act, gated):
    case(gpu_lib, m, n, k, mx, act, gated, bias=m != 16, residual=n != 40, dtype=BF if (m + n) % 2 else F)


@pytest.mark.parametrize("m", [1, 20, 140])
@pytest.mark.parametrize("k", [16, 48, 144, 2000])
@pytest.mark.parametrize("gated", [False, True])
def test_fused_k_of_16(gpu_lib, m, k, gated):
    case(gpu_lib, m, 72, k, False, "silu", gated, bias=True, residual=False, dtype=BF)


@pytest.mark.parametrize("m,n,k", [(700, 1000, 640), (1100, 520, 256), (515, 2050, 1152), (2000, 1032, 128), (64, 4096, 512)])
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [BF, F])
def test_fused_large(gpu_lib, m, n, k, mx, gated, dtype):
    case(gpu_lib, m, n, k, mx, "silu" if gated else "none", gated, bias=True, residual=True, dtype=dtype, wide=True)


# K that ends inside a stage, rows of scales that are no whole dwords, rows of D that are no whole vectors
@pytest.mark.parametrize("m,n,k", [(600, 1032, 672), (515, 2050, 160), (700, 1001, 992), (1400, 523, 1056), (129, 255, 4192), (80, 131, 8224)])
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [BF, F])
def test_fused_tails(gpu_lib, m, n, k, mx, gated, dtype):
    case(gpu_lib, m, n, k, mx, "silu" if gated else "none", gated, bias=n % 2 == 1, residual=True, dtype=dtype)


# few tiles and a long K: partial sums of K ranges
@pytest.mark.parametrize("m,n,k", [(64, 512, 8192), (200, 256, 6144), (33, 1000, 16384), (129, 130, 4160)])
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_fused_long_k(gpu_lib, m, n, k, mx, gated):
    case(gpu_lib, m, n, k, mx, "gelu_tanh" if gated else "none", gated, bias=True, residual=True, dtype=BF if n % 2 else F)


@pytest.mark.parametrize("mx", [False, True])
def test_fused_empty(gpu_lib, mx):
    call = call_of(gpu_lib, mx)
    for m, n in ((0, 16), (5, 0)):
        A, sa = operand(rng(1), m, 64, mx)
        B, sb = operand(rng(2), n, 64, mx)
        assert call(m, n, 64, dev(A), dev(B), dev(sa), dev(sb)).shape == (m, n)
    A, sa = operand(rng(1), 5, 0, mx)
    B, sb = operand(rng(2), 2 * 24, 0, mx)
    bias = rng(3).standard_normal(48).astype(np.float32)
    got = call(5, 24, 0, dev(A), dev(B), dev(sa), dev(sb), bias=dev(bias), act="silu", gated=True, out_dtype=F)
    exact, tol = want(A, B, sa, sb, mx, bias, "silu", True, None)
    close(host(got), exact, rounded(exact, tol, F), "k = 0")


@pytest.mark.parametrize("m,n", [(300, 200), (700, 1031)])
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_no_k_of_many_rows(gpu_lib, m, n, mx, gated):
    case(gpu_lib, m, n, 0, mx, "silu", gated, bias=True, residual=True, dtype=BF)
    if not gated:
        experts_case(gpu_lib, m, 3, n, 0, mx, False, "even", True, F, True)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_activations_over_their_range(gpu_lib, act):
    """k = 0 and a bias: the activation alone, from far negative to far positive."""
    z = np.concatenate([np.linspace(-120, 120, 4001), [0.0, -0.0, 1e-30, -1e-30, 1e20, -1e20, 3e38, -3e38]]).astype(np.float32)
    n = len(z)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    got = gpu_lib.fp8_gemm_fused(1, n, 0, none.view(1, 0), none.view(n, 0), dev(np.ones(1, np.float32)), dev(np.ones(n, np.float32)),
                                 bias=dev(z), act=act, out_dtype=F)
    from oracle import ffn
    v, own = ffn.activate(z.astype(np.float64), act)
    # past |p| of 87 the exponential passes 2^126: results below the smallest normal may be 0
    close(host(got)[0], v, own + 2.0 ** -24 * np.abs(v) + 2.0 ** -126 * np.maximum(1, np.abs(z.astype(np.float64))), act)


# ------------------------------------------------------------------ experts

def split(r, S, E, how):
    """Expert starts of S slots: even, one takes nearly all, or many without a slot."""
    if how == "even":
        cuts = np.sort(r.integers(0, S + 1, E - 1)) if E > 1 else []
        return np.concatenate([[0], cuts, [S]]).astype(np.int32)
    if how == "one":
        cut = np.full(E + 1, S)
        cut[:E // 2 + 1] = 0
        return cut.astype(np.int32)
    cut = np.sort(r.integers(0, max(1, S - S // 5) + 1, E + 1))
    cut[1::3] = cut[0::3][:len(cut[1::3])]                     # every third expert has none; slots left over at both ends
    return np.sort(cut).astype(np.int32)


def experts_case(gpu_lib, S, E, n, k, mx, gated, how, gather, dtype, bias):
    r = rng(S, E, n, k, mx, gather)
    rows = 2 * n if gated else n
    Ra = max(1, S // 3) if gather else S
    A, sa = operand(r, Ra, k, mx)
    B, sb = operand(r, E * rows, k, mx)
    B, sb = B.reshape(E, rows, k), sb.reshape(E, rows, -1) if mx else sb.reshape(E, rows)
    start = split(r, S, E, how)
    index = r.integers(0, Ra, S).astype(np.int32) if gather else None
    b = r.standard_normal((E, rows)).astype(np.float32) if bias else None
    act = "silu" if gated else "none"
    say("experts", S, E, n, k, mx, gated, how, gather, dtype)
    D = torch.full((S, n), 777.0, dtype=dtype, device="cuda")
    before = host(D)                                            # 776 in bf16
    call = gpu_lib.mxfp8_moe_gemm if mx else gpu_lib.fp8_moe_gemm
    got = call(dev(A), dev(B), dev(sa), dev(sb), dev(start), rows=dev(index), bias=dev(b), act=act, gated=gated, D=D)
    assert got.data_ptr() == D.data_ptr()
    got = host(got)
    seen = np.zeros(S, bool)
    for e in range(E):
        a, z = start[e], start[e + 1]
        if z == a:
            continue
        seen[a:z] = True
        at = np.arange(a, z) if index is None else index[a:z]
        exact, tol = want(A[at], B[e], sa[at], sb[e], mx, None if b is None else b[e], act, gated, None)
        close(got[a:z], exact, rounded(exact, tol, dtype), "expert %d" % e)
    assert (got[~seen] == before[~seen]).all()


@pytest.mark.parametrize("S,E,n,k", [(1, 1, 16, 64), (6, 8, 40, 96), (48, 8, 128, 512), (200, 5, 72, 160), (333, 16, 48, 256),
                                     (900, 3, 136, 128), (1500, 4, 64, 384)])
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("how", ["even", "one", "gaps"])
def test_experts(gpu_lib, S, E, n, k, mx, gated, how):
    experts_case(gpu_lib, S, E, n, k, mx, gated, how, gather=gated or S % 2 == 0, dtype=BF if n % 16 else F, bias=how == "even")


@pytest.mark.parametrize("S,E,n,k", [(3000, 5, 264, 256), (2500, 2, 1000, 640), (700, 40, 33, 128)])
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("gather", [False, True])
def test_experts_large(gpu_lib, S, E, n, k, mx, gather):
    experts_case(gpu_lib, S, E, n, k, mx, not gather, "even", gather, BF, True)


@pytest.mark.parametrize("S,E,n,k", [(2000, 3, 264, 672), (1500, 2, 1001, 160), (600, 5, 130, 1056), (12, 4, 72, 1120)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_experts_tails(gpu_lib, S, E, n, k, gather, gated):
    experts_case(gpu_lib, S, E, n, k, True, gated, "gaps", gather, BF, True)


def test_experts_wrong_indices_stay_inside(gpu_lib):
    """Starts and rows outside the arrays: other rows come out right, and nothing outside is touched."""
    r = rng(5)
    S, E, n, k, Ra = 40, 4, 32, 128, 9
    A, sa = operand(r, Ra, k, False)
    B, sb = operand(r, E * n, k, False)
    index = r.integers(0, Ra, S).astype(np.int32)
    index[::7] = [-1, 1 << 30, -(1 << 31), Ra, 99, 1 << 20]
    start = np.array([-5, 10, 10, 30, 1 << 30], np.int32)
    D = gpu_lib.fp8_moe_gemm(dev(A), dev(B.reshape(E, n, k)), dev(sa), dev(sb.reshape(E, n)), dev(start), rows=dev(index))
    fine = (index >= 0) & (index < Ra)
    for e, (a, z) in enumerate(((0, 10), (10, 10), (10, 30), (30, 40))):
        at = np.arange(a, z)[fine[a:z]]
        if len(at):
            exact, tol = want(A[index[at]], B[e * n:e * n + n], sa[index[at]], sb[e * n:e * n + n], False, None, None, False, None)
            close(host(D)[at], exact, rounded(exact, tol, BF), "expert %d" % e)
