"""The C ABI of the feed-forward half's operators on the CPU: every declared
function is exported, and bad arguments are refused with the documented status
before any HIP call.  Pointers here are integers that are never dereferenced;
calls that would pass every check are not made."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as fp8g
from oracle import ffn

OK, NULL, SHAPE, ALIGN, DTYPE, OVERLAP, UNSUPPORTED = range(7)
GB = 1 << 30


def P(i, off=0):
    return ctypes.c_void_p(0x100000 + i * (64 * GB) + off)


@pytest.fixture(scope="module")
def lib():
    return fp8g.load()


def test_exports_every_header_function(lib):
    text = open(os.path.join(os.path.dirname(fp8g.HEADER_PATH), "fp8g_ffn.h")).read()
    names = re.findall(r"^(?:int|int64_t)\s+(\w+)\s*\(", text, flags=re.M)
    assert set(names) == {"add_rms_norm_quantize", "fp8_gemm_fused", "mxfp8_gemm_fused", "gemm_fused_workspace", "moe_route", "moe_route_workspace",
                          "fp8_moe_gemm", "mxfp8_moe_gemm", "moe_gemm_workspace", "moe_combine"}
    for name in names:
        assert hasattr(lib, name)


def norm(lib, x=P(0), xs=256, res=P(1), rs=256, dtype=1, rows=4, cols=256, w=P(2), gran=0, fmt=0, total=P(3), norm=P(4),
         q=P(5), scale=P(6)):
    return lib.add_rms_norm_quantize(x, xs, res, rs, dtype, rows, cols, w, 1e-6, gran, fmt, total, norm, q, scale, None)


def test_norm_refusals(lib):
    for bad in ({"rows": -1}, {"cols": -16}, {"xs": 255}, {"rs": 248}, {"gran": 2, "cols": 240}):
        assert norm(lib, **bad) == SHAPE, bad
    for bad in ({"dtype": 2}, {"gran": 1}, {"gran": 3}, {"fmt": 2}, {"gran": 2, "fmt": 1}):
        assert norm(lib, **bad) == DTYPE, bad
    for bad in ({"cols": 248}, {"xs": 260}, {"rs": 257}, {"rows": 1 << 24}, {"cols": 1 << 28, "xs": 1 << 28, "rs": 1 << 28}):
        assert norm(lib, **bad) == UNSUPPORTED, bad
    assert norm(lib, rows=0) == OK and norm(lib, cols=0) == OK
    for name in ("x", "q", "scale"):
        assert norm(lib, **{name: None}) == NULL
    for i, name in enumerate(("x", "res", "w", "total", "norm", "q", "scale")):
        assert norm(lib, **{name: P(i, 2)}) == ALIGN, name
    assert norm(lib, total=P(0), xs=512) == OVERLAP                # in place, but not dense
    assert norm(lib, total=P(0, 16)) == OVERLAP and norm(lib, total=P(1, 16)) == OVERLAP
    for name in ("norm", "q", "scale"):
        for i in (0, 1, 2, 3):
            assert norm(lib, **{name: P(i)}) == OVERLAP, (name, i)
    assert norm(lib, q=P(4)) == OVERLAP and norm(lib, scale=P(5)) == OVERLAP and norm(lib, total=P(2)) == OVERLAP


def gemm(lib, mx=False, m=4, n=64, k=256, A=P(0), B=P(1), sa=P(2), sb=P(3), bias=P(4), act=1, gated=1, res=P(5), D=P(6), out=0,
         ws=P(9), size=1 << 40):
    call = lib.mxfp8_gemm_fused if mx else lib.fp8_gemm_fused
    return call(m, n, k, A, B, sa, sb, bias, act, gated, res, D, out, ws, size, None)


def moe(lib, mx=False, S=8, n=64, k=256, E=4, A=P(0), Ra=5, rows=P(7), start=P(8), B=P(1), sa=P(2), sb=P(3), bias=P(4), act=1,
        gated=1, D=P(6), out=0, ws=P(9), size=1 << 40):
    call = lib.mxfp8_moe_gemm if mx else lib.fp8_moe_gemm
    return call(S, n, k, E, A, Ra, rows, start, B, sa, sb, bias, act, gated, D, out, ws, size, None)


@pytest.mark.parametrize("mx", [False, True])
def test_product_refusals(lib, mx):
    for call, rows in ((gemm, "m"), (moe, "S")):
        for name in (rows, "n", "k"):
            assert call(lib, mx, **{name: -1}) == SHAPE
        assert call(lib, mx, out=2) == DTYPE and call(lib, mx, act=3) == DTYPE and call(lib, mx, act=-1) == DTYPE
        assert call(lib, mx, k=1 << 23) == UNSUPPORTED and call(lib, mx, n=1 << 21) == UNSUPPORTED
        assert call(lib, mx, n=1 << 20, out=1) == UNSUPPORTED and call(lib, mx, n=1 << 22, gated=0) == UNSUPPORTED
        assert call(lib, mx, **{rows: 1 << 31}) == UNSUPPORTED
        assert call(lib, mx, **{rows: 0, **({"Ra": 0} if call is moe else {})}) == OK and call(lib, mx, n=0) == OK
        for name in ("A", "B", "sa", "sb", "D"):
            assert call(lib, mx, **{name: None}) == NULL, name
        for i, name in ((0, "A"), (1, "B"), (2, "sa"), (3, "sb"), (6, "D")):
            assert call(lib, mx, **{name: P(i, 8)}) == ALIGN, name
        assert call(lib, mx, bias=P(4, 2)) == ALIGN
        for i in (0, 1, 2, 3, 4):
            assert call(lib, mx, D=P(i)) == OVERLAP, i
    assert gemm(lib, mx, k=264) == (SHAPE if mx else UNSUPPORTED) and moe(lib, mx, k=264) == (SHAPE if mx else UNSUPPORTED)
    assert gemm(lib, mx, res=P(5, 4)) == ALIGN and gemm(lib, mx, D=P(5, 16)) == OVERLAP
    need = lib.gemm_fused_workspace(256, 1024, 8192, 1, mx)          # few tiles, a long K: split
    split = {"m": 256, "n": 1024, "k": 8192}
    assert need > 0 and gemm(lib, mx, size=need - 1, **split) == UNSUPPORTED and gemm(lib, mx, ws=None, **split) == NULL
    for i in (0, 1, 2, 3, 4, 5, 6):
        assert gemm(lib, mx, ws=P(i), **split) == OVERLAP
    assert lib.gemm_fused_workspace(64, 1024, 8200, 1, mx) == -1 and lib.gemm_fused_workspace(0, 1024, 8192, 1, mx) == 0
    assert moe(lib, mx, E=-1) == SHAPE and moe(lib, mx, Ra=-1) == SHAPE and moe(lib, mx, Ra=0) == SHAPE
    assert moe(lib, mx, rows=None) == SHAPE                        # 5 rows of A for 8 slots
    assert moe(lib, mx, E=1025) == UNSUPPORTED and moe(lib, mx, S=1 << 28) == UNSUPPORTED
    assert moe(lib, mx, Ra=(1 << 31) // 256) == UNSUPPORTED        # offsets of gathered rows
    assert moe(lib, mx, E=0) == OK and moe(lib, mx, start=None) == NULL
    assert moe(lib, mx, rows=P(7, 2)) == ALIGN and moe(lib, mx, start=P(8, 1)) == ALIGN and moe(lib, mx, ws=P(9, 8)) == ALIGN
    assert moe(lib, mx, D=P(7)) == OVERLAP and moe(lib, mx, D=P(8)) == OVERLAP
    for S, n, k, E, gathered in ((8, 64, 256, 4, 1), (70000, 4096, 4096, 128, 1), (70000, 4096, 4096, 128, 0)):
        need = lib.moe_gemm_workspace(S, n, k, E, gathered, 1, mx)
        assert need >= 0
        if need:
            more = {"Ra": 5 if gathered else S, "rows": P(7) if gathered else None, "S": S, "n": n, "k": k, "E": E}
            assert moe(lib, mx, size=need - 1, **more) == UNSUPPORTED and moe(lib, mx, ws=None, **more) == NULL
            assert moe(lib, mx, ws=P(6), **more) == OVERLAP and moe(lib, mx, ws=P(1), **more) == OVERLAP
    assert lib.moe_gemm_workspace(8, 64, 250, 4, 1, 0, mx) == -1 and lib.moe_gemm_workspace(8, 64, 256, 1025, 1, 0, mx) == -1
    assert lib.moe_gemm_workspace(0, 64, 256, 4, 1, 0, mx) == 0


def route(lib, x=P(0), dtype=0, T=70, E=64, k=4, bias=P(1), score=0, groups=8, top=3, each=2, ids=P(2), w=P(3), start=P(4),
          rows=P(5), slots=P(6), ws=P(7), size=1 << 40):
    return lib.moe_route(x, dtype, T, E, k, bias, score, groups, top, each, 1, 1.0, ids, w, start, rows, slots, ws, size, None)


def test_route_refusals(lib):
    for bad in ({"T": -1}, {"E": 0}, {"k": 0}, {"k": 65}, {"groups": 0}, {"groups": 7}, {"top": 0}, {"top": 9}, {"each": 0},
                {"each": 3}, {"groups": 64, "each": 2}):
        assert route(lib, **bad) == SHAPE, bad
    assert route(lib, dtype=2) == DTYPE and route(lib, score=2) == DTYPE and route(lib, score=-1) == DTYPE
    for bad in ({"E": 1032}, {"k": 33}, {"groups": 128, "E": 256}, {"T": 1 << 26}, {"T": 1 << 28}):
        assert route(lib, **bad) == UNSUPPORTED, bad
    for name in ("x", "ids", "w", "start", "rows", "slots", "ws"):
        assert route(lib, **{name: None}) == NULL, name
    for i, name in enumerate(("x", "bias", "ids", "w", "start", "rows", "slots", "ws")):
        assert route(lib, **{name: P(i, 2)}) == ALIGN, name
    for i, name in ((2, "ids"), (3, "w"), (4, "start"), (5, "rows"), (6, "slots"), (7, "ws")):
        for j in range(8):
            if i != j:
                assert route(lib, **{name: P(j)}) == OVERLAP, (name, j)
    need = lib.moe_route_workspace(70, 64, 4)
    assert need > 0 and route(lib, size=need - 1) == UNSUPPORTED
    assert lib.moe_route_workspace(24, 64, 4) == 0                  # one workgroup does it all
    assert lib.moe_route_workspace(7, 64, 65) == -1 and lib.moe_route_workspace(7, 1025, 2) == -1


def combine(lib, y=P(0), S=20, slots=P(1), w=P(2), res=P(3), dtype=0, T=4, k=2, H=64, out=P(4)):
    return lib.moe_combine(y, S, slots, w, res, dtype, T, k, H, out, None)


def test_combine_refusals(lib):
    for name in ("S", "T", "k", "H"):
        assert combine(lib, **{name: -1}) == SHAPE
    assert combine(lib, dtype=2) == DTYPE
    for bad in ({"H": 60}, {"H": 2, "dtype": 1}, {"H": 1 << 28}, {"T": 1 << 28}, {"k": 1 << 28}, {"S": 1 << 28},
                {"T": (1 << 28) - 1, "H": 1 << 16}):
        assert combine(lib, **bad) == UNSUPPORTED, bad
    assert combine(lib, T=0) == OK and combine(lib, H=0) == OK
    for name in ("y", "slots", "w", "out"):
        assert combine(lib, **{name: None}) == NULL
    for i, name in enumerate(("y", "slots", "w", "res", "out")):
        assert combine(lib, **{name: P(i, 2)}) == ALIGN
    for i in (0, 1, 2):
        assert combine(lib, out=P(i)) == OVERLAP
    assert combine(lib, out=P(3, 16)) == OVERLAP


def test_python_refuses_unknown_choices():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="act must be"):
        fp8g.fp8_gemm_fused(4, 4, 64, x, x, x, x, act="tanh")
    with pytest.raises(ValueError, match="act must be"):
        fp8g.mxfp8_moe_gemm(x, x, x, x, x, act=["silu"])
    with pytest.raises(ValueError, match="score must be"):
        fp8g.moe_route(x, 2, score="linear")
    with pytest.raises(TypeError, match="out_dtype"):
        fp8g.fp8_gemm_fused(4, 4, 64, x, x, x, x, out_dtype=torch.float16)
    assert fp8g.moe_route_workspace(0, 8, 2) >= 0
    with pytest.raises(fp8g.Fp8gError):
        fp8g.moe_route_workspace(4, 8, 9)
    with pytest.raises(fp8g.Fp8gError):
        fp8g.moe_gemm_workspace(4, 8, 100, 2, mx=True)


# ------------------------------------------------------------------ the oracle

def test_route_oracle_by_hand():
    x = np.array([[1.0, 3.0, 2.0, 3.0], [-np.inf, 0.0, -np.inf, -np.inf], [-np.inf] * 4])
    ids, w, start, rows, slots = ffn.route(x, 2, renormalize=False)
    e = np.exp(x[0] - 3.0)
    assert ids.tolist() == [[1, 3], [1, -1], [-1, -1]]
    assert np.allclose(w, [[1 / e.sum(), 1 / e.sum()], [1.0, 0.0], [0.0, 0.0]])
    assert start.tolist() == [0, 0, 2, 2, 3] and rows.tolist() == [0, 1, 0, -1, -1, -1]
    assert slots.tolist() == [[0, 2], [1, -1], [-1, -1]]
    # groups {0, 1}, {2, 3}: sums of two sigmoids; the bias turns the choice, not the weight
    ids, w, *_ = ffn.route(np.array([[4.0, -9.0, 1.0, 0.5]]), 1, score="sigmoid", groups=2, top_groups=1, scale=3.0)
    assert ids.tolist() == [[2]] and np.allclose(w, 3.0)
    ids, w, *_ = ffn.route(np.array([[4.0, -9.0, 1.0, 0.5]]), 1, bias=[0.0, 2.0, 0.0, 0.0], score="sigmoid", groups=2,
                           top_groups=1, renormalize=False)
    assert ids.tolist() == [[1]] and np.allclose(w, 1 / (1 + np.exp(9.0)))


def test_fused_oracle_by_hand():
    one = np.full((1, 32), 0x38, np.uint8)                         # 1.0
    B = np.concatenate([one, one + 8])                              # rows of 1.0 and of 2.0
    T = np.zeros((1, 2))
    v, tol = ffn.fused(one, B, [0.5], [1.0, 0.25], False, [1.0, -2.0], "silu", True, [[3.0]], T)
    g, u = 16.0 + 1.0, 8.0 - 2.0
    assert np.allclose(v, g / (1 + np.exp(-g)) * u + 3.0) and (tol > 0).all()
    v, _ = ffn.fused(one, B, [[127]], [[128], [126]], True, None, "none", False, None, T)
    assert np.allclose(v, [[64.0, 32.0]])
    x = np.linspace(-6, 6, 101)
    v, _ = ffn.activate(x, "gelu_tanh")
    assert np.allclose(v, 0.5 * x * (1 + np.tanh(np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3))))
    assert np.abs(np.diff(v) / np.diff(x)).max() < ffn.SLOPE
    assert np.allclose(ffn.rms_norm([[3.0, 4.0]], [1.0, 2.0], 0.0), [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    out, size = ffn.combine([[1.0, 2.0], [3.0, -4.0]], np.array([[1, -1], [0, 5]]), np.array([[0.5, 9.0], [2.0, 9.0]]), None)
    assert out.tolist() == [[1.5, -2.0], [2.0, 4.0]] and size.tolist() == [[1.5, 2.0], [2.0, 4.0]]
