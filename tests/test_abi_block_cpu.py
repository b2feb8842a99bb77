"""The C ABI of the attention block's operators on the CPU: every declared
function is exported, and bad arguments are refused with the documented status
before any HIP call.  Pointers here are integers that are never dereferenced;
calls that would pass every check are not made."""

import ctypes
import re
import os

import numpy as np
import pytest
import torch

import fp8_scaled_gemm_amd as fp8g
from oracle import block

OK, NULL, SHAPE, ALIGN, DTYPE, OVERLAP, UNSUPPORTED = range(7)
GB = 1 << 30


def P(i, off=0):
    return ctypes.c_void_p(0x100000 + i * (64 * GB) + off)


@pytest.fixture(scope="module")
def lib():
    return fp8g.load()


def test_exports_every_header_function(lib):
    text = open(os.path.join(os.path.dirname(fp8g.HEADER_PATH), "fp8g_block.h")).read()
    names = re.findall(r"^(?:int|int64_t)\s+(\w+)\s*\(", text, flags=re.M)
    assert set(names) == {"lora_add", "lora_add_workspace", "qk_norm_rope", "kv4_append", "kv4_gather", "kv4_attention",
                          "kv4_attention_workspace"}
    for name in names:
        assert hasattr(lib, name)


def lora(lib, base=P(0), x=P(1), A=P(2), B=P(3), scale=P(4), start=P(5), adapter=P(6), tokens=8, n=64, k=64, rank=16,
         adapters=2, segments=3, dtype=0, out=P(7), ws=P(8), size=1 << 40):
    return lib.lora_add(base, x, A, B, scale, start, adapter, tokens, n, k, rank, adapters, segments, dtype, out, ws, size, None)


def test_lora_refusals(lib):
    for name in ("tokens", "n", "k", "rank", "adapters", "segments"):
        assert lora(lib, **{name: -1}) == SHAPE
    assert lora(lib, dtype=2) == DTYPE
    for bad in ({"rank": 12}, {"rank": 264}, {"k": 60}, {"tokens": 1 << 28}, {"n": 1 << 28}, {"k": 1 << 28},
                {"adapters": 1 << 28}, {"segments": (1 << 20) + 1}):
        assert lora(lib, **bad) == UNSUPPORTED
    assert lora(lib, tokens=0) == OK and lora(lib, n=0) == OK
    for name in ("base", "x", "A", "B", "scale", "start", "adapter", "out", "ws"):
        assert lora(lib, **{name: None}) == NULL
    for i, name in enumerate(("base", "x", "A", "B")):
        assert lora(lib, **{name: P(i, 8)}) == ALIGN
    assert lora(lib, out=P(7, 8)) == ALIGN and lora(lib, ws=P(8, 4)) == ALIGN and lora(lib, scale=P(4, 2)) == ALIGN
    for i in (1, 2, 3, 4, 5, 6):
        assert lora(lib, out=P(i)) == OVERLAP
    assert lora(lib, out=P(0, 16)) == OVERLAP          # part of base, not base itself
    assert lora(lib, ws=P(7)) == OVERLAP and lora(lib, ws=P(1)) == OVERLAP
    need = lib.lora_add_workspace(8, 64, 64, 16, 2, 3)
    assert need > 0 and lora(lib, size=need - 1) == UNSUPPORTED
    assert lib.lora_add_workspace(8, 64, 64, 12, 2, 3) == -1
    assert lib.lora_add_workspace(0, 64, 64, 16, 2, 3) == 0


def qk(lib, q=P(0), qs=512, k=P(1), ks=256, dtype=0, tokens=4, hq=4, hk=2, dim=128, wq=P(2), wk=P(3), positions=P(4),
       axes=1, axis=None, table=P(5), P_max=100, rotary=128, qo=P(6), qos=512, ko=P(7), kos=256):
    return lib.qk_norm_rope(q, qs, k, ks, dtype, tokens, hq, hk, dim, wq, wk, 1e-6, positions, axes, axis, table, P_max,
                            rotary, 0, qo, qos, ko, kos, None)


def test_qk_refusals(lib):
    for bad in ({"tokens": -1}, {"hq": -1}, {"hk": -1}, {"dim": -8}, {"rotary": 144}, {"rotary": 0}, {"axes": 0},
                {"P_max": 0}, {"qs": 511}, {"kos": 248}, {"axes": 2}):
        assert qk(lib, **bad) == SHAPE, bad
    assert qk(lib, dtype=3) == DTYPE
    for bad in ({"dim": 132, "qs": 1 << 20, "ks": 1 << 20, "qos": 1 << 20, "kos": 1 << 20},
                {"dim": 264, "qs": 1 << 20, "ks": 1 << 20, "qos": 1 << 20, "kos": 1 << 20}, {"rotary": 24},
                {"qs": 516}, {"kos": 260}, {"tokens": 1 << 31}, {"tokens": 1 << 29}):
        assert qk(lib, **bad) == UNSUPPORTED, bad
    assert qk(lib, tokens=0) == OK and qk(lib, hq=0, hk=0) == OK
    for name in ("q", "k", "positions", "table", "qo", "ko"):
        assert qk(lib, **{name: None}) == NULL
    assert qk(lib, q=P(0, 8)) == ALIGN and qk(lib, ko=P(7, 2)) == ALIGN and qk(lib, wq=P(2, 2)) == ALIGN
    assert qk(lib, qo=P(0, 16)) == OVERLAP and qk(lib, qo=P(1)) == OVERLAP and qk(lib, ko=P(6)) == OVERLAP
    assert qk(lib, qo=P(4)) == OVERLAP and qk(lib, ko=P(5)) == OVERLAP
    # in place but with another stride
    assert qk(lib, qo=P(0), qos=520) == OVERLAP
    # q and k side by side in rows of 1024: in place overlaps nothing, shifted by 8 heads it does
    assert qk(lib, q=P(0), qs=1024, k=P(0, 512), ks=1024, qo=P(0), qos=1024, ko=P(0, 512), kos=1024) == OVERLAP


def rows(lib, k=P(0), ks=256, v=P(1), vs=256, dtype=1, tokens=4, heads=2, dk=128, dv=128, slots=P(2), pages=5, page=16,
         kc=P(3), ksc=P(4), vc=P(5), vsc=P(6)):
    return lib.kv4_append(k, ks, v, vs, dtype, tokens, heads, dk, dv, slots, pages, page, kc, ksc, vc, vsc, None)


def gather(lib, ko=P(0), vo=P(1), dtype=0, tokens=4, heads=2, dk=128, dv=128, slots=P(2), pages=5, page=16, kc=P(3),
           ksc=P(4), vc=P(5), vsc=P(6)):
    return lib.kv4_gather(kc, ksc, vc, vsc, pages, page, heads, dk, dv, slots, tokens, dtype, ko, vo, None)


def test_cache_refusals(lib):
    for call in (rows, gather):
        for bad in ({"tokens": -1}, {"heads": -1}, {"pages": -1}, {"page": 0}):
            assert call(lib, **bad) == SHAPE
        assert call(lib, dtype=2) == DTYPE
        for bad in ({"dk": 96}, {"dv": 64}, {"page": 24}, {"heads": 65537}, {"tokens": 1 << 31}):
            assert call(lib, **bad) == UNSUPPORTED
        assert call(lib, tokens=0) == OK and call(lib, heads=0) == OK
        for name in ("slots", "kc", "ksc", "vc", "vsc"):
            assert call(lib, **{name: None}) == NULL
        assert call(lib, kc=P(3, 8)) == ALIGN and call(lib, vsc=P(6, 4)) == ALIGN and call(lib, slots=P(2, 4)) == ALIGN
    assert rows(lib, ks=255) == SHAPE and rows(lib, ks=260) == UNSUPPORTED
    assert rows(lib, k=None) == NULL and rows(lib, v=P(1, 4)) == ALIGN
    assert rows(lib, kc=P(0)) == OVERLAP and rows(lib, vc=P(3)) == OVERLAP and rows(lib, ksc=P(2)) == OVERLAP
    assert gather(lib, ko=None) == NULL and gather(lib, vo=P(1, 4)) == ALIGN
    assert gather(lib, ko=P(1)) == OVERLAP and gather(lib, vo=P(5)) == OVERLAP


def attn(lib, q=P(0), qs=1024, queries=4, hq=8, kc=P(1), ksc=P(2), vc=P(3), vsc=P(4), pages=9, page=16, hk=2, dk=128,
         dv=128, table=P(5), batch=3, most=40, start=P(6), length=P(7), causal=1, window=0, out=P(8), lse=P(9), ws=P(10),
         size=1 << 40):
    return lib.kv4_attention(q, qs, queries, hq, kc, ksc, vc, vsc, pages, page, hk, dk, dv, table, batch, most, start,
                             length, 0.1, causal, window, out, lse, ws, size, None)


def test_attention_refusals(lib):
    for bad in ({"queries": -1}, {"hq": -8}, {"hk": -1}, {"pages": -1}, {"page": 0}, {"batch": -1}, {"most": -1},
                {"window": -1}, {"window": 5, "causal": 0}, {"qs": 1023}, {"hk": 0}):
        assert attn(lib, **bad) == SHAPE, bad
    for bad in ({"dk": 80}, {"dv": 64}, {"page": 8}, {"hk": 3}, {"most": 1 << 27}, {"qs": 1028}, {"queries": 1 << 28},
                {"batch": (1 << 20) + 1}):
        assert attn(lib, **bad) == UNSUPPORTED, bad
    assert attn(lib, queries=0) == OK and attn(lib, batch=0) == OK and attn(lib, hq=0) == OK
    for name in ("q", "kc", "ksc", "vc", "vsc", "table", "start", "length", "out", "ws"):
        assert attn(lib, **{name: None}) == NULL, name
    for i, name in ((0, "q"), (1, "kc"), (4, "vsc"), (8, "out"), (10, "ws")):
        assert attn(lib, **{name: P(i, 8)}) == ALIGN
    assert attn(lib, table=P(5, 2)) == ALIGN and attn(lib, lse=P(9, 2)) == ALIGN
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 9, 10):
        assert attn(lib, out=P(i)) == OVERLAP
    assert attn(lib, lse=P(0)) == OVERLAP and attn(lib, ws=P(1)) == OVERLAP
    need = lib.kv4_attention_workspace(4, 8, 2, 128, 128, 3, 40, 16, 0)
    assert need > 0 and attn(lib, size=need - 1) == UNSUPPORTED
    assert lib.kv4_attention_workspace(4, 8, 3, 128, 128, 3, 40, 16, 0) == -1


def test_python_refuses_host_tensors():
    x = torch.zeros(4, 32)
    if not torch.cuda.is_available():
        pytest.skip("current_device needs a device")
    with pytest.raises(ValueError):
        fp8g.lora_add(x, x.bfloat16(), x.view(1, 4, 32).bfloat16(), x.view(1, 32, 4).bfloat16(), x[0, :1], x, x)


# ------------------------------------------------------------------ the oracle

def test_mxfp4_quantizer_by_search():
    """Codes and scales against a search over all codes and exponents."""
    r = np.random.default_rng(3)
    x = (r.standard_normal((40, 32)) * np.exp(4 * r.standard_normal((40, 1)))).astype(np.float32).astype(np.float64)
    x[0], x[1, 5:] = 0.0, 0.0
    x[2, :8] = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    x[2, 8:] = 0.3
    codes, scales = block.mxfp4_quantize(x)
    grid = np.concatenate([block.E2M1, -block.E2M1])
    for row in range(len(x)):
        amax = np.abs(x[row]).max()
        fit = [e for e in range(-127, 128) if amax <= 6.0 * 2.0 ** e]
        assert scales[row, 0] == fit[0] + 127
        y = x[row] / 2.0 ** fit[0]
        assert np.abs(np.abs(grid[codes[row]]) - np.abs(y)).max() <= 1.0
        best = np.abs(grid[None] - y[:, None]).min(1)
        assert np.array_equal(np.abs(grid[codes[row]] - y), best)
        assert np.array_equal(codes[row] >= 8, np.signbit(x[row]))
    assert np.array_equal(codes[2, :8], [0, 2, 2, 4, 4, 6, 6, 7])
    assert np.array_equal(block.unpack(block.pack(codes)), codes)


def test_attention_oracle_by_hand():
    q = np.array([[[1.0] + [0.0] * 63]])
    k = [np.zeros((2, 1, 64))]
    k[0][0, 0, 0], k[0][1, 0, 0] = np.log(3.0), 0.0
    v = [np.array([[[4.0] * 64], [[8.0] * 64]])]
    out, lse, weight, _ = block.attention(q, k, v, [0, 1], [2], 1.0, True, 0)
    assert np.allclose(out, 5.0) and np.allclose(lse, np.log(4.0)) and np.allclose(weight, 5.0)
    out, lse, _, _ = block.attention(q, k, v, [0, 1], [2], 1.0, True, 1)
    assert np.allclose(out, 8.0) and np.allclose(lse, 0.0)
    out, lse, _, _ = block.attention(q, [k[0][:0]], [v[0][:0]], [0, 1], [0], 1.0, True, 0)
    assert (out == 0).all() and (lse == -np.inf).all()
