"""add_rms_norm_quantize and moe_combine against the float64 definitions."""

import numpy as np
import pytest
import torch

from block_util import bf16, close, f32, half_ulp, host, rng, typed
from ffn_util import dev
from gpu_util import say
from oracle import e4m3, e5m2, ffn

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def stream(r, rows, cols, dtype):
    x = r.standard_normal((rows, cols)) * np.exp(2 * r.standard_normal((rows, 1))) * np.exp(0.7 * r.standard_normal((1, cols)))
    if rows > 2:
        x[0] = 0.0
        x[1, ::2] = -0.0
        x[2] *= 2.0 ** -60
    if rows > 4:
        x[3] *= 2.0 ** 90                                       # its squares pass fp32's range
        x[4, 1:] = 0.0
    return typed(x, dtype)


WHAT64 = 2.0 ** -46        # fp64's own error, of the kernel (2^-48) and of numpy's sums


def nearest(x, fmt):
    """x to FP8's values, ties to even, and how far x is from the nearest tie, relative to x."""
    bits, low, most = (3, -6, 448.0) if fmt == 0 else (2, -14, 57344.0)
    size = np.abs(x)
    e = np.maximum(np.floor(np.log2(np.maximum(size, 2.0 ** -200))), low)
    step = 2.0 ** (e - bits)
    place = size / step
    tie = np.abs(place - np.floor(place) - 0.5) * step
    return np.sign(x) * np.minimum(np.round(place) * step, most), tie / np.maximum(size, 2.0 ** -200)


def check_codes(y, q, scale, mx, fmt):
    """q and scale against the exact y: equal but for ties and borders that fp64 cannot tell."""
    value = (e4m3 if fmt == 0 else e5m2).decode(q)
    most = 448.0 if fmt == 0 else 57344.0
    if mx:
        amax = np.abs(y.reshape(len(y), -1, 32)).max(2)
        e = np.clip(np.ceil(np.log2(np.maximum(amax, 2.0 ** -300) / most)), -127, 127)
        e = np.where((e > -127) & (amax <= most * 2.0 ** (e - 1)), e - 1, e)             # log2's own rounding
        e = np.where(amax > most * 2.0 ** e, np.minimum(e + 1, 127), e)
        border = np.abs(amax / (most * 2.0 ** np.round(np.log2(np.maximum(amax, 2.0 ** -300) / most))) - 1) < WHAT64
        assert (border | (scale.astype(int) - 127 == e)).all()
        exact = y / (2.0 ** (scale.astype(np.float64) - 127)).repeat(32, 1)
    else:
        amax = np.abs(y).max(1)
        close(scale.astype(np.float64), amax / most, (2.0 ** -24 + WHAT64) * amax / most + 2.0 ** -150, "scale")
        s = scale.astype(np.float64)
        by = np.where(s > 0, most / np.where(amax > 0, amax, 1.0), 0.0)
        exact = y * by[:, None]
    want, tie = nearest(exact, fmt)
    assert ((value == want) | (tie < WHAT64)).all()
    assert np.array_equal(np.signbit(value), np.signbit(y))                              # of zeros too


@pytest.mark.parametrize("rows,cols", [(1, 32), (7, 512), (33, 2048), (5, 2080), (300, 4096), (9, 8160), (3, 16384),
                                       (2, 16416), (4, 40000)])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("mode", ["row", "row_e5m2", "mx"])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(gpu_lib, rows, cols, dtype, mode, residual):
    r = rng(rows, cols, residual)
    mx, fmt = mode == "mx", 1 if mode == "row_e5m2" else 0
    x64, x = stream(r, rows, cols, dtype)
    r64, res = stream(r, rows, cols, dtype)
    w64, w = f32(1 + 0.3 * r.standard_normal(cols))
    say("norm", rows, cols, dtype, mode, residual)
    got = gpu_lib.add_rms_norm_quantize(x.cuda(), w.cuda(), residual=res.cuda() if residual else None, eps=1e-6, mx=mx, fmt=fmt,
                                        return_norm=True)
    s64 = x64
    if residual:
        s64, s = typed(x64.astype(np.float32) + r64.astype(np.float32), dtype)
        assert torch.equal(got.sum.cpu(), s)
    else:
        assert got.sum is None
    y = ffn.rms_norm(s64, w64, float(np.float32(1e-6)))
    # fp64, rounded to fp32 and then to the type
    close(host(got.norm), y, (half_ulp(dtype) + 2.0 ** -24) * (1 + 2.0 ** -20) * np.abs(y) + 2.0 ** -149, "norm")
    q, scale = got.q.view(torch.uint8).cpu().numpy(), got.scale.cpu().numpy()
    check_codes(y, q, scale, mx, fmt)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("cols", [512, 4096, 17408])
def test_norm_in_place_strided_without_weight(gpu_lib, dtype, cols):
    r = rng(cols, 3)
    x64, x = stream(r, 6, cols, dtype)
    r64, res = stream(r, 6, cols, dtype)
    wide = torch.full((6, 3 * cols), 7.0, dtype=dtype)
    wide[:, cols:2 * cols] = x
    wide = wide.cuda()
    plain = gpu_lib.add_rms_norm_quantize(x.cuda(), residual=res.cuda())
    here = res.cuda()
    got = gpu_lib.add_rms_norm_quantize(wide[:, cols:2 * cols], residual=here, sum=here)
    assert got.sum.data_ptr() == here.data_ptr()
    for a, b in zip(plain[:3], got[:3]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert (wide[:, :cols] == 7.0).all() and (wide[:, 2 * cols:] == 7.0).all()
    close(host(got.scale), np.abs(ffn.rms_norm(host(got.sum), None, float(np.float32(1e-6)))).max(1) / 448,
          (2.0 ** -24 + WHAT64) * host(got.scale) + 2.0 ** -149, "scale")


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("cols", [1024, 20000])
def test_norm_rows_with_nan_and_infinity(gpu_lib, mx, cols):
    cols -= cols % 32
    r = rng(cols, mx)
    _, x = f32(r.standard_normal((6, cols)))
    clean = x.clone()
    x[1, 5], x[3, cols - 1], x[4, 7] = float("nan"), float("inf"), -float("inf")
    got = gpu_lib.add_rms_norm_quantize(x.cuda(), mx=mx, return_norm=True)
    same = gpu_lib.add_rms_norm_quantize(clean.cuda(), mx=mx, return_norm=True)
    for t in (1, 3, 4):
        assert (got.q[t].view(torch.uint8) == 0).all() and torch.isnan(got.norm[t]).all()
        assert (got.scale[t] == 255).all() if mx else torch.isnan(got.scale[t])
    for t in (0, 2, 5):
        assert torch.equal(got.q[t].view(torch.uint8), same.q[t].view(torch.uint8))
        assert torch.equal(got.scale[t], same.scale[t]) and torch.equal(got.norm[t], same.norm[t])


@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (1, 8, 4096), (37, 6, 520), (300, 2, 1024), (5, 9, 16392), (3, 0, 64)])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("residual", [False, True])
def test_combine(gpu_lib, T, k, H, dtype, residual):
    r = rng(T, k, H)
    S = T * k + 3
    y64, y = typed(r.standard_normal((S, H)), dtype)
    slots = r.permutation(S)[:T * k].reshape(T, k).astype(np.int32)
    slots[r.random((T, k)) < 0.15] = -1
    if slots.size:
        slots[0, 0], slots[-1, -1] = S, -(1 << 31)              # outside: nothing
    w64, w = f32(r.random((T, k)))
    res64, res = typed(r.standard_normal((T, H)), dtype)
    say("combine", T, k, H, dtype, residual)
    out, size = ffn.combine(y64, slots, w64, res64 if residual else None)
    got = gpu_lib.moe_combine(y.cuda(), dev(slots), w.cuda(), residual=res.cuda() if residual else None)
    bound = (k + 1) * 2.0 ** -24 * size + half_ulp(dtype) * (np.abs(out) + (k + 1) * 2.0 ** -24 * size)
    close(host(got), out, bound, "combine")
    if residual:
        here = res.cuda()
        assert torch.equal(gpu_lib.moe_combine(y.cuda(), dev(slots), w.cuda(), residual=here, out=here), got)
