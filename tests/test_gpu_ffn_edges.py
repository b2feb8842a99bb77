"""The feed-forward half's products and norm at the borders of what they take."""

import numpy as np
import pytest
import torch

from block_util import close, host, rng
from ffn_util import dev, operand
from gpu_util import say
from oracle import ffn
from test_gpu_ffn_gemm import case
from test_gpu_ffn_limits import guarded, same_but_for_a_step

pytestmark = pytest.mark.gpu


INF = float("inf")


# the row kernel, small and large tiles, and K ranges
@pytest.mark.parametrize("m,k", [(1, 0), (1, 64), (100, 64), (100, 4096), (600, 128), (3000, 128), (3000, 160)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("mx", [False, True])
def test_activations_of_infinities(gpu_lib, m, k, act, mx):
    """z = bias alone (codes of zero): act(+inf) = +inf, NaN stays, and the largest finite values are themselves."""
    z = torch.tensor([INF, -INF, float("nan"), 3.4028234e38, -3.4028234e38, 2.0 ** 64, 0.0, -INF], device="cuda")
    n = 2200 if k == 128 else 264
    bias = z.repeat(n // 8)
    call = gpu_lib.mxfp8_gemm_fused if mx else gpu_lib.fp8_gemm_fused
    A, B = (torch.zeros(i, k, dtype=torch.uint8, device="cuda") for i in (m, 2 * n))
    sa, sb = (torch.full((i, k // 32), 127, dtype=torch.uint8, device="cuda") if mx else torch.ones(i, device="cuda") for i in (m, 2 * n))
    say("infinities", m, k, act, mx)
    want = torch.tensor([INF, float("nan"), float("nan"), 3.4028234e38, -0.0, 2.0 ** 64, 0.0, float("nan")], device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        got = call(m, n, k, A, B[:n], sa, sb[:n], bias=bias, act=act, out_dtype=dtype)
        torch.testing.assert_close(got, want.to(dtype).repeat(m, n // 8), rtol=0, atol=0, equal_nan=True)
        # gated: act(z) times an up projection of 0.5
        got = call(m, n, k, A, B, sa, sb, bias=torch.cat([bias, torch.full((n,), 0.5, device="cuda")]), act=act, gated=True,
                   out_dtype=dtype)
        torch.testing.assert_close(got, (0.5 * want).to(dtype).repeat(m, n // 8), rtol=0, atol=0, equal_nan=True)
    if m > 1 and k < 4096:
        start = torch.tensor([0, m // 2, m], dtype=torch.int32, device="cuda")
        many = (lambda t: torch.stack([t[:n], t[:n]]))                     # noqa: E731
        moe = gpu_lib.mxfp8_moe_gemm if mx else gpu_lib.fp8_moe_gemm
        got = moe(A, many(B), sa, many(sb), start, bias=torch.stack([bias, bias]), act=act)
        torch.testing.assert_close(got, want.to(torch.bfloat16).repeat(m, n // 8), rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_activations_of_every_size(gpu_lib, act):
    """Powers of two and their neighbours of both signs, over fp32's range."""
    z = 2.0 ** np.arange(-126, 128)
    z = np.concatenate([z, 1.5 * z, z * (1 + 2.0 ** -23), z * (2 - 2.0 ** -23)]).astype(np.float32)
    z = np.concatenate([z, -z])
    n = len(z)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    got = gpu_lib.fp8_gemm_fused(1, n, 0, none.view(1, 0), none.view(n, 0), dev(np.ones(1, np.float32)), dev(np.ones(n, np.float32)),
                                 bias=dev(z), act=act, out_dtype=torch.float32)
    z = z.astype(np.float64)
    v, own = ffn.activate(z, act)
    # where 1 + exp(-p) passes 2^126 the result may be 0, and below the smallest normal the rounding is absolute
    close(host(got)[0], v, own + 2.0 ** -24 * np.abs(v) + 2.0 ** -126 * np.maximum(1, np.where(z < -8, -z, 0)), act)


@pytest.mark.parametrize("starts", ["0 S 0 S", "one step back", "falling"])
@pytest.mark.parametrize("S,E,n,k", [(3000, 64, 136, 256), (500, 40, 72, 160), (2000, 1024, 40, 32)])
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("gathered", [False, True])
def test_starts_that_are_not_ascending_stay_inside(gpu_lib, starts, S, E, n, k, mx, gathered):
    """Experts that claim the same slots: more tile rows than slots, of which the plan takes what it has room for."""
    r = rng(S, E, mx, gathered)
    Ra = 200 if gathered else S
    A, sa = operand(r, Ra, k, mx)
    B, sb = operand(r, E * n, k, mx)
    B, sb = dev(B.reshape(E, n, k)), dev(sb.reshape(E, n, k // 32) if mx else sb.reshape(E, n))
    start = np.sort(r.integers(0, S + 1, E + 1)).astype(np.int32)
    if starts == "0 S 0 S":
        start[0::2], start[1::2] = 0, S
    elif starts == "falling":
        start = start[::-1].copy()
    else:
        start[E // 2] = 0
    rows = dev(r.integers(0, Ra, S).astype(np.int32)) if gathered else None
    say("starts", starts, S, E, n, k, mx, gathered)
    call = gpu_lib.mxfp8_moe_gemm if mx else gpu_lib.fp8_moe_gemm
    need = gpu_lib.moe_gemm_workspace(S, n, k, E, gathered, False, mx)
    ws, ws_check = guarded(max(need, 16))
    D, D_check = guarded(S * n * 4)
    D = D.view(torch.float32).view(S, n)
    D.fill_(float("nan"))
    call(dev(A), B, dev(sa), sb, dev(start), rows=rows, D=D, workspace=ws)
    torch.cuda.synchronize()
    ws_check()
    D_check()
    # rows that no expert claims are not written
    claims = np.zeros(S, int)
    for e in range(E):
        claims[start[e]:max(start[e], start[e + 1])] += 1
    written = ~torch.isnan(D).all(1).cpu().numpy()
    assert not written[claims == 0].any()
    if starts == "falling":
        assert not written.any()


@pytest.mark.parametrize("mode", ["row", "row_e5m2", "mx"])
@pytest.mark.parametrize("cols", [64, 4096, 20000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_without_a_norm(gpu_lib, mode, cols, dtype):
    """0 / sqrt(0 + 0), and roots of negative numbers and NaN: codes 0, a scale of NaN; other rows keep their own."""
    x = torch.randn(5, cols, generator=torch.Generator(device="cuda").manual_seed(cols), device="cuda").to(dtype)
    x[0], x[3, ::2], x[3, 1::2] = 0.0, -0.0, 0.0
    how = {"mx": mode == "mx", "fmt": 1 if mode == "row_e5m2" else 0}
    for eps, bad in ((0.0, (0, 3)), (-1e-3, (0, 3)), (float("nan"), range(5)), (-1e9, range(5))):
        say("no norm", mode, cols, dtype, eps)
        got = gpu_lib.add_rms_norm_quantize(x, eps=eps, return_norm=True, **how)
        for t in range(5):
            if t in bad:
                assert (got.q[t].view(torch.uint8) == 0).all() and torch.isnan(got.norm[t]).all()
                assert (got.scale[t] == 255).all() if mode == "mx" else torch.isnan(got.scale[t])
            else:
                same = gpu_lib.add_rms_norm_quantize(x[t:t + 1], eps=eps, return_norm=True, **how)
                assert torch.equal(got.q[t].view(torch.uint8), same.q[0].view(torch.uint8)) and torch.equal(got.scale[t], same.scale[0])
                assert torch.isfinite(got.norm[t]).all()


def test_more_blocks_of_rows_than_a_launch_holds(gpu_lib):
    """2^35 outputs of one K step on the row kernel, 32 columns x 64 rows a workgroup: 2^24 workgroups of 256
    threads would be 2^32 threads, so that some go round twice."""
    m, n, k = 1 << 15, 1 << 20, 16
    r = rng(35)
    A, sa = operand(r, 64, k, False)
    B, sb = operand(r, n, k, False)
    A, sa, B, sb = dev(A), dev(sa), dev(B), dev(sb)
    say("row kernel", m, n, k)
    D = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")               # 69 GB
    gpu_lib.fp8_gemm_fused(m, n, k, A.repeat(m // 64, 1), B, sa.repeat(m // 64), sb, D=D)
    for at in range(64, m, 64):
        assert torch.equal(D[at:at + 64], D[:64]), at
    for at in (0, n - 5000):
        want = gpu_lib.fp8_gemm_fused(64, 5000, k, A, B[at:at + 5000], sa, sb[at:at + 5000])
        same_but_for_a_step(D[:64, at:at + 5000], want)


@pytest.mark.parametrize("m,k", [(33, 11264), (48, 12288), (64, 10784), (17, 16384)])
def test_block_scales_and_sums_past_64_kb(gpu_lib, m, k):
    """The row kernel's largest LDS: 32 KB of sums beside up to 40 KB of block scales (the last: less of one)."""
    n = 2624 if k == 12288 else 2112
    assert gpu_lib.gemm_fused_workspace(m, n, k, True, True) == 0                           # K is not split
    case(gpu_lib, m, n, k, True, "silu", True, bias=True, residual=True, dtype=torch.bfloat16)
