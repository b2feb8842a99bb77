"""Arrays past 4 GiB, workspaces of exactly their size, other streams, host tensors."""

import numpy as np
import pytest
import torch

from block_util import rng
from ffn_util import dev, operand
from gpu_util import say
from test_gpu_block_limits import guarded

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def same_but_for_a_step(a, b):
    """Two roundings of sums that differ by their order: a step of bf16 (2^-7 of the value),
    and 128 products at 2^-24 of the largest."""
    a, b = a.double(), b.double()
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -16 * b.abs().max()).all()


def test_rows_past_4_gib(gpu_lib):
    R, C = 280000, 8192                                   # x, sum: 4.6 GB each
    part = torch.randn(1000, C, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF)
    w = torch.rand(C, device="cuda") + 0.5
    x = part.repeat(R // 1000, 1)
    say("norm", R, C)
    n = gpu_lib.add_rms_norm_quantize(x, w, x)
    want = gpu_lib.add_rms_norm_quantize(part, w, part)
    for at in (0, 131000, R - 1000):
        assert torch.equal(n.q[at:at + 1000], want.q) and torch.equal(n.scale[at:at + 1000], want.scale)
        assert torch.equal(n.sum[at:at + 1000], want.sum)
    del n
    say("combine", R, C)
    slots = torch.tensor([[R - 1, 0], [5, R - 1000], [-1, 262144]], dtype=torch.int32, device="cuda")
    out = gpu_lib.moe_combine(x, slots, torch.ones(3, 2, device="cuda"))
    p = part.double()
    assert torch.equal(out, torch.stack([p[999] + p[0], p[5] + p[0], p[144]]).to(BF))


@pytest.mark.parametrize("mx", [False, True])
def test_products_past_4_gib(gpu_lib, mx):
    S, n, k, E = 280000, 8200, 96, 3                      # D: 4.6 GB
    r = rng(7)
    A, sa = operand(r, 4000, k, mx)
    B, sb = operand(r, E * n, k, mx)
    A, sa, B, sb = dev(A), dev(sa), dev(B), dev(sb)
    many, s_many = A.repeat(70, 1), sa.repeat(*((70, 1) if mx else (70,)))
    fused, moe = (gpu_lib.mxfp8_gemm_fused, gpu_lib.mxfp8_moe_gemm) if mx else (gpu_lib.fp8_gemm_fused, gpu_lib.fp8_moe_gemm)
    say("fused", S, n, k, mx)
    D = fused(S, n, k, many, B[:n], s_many, sb[:n], act="silu")
    want = fused(4000, n, k, A, B[:n], sa, sb[:n], act="silu")
    for at in (0, 128000, S - 4000):
        same_but_for_a_step(D[at:at + 4000], want)
    say("experts", S, n, k, mx)
    start = torch.tensor([0, 40, 4000, S], dtype=torch.int32, device="cuda")
    rows = (torch.arange(S, device="cuda") % 4000).int()
    moe(A, B.view(E, n, k), sa, sb.view(E, n, -1) if mx else sb.view(E, n), start, rows=rows, act="silu", D=D)
    want = fused(4000, n, k, A, B[2 * n:], sa, sb[2 * n:], act="silu")
    for at in (4000, S - 4000):
        same_but_for_a_step(D[at:at + 4000], want)


@pytest.mark.parametrize("m,n,k,mx,gated", [(200, 256, 6144, False, True), (200, 256, 6144, True, False), (700, 1000, 672, True, True),
                                            (129, 130, 4160, True, False)])
def test_fused_workspace(gpu_lib, m, n, k, mx, gated):
    r = rng(m, k)
    rows = 2 * n if gated else n
    A, sa = operand(r, m, k, mx)
    B, sb = operand(r, rows, k, mx)
    call = gpu_lib.mxfp8_gemm_fused if mx else gpu_lib.fp8_gemm_fused
    need = gpu_lib.gemm_fused_workspace(m, n, k, gated, mx)
    assert need > 0
    args = (m, n, k, dev(A), dev(B), dev(sa), dev(sb))
    want = call(*args, gated=gated)
    ws, check = guarded(need)
    for fill in (0x00, 0xFF):
        ws.fill_(fill)
        assert torch.equal(call(*args, gated=gated, workspace=ws), want)
        check()
    with pytest.raises(Exception):
        call(*args, gated=gated, workspace=ws[:need - 16])


@pytest.mark.parametrize("S,n,k,mx,gathered", [(900, 136, 128, False, True), (900, 136, 672, True, True), (900, 136, 672, True, False),
                                               (900, 136, 128, False, False)])
def test_experts_workspace(gpu_lib, S, n, k, mx, gathered):
    r = rng(S, k)
    A, sa = operand(r, 300 if gathered else S, k, mx)
    B, sb = operand(r, 3 * n, k, mx)
    start = torch.tensor([7, 200, 200, 880], dtype=torch.int32, device="cuda")
    rows = torch.from_numpy(r.integers(0, 300, S).astype(np.int32)).cuda() if gathered else None
    call = gpu_lib.mxfp8_moe_gemm if mx else gpu_lib.fp8_moe_gemm
    args = (dev(A), dev(B).view(3, n, k), dev(sa), dev(sb).view(3, n, -1) if mx else dev(sb).view(3, n), start)
    ws, check = guarded(gpu_lib.moe_gemm_workspace(S, n, k, 3, gathered, False, mx))
    want = call(*args, rows=rows)
    for fill in (0x00, 0xFF):
        ws.fill_(fill)
        got = call(*args, rows=rows, workspace=ws)
        check()
        assert torch.equal(got[7:880], want[7:880])


def test_route_workspace_and_largest_sizes(gpu_lib):
    for T, E, k in ((25, 8, 2), (3000, 1024, 32), (5000, 33, 8)):
        logits = torch.randn(T, E, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda")
        want = gpu_lib.moe_route(logits, k)
        ws, check = guarded(gpu_lib.moe_route_workspace(T, E, k))
        for fill in (0x00, 0xFF):
            ws.fill_(fill)
            got = gpu_lib.moe_route(logits, k, workspace=ws)
            check()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(logits.gather(1, want.ids.long()), logits.topk(k).values)


def test_two_streams_at_once(gpu_lib):
    r = rng(3)
    A, sa = operand(r, 200, 6144, False)
    B, sb = operand(r, 512, 6144, False)
    args = (200, 256, 6144, dev(A), dev(B), dev(sa), dev(sb))
    logits = torch.randn(300, 64, device="cuda")
    want, routed = gpu_lib.fp8_gemm_fused(*args, gated=True, act="silu"), gpu_lib.moe_route(logits, 4)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((gpu_lib.fp8_gemm_fused(*args, gated=True, act="silu"), gpu_lib.moe_route(logits, 4)))
    torch.cuda.synchronize()
    for D, route in got:
        assert torch.equal(D, want) and all(torch.equal(a, b) for a, b in zip(route, routed))


def test_host_tensors_are_refused(gpu_lib):
    x = torch.randn(4, 64, device="cuda").to(BF)
    q = torch.zeros(4, 64, dtype=torch.uint8, device="cuda")
    s = torch.ones(4, device="cuda")
    start = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    slots = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.ones(4, 2, device="cuda")
    calls = [(gpu_lib.add_rms_norm_quantize, (x, torch.ones(64, device="cuda"), x)),
             (lambda a, b, c, d: gpu_lib.fp8_gemm_fused(4, 4, 64, a, b, c, d), (q, q, s, s)),
             (lambda a, b, c, d, e: gpu_lib.fp8_moe_gemm(a, b, c, d, e), (q, q[None], s, s[None], start)),
             (lambda a: gpu_lib.moe_route(a, 2), (x,)), (gpu_lib.moe_combine, (x, slots, w, x))]
    for call, args in calls:
        call(*args)
        for i in range(len(args)):
            with pytest.raises(Exception):
                call(*args[:i], args[i].cpu(), *args[i + 1:])
