"""The feed-forward half's products and norm at the borders of what they take."""

import numpy as np
import pytest
import torch

from block_util import rng
from ffn_util import dev, operand
from gpu_util import say
from test_gpu_ffn_limits import guarded

pytestmark = pytest.mark.gpu


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
