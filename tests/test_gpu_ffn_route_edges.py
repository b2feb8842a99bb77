"""moe_route where the fp32 look at the choices and the fp64 one part, and where
groups have few available experts: the definition, token by token."""

import numpy as np
import pytest
import torch

from block_util import f32, rng
from gpu_util import say
from test_gpu_ffn_route import check

pytestmark = pytest.mark.gpu


# experts a lane: 1, 4, 8 and 16; groups of 8 (several lanes, or a lane), of 5 (lanes shared by two) and of 64
SIZES = [(16, 2), (15, 3), (256, 32), (250, 50), (512, 64), (1024, 16)]


@pytest.mark.parametrize("E,groups", SIZES)
@pytest.mark.parametrize("renormalize", [False, True])
def test_groups_that_only_fp64_tells_apart(gpu_lib, E, groups, renormalize):
    """All sigmoids are 1 in fp32, where the first group wins; in fp64 the second one does, which has two experts."""
    width = E // groups
    x = np.full((9, E), 20.0)
    x[:, width:2 * width] = -np.inf
    x[:, width:width + 2] = 21.0
    x[1::3, 2 * width - 1] = np.nan
    say("close groups", E, groups)
    check(gpu_lib, *f32(x), 4, None, score="sigmoid", groups=groups, top_groups=1, renormalize=renormalize)


@pytest.mark.parametrize("E,groups", SIZES)
@pytest.mark.parametrize("group_top", [1, 2])
def test_close_groups_of_masked_experts(gpu_lib, E, groups, group_top):
    """Whole logits of 20 to 32, whose sigmoids are 1 in fp32 and far apart in fp64, most of them masked."""
    r = rng(E, groups, group_top)
    x = r.integers(20, 33, (120, E)).astype(np.float64)
    x[r.random(x.shape) < np.linspace(0.2, 1.0, 120)[:, None]] = -np.inf
    say("masked groups", E, groups, group_top)
    for top_groups in {1, 2, groups - 1}:
        check(gpu_lib, *f32(x), 6, None, score="sigmoid", groups=groups, top_groups=top_groups, group_top=group_top)


@pytest.mark.parametrize("E,groups", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_of_infinity(gpu_lib, E, groups, score):
    """A bias of +inf puts an expert first, but not its group before those with enough experts."""
    r = rng(E, groups)
    width = E // groups
    x = 2 * r.standard_normal((12, E))
    bias = 0.1 * r.standard_normal(E)
    bias[1] = np.inf
    bias[width + 1:width + 3] = np.inf
    x[::2, :width] = np.where(np.arange(width) == 1, 0.5, -np.inf)          # group 0: its only expert
    x[1::4, width:2 * width] = -np.inf
    say("infinite bias", E, groups, score)
    for top_groups in {1, groups - 1}:
        check(gpu_lib, *f32(x), 5, f32(bias)[1], score=score, groups=groups, top_groups=top_groups)


@pytest.mark.parametrize("E,groups", [(16, 8), (60, 20), (256, 32), (1024, 64)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [3.0, 1000.0, 3e5])
def test_biases_that_cancel(gpu_lib, E, groups, score, size):
    """Groups whose two best choices are size + p and p - size: their sums are as close as p's fp32 rounding at that size."""
    r = rng(E, groups, score == "softmax")
    width = E // groups
    x = 0.01 * r.standard_normal((200, E))
    bias = np.full(E, -4.0 * size)
    bias[::width], bias[1::width] = size, -size
    say("cancelling biases", E, groups, score, size)
    for top_groups in (1, groups // 2):
        check(gpu_lib, *f32(x), 2, f32(bias)[1], score=score, groups=groups, top_groups=top_groups)


def test_groups_that_are_refused(gpu_lib):
    """One group has no other to choose from; None stands for a group_top that fits."""
    x = torch.randn(3, 8, device="cuda")
    want = gpu_lib.moe_route(x, 2)
    for how in ({"groups": 1, "top_groups": 1}, {"group_top": 1}, {"group_top": 2}):
        assert all(torch.equal(a, b) for a, b in zip(gpu_lib.moe_route(x, 2, **how), want)), how
    gpu_lib.moe_route(x[:, :1].contiguous(), 1)
    for how in ({"top_groups": 2}, {"top_groups": 0}, {"group_top": 3}, {"group_top": 0}, {"groups": 4, "top_groups": 5},
                {"groups": 8, "group_top": 2}, {"groups": 3}):
        with pytest.raises(gpu_lib.Fp8gError):
            gpu_lib.moe_route(x, 2, **how)
