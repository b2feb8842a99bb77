"""moe_route against the definition, token by token."""

import numpy as np
import pytest
import torch

from block_util import close, f32, rng, typed
from gpu_util import say
from oracle import ffn

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def check(gpu_lib, logits64, logits, k, bias=None, **how):
    want = ffn.route(logits64, k, None if bias is None else bias.double().numpy(), **how)
    got = gpu_lib.moe_route(logits.cuda(), k, bias=None if bias is None else bias.cuda(), **how)
    for name, w, g in zip(got._fields, want, got):
        g = g.cpu().numpy()
        assert g.shape == w.shape, name
        if name == "weights":
            # fp64 scores, one rounding at the end; the exponential's own error is below 2^-48
            close(g.astype(np.float64), w, 2.0 ** -24 * (1 + 2.0 ** -20) * np.abs(w) + 2.0 ** -149, name)
        else:
            assert np.array_equal(g, w), (name, np.argwhere(g != w)[:5])
    return got


@pytest.mark.parametrize("T", [0, 1, 3, 65, 700])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (60, 4), (64, 6), (65, 8), (256, 8), (300, 32), (1024, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(gpu_lib, T, E, k, score):
    r = rng(T, E, k)
    say("route", T, E, k, score)
    for dtype, bias in ((F, None), (BF, f32(0.1 * r.standard_normal(E))[1])):     # bf16 logits: many ties
        check(gpu_lib, *typed(2 * r.standard_normal((T, E)), dtype), k, bias, score=score, renormalize=T != 65, scale=2.5)
    check(gpu_lib, *typed(2 * r.standard_normal((T, E)), BF), k, None, score=score)


@pytest.mark.parametrize("E,groups,top_groups,group_top,k", [(256, 8, 4, 2, 8), (160, 8, 3, 1, 6), (64, 64, 5, 1, 5),
                                                            (48, 3, 3, 2, 7), (192, 64, 20, 2, 10), (20, 4, 1, 2, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_groups(gpu_lib, E, groups, top_groups, group_top, k, score, with_bias):
    r = rng(E, groups, k)
    say("route groups", E, groups, score, with_bias)
    bias = f32(0.2 * r.standard_normal(E))[1] if with_bias else None
    for dtype in (F, BF):
        check(gpu_lib, *typed(2 * r.standard_normal((150, E)), dtype), k, bias, score=score, groups=groups,
              top_groups=top_groups, group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_masked_tied_and_infinite(gpu_lib, score, groups, with_bias):
    r = rng(groups, with_bias)
    E, k = 80, 6
    x = 3 * r.standard_normal((40, E))
    x[0] = -np.inf                                             # a padded token
    x[1, 3:] = -np.inf                                         # fewer than top_k
    x[2] = 1.5                                                 # all tied
    x[3, ::3] = np.nan
    x[4] = np.nan
    x[5, 7], x[5, 70] = np.inf, np.inf
    x[6, 1:] = -3.3e38                                         # the lowest values, but there
    x[7] = np.where(np.arange(E) % 2, 0.0, -0.0)               # zeros of both signs are equal
    x[8, 20:] = -np.inf
    x[9] = 60.0 + np.arange(E) % 7                             # sigmoids that all round to 1
    x[10, 5] = 3.3e38
    bias = f32(0.05 * r.standard_normal(E))[1] if with_bias else None
    if with_bias:
        bias[9], bias[33] = -np.inf, np.nan                    # experts taken out by their bias
    check(gpu_lib, *f32(x), k, bias, score=score, groups=groups, top_groups=max(1, groups // 2))


@pytest.mark.parametrize("T,E,k", [(16385, 128, 1), (3000, 16, 16), (20001, 7, 2)])
def test_route_many_tokens(gpu_lib, T, E, k):
    """Sizes that the definition's loops would take long for: the parts against each other."""
    r = rng(T, E)
    x64, x = f32(r.standard_normal((T, E)))
    x[5::7] = -np.inf
    x64 = x.double().numpy()
    got = [t.cpu().numpy() for t in gpu_lib.moe_route(x.cuda(), k)]
    ids, weights, start, rows, slots = got
    there = np.isfinite(x64[:, 0])
    want = np.argsort(-x64, 1, kind="stable")[:, :k]
    assert np.array_equal(ids, np.where(there[:, None], want, -1))
    flat = np.where(ids < 0, E, ids).reshape(-1)
    order = np.argsort(flat, kind="stable")
    assert np.array_equal(start, np.searchsorted(flat[order], np.arange(E + 1)))
    assert np.array_equal(rows, np.where(flat[order] < E, order // k, -1))
    back = np.empty(T * k, np.int64)
    back[order] = np.arange(T * k)
    assert np.array_equal(slots, np.where(ids < 0, -1, back.reshape(T, k)))
    again = gpu_lib.moe_route(x.cuda(), k)
    assert all(np.array_equal(a, b.cpu().numpy()) for a, b in zip(got, again))
