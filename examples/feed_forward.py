"""The feed-forward half of a served layer, end to end on this library, dense or
with routed experts:

  x, residual -> add_rms_norm_quantize
    dense:   -> fp8_gemm_fused (gate and up) -> fp8_quantize_ex -> fp8_gemm_fused (down, + residual)
    experts: -> moe_route -> fp8_moe_gemm (gate and up, gathered) -> fp8_quantize_ex -> fp8_moe_gemm (down)
             -> moe_combine (+ residual)

    python examples/feed_forward.py
"""

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_scaled_gemm_amd as fp8g  # noqa: E402


def random(generator, *shape, scale=1.0):
    return torch.randn(*shape, generator=generator, device="cuda") * scale


def quantized(generator, rows, k):
    """A random weight [rows, k] as codes and their row scales."""
    return fp8g.fp8_quantize_rowwise(random(generator, rows, k, scale=k ** -0.5))


class FeedForward:
    """Random weights of one layer's dense feed-forward half."""

    def __init__(self, hidden=4096, inner=14336, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.inner = hidden, inner
        self.norm = 1 + random(g, hidden, scale=0.1)
        self.w_in, self.w_out = quantized(g, 2 * inner, hidden), quantized(g, hidden, inner)

    def __call__(self, x, residual):
        """x, residual [T, hidden] bf16: the layer's output with the residual stream added."""
        n = fp8g.add_rms_norm_quantize(x, self.norm, residual)
        h = fp8g.fp8_gemm_fused(x.shape[0], self.inner, self.hidden, n.q, self.w_in[0], n.scale, self.w_in[1], act="silu", gated=True)
        q, scale = fp8g.fp8_quantize_ex(h)
        # over the residual stream itself
        return fp8g.fp8_gemm_fused(x.shape[0], self.hidden, self.inner, q, self.w_out[0], scale, self.w_out[1], residual=n.sum, D=n.sum)


class Experts:
    """Random weights of one layer's routed experts."""

    def __init__(self, hidden=4096, inner=1024, experts=64, top_k=6, groups=1, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.inner, self.experts, self.top_k, self.groups = hidden, inner, experts, top_k, groups
        self.norm = 1 + random(g, hidden, scale=0.1)
        self.router = random(g, experts, hidden, scale=hidden ** -0.5)
        self.bias = random(g, experts, scale=0.01)
        stack = lambda rows, k: [t.unflatten(0, (experts, rows)) for t in quantized(g, experts * rows, k)]   # noqa: E731
        self.w_in, self.w_out = stack(2 * inner, hidden), stack(hidden, inner)

    def route(self, normed):
        logits = normed.float() @ self.router.T
        return fp8g.moe_route(logits, self.top_k, bias=self.bias, score="sigmoid", groups=self.groups,
                              top_groups=max(1, self.groups // 2), group_top=2 if self.groups > 1 else 1)

    def experts_of(self, n, r):
        """The experts' rows of normed tokens n, in the order of route r."""
        h = fp8g.fp8_moe_gemm(n.q, self.w_in[0], n.scale, self.w_in[1], r.expert_start, rows=r.rows, act="silu", gated=True)
        q, scale = fp8g.fp8_quantize_ex(h)
        return h, fp8g.fp8_moe_gemm(q, self.w_out[0], scale, self.w_out[1], r.expert_start)

    def __call__(self, x, residual):
        n = fp8g.add_rms_norm_quantize(x, self.norm, residual, return_norm=True)
        r = self.route(n.norm)
        return fp8g.moe_combine(self.experts_of(n, r)[1], r.slots, r.weights, residual=n.sum, out=n.sum)


def main():
    for name, layer in (("dense 4096 -> 2 x 14336", FeedForward()), ("64 experts 4096 -> 2 x 1024, 6 a token", Experts()),
                        ("128 experts in 8 groups", Experts(inner=512, experts=128, top_k=8, groups=8))):
        for tokens in (1, 64, 4096):
            x, residual = (random(torch.Generator(device="cuda").manual_seed(s), tokens, layer.hidden).bfloat16() for s in (1, 2))
            layer(x, residual)
            torch.cuda.synchronize()
            t = time.perf_counter()
            y = layer(x, residual)
            torch.cuda.synchronize()
            print("%-40s %5d tokens  %8.1f us  |y| %.4f" % (name, tokens, 1e6 * (time.perf_counter() - t), y.float().norm() / y.numel() ** 0.5))


if __name__ == "__main__":
    main()
