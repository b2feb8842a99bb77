"""Seeded inputs and bounds for the tests of the attention block's operators."""

import numpy as np
import torch

from oracle import block

BF16_HALF = 2.0 ** -8      # largest relative error of a rounding to bf16 (8 significant bits)
F32_HALF = 2.0 ** -24


def rng(*key):
    return np.random.default_rng([abs(int(k)) for k in key])


def bf16(a):
    """float64 array rounded to bf16 values, and the bf16 tensor of them (host)."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t


def f32(a):
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32))
    return t.double().numpy(), t


def typed(a, dtype):
    return bf16(a) if dtype == torch.bfloat16 else f32(a)


def half_ulp(dtype):
    return BF16_HALF if dtype == torch.bfloat16 else F32_HALF


def host(t):
    return t.detach().cpu().double().numpy()


def close(got, want, tol, what):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d of %d over the bound; worst error / bound %.3g at %s" % (
        what, bad.sum(), bad.size, np.max(np.where(bad, err / np.maximum(tol, 1e-300), 0)),
        np.unravel_index(np.argmax(np.where(np.isnan(err), np.inf, err / np.maximum(tol, 1e-300))), err.shape))


class Paged:
    """A paged cache with sequences of given lengths in shuffled pages; bytes
    that no sequence owns hold 0xFF (scale code 255: NaN)."""

    def __init__(self, lengths, heads, dk, dv, page, seed, spare=3, channel=1.0):
        r = rng(seed, 77)
        counts = [(n + page - 1) // page for n in lengths]
        self.pages = max(1, sum(counts)) + spare
        self.page, self.heads, self.dk, self.dv = page, heads, dk, dv
        order = r.permutation(self.pages)
        self.max_pages = max(counts + [1]) + 1
        self.table = r.choice([-7, 1 << 30, -(1 << 31), 0], size=(len(lengths), self.max_pages)).astype(np.int32)
        self.k, self.v, at = [], [], 0
        full = lambda *s: np.full(s, 255, np.uint8)   # noqa: E731
        self.arrays = [full(self.pages, heads, page, dk // 2), full(self.pages, heads, dk // 32, page),
                       full(self.pages, heads, page, dv // 2), full(self.pages, heads, dv // 32, page)]
        for b, n in enumerate(lengths):
            ids = order[at:at + counts[b]]
            at += counts[b]
            self.table[b, :counts[b]] = ids
            for dim, c, s, keep in ((dk, 0, 1, self.k), (dv, 2, 3, self.v)):
                x = r.standard_normal((n, heads, dim)) * np.exp(channel * r.standard_normal((1, heads, dim)))
                codes, scales = block.mxfp4_quantize(x.astype(np.float32)) if n else (
                    np.zeros((0, heads, dim), np.uint8), np.zeros((0, heads, dim // 32), np.uint8))
                for j in range(n):
                    self.arrays[c][ids[j // page], :, j % page] = block.pack(codes[j])
                    self.arrays[s][ids[j // page], :, :, j % page] = scales[j]
                keep.append(block.mxfp4_values(codes, scales))

    def device(self, fp8g):
        return fp8g.KV4Cache(*[torch.from_numpy(a).cuda() for a in self.arrays])
