"""The attention half of a served layer, end to end on this library:

  x -> fp8_quantize_ex -> fp8_gemm_scaled (QKV) -> lora_add -> qk_norm_rope
    -> kv4_append -> kv4_attention -> fp8_quantize_ex -> fp8_gemm_scaled (output) -> lora_add

for a batch of requests that hold different numbers of tokens and different
adapters, over one paged MXFP4 cache.  A step takes any mix of prompts and single
decoded tokens.

    python examples/attention_block.py
"""

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_scaled_gemm_amd as fp8g  # noqa: E402


class AttentionBlock:
    """Random weights of one layer, its adapters and its cache."""

    def __init__(self, hidden=4096, q_heads=32, kv_heads=8, dim=128, rank=16, adapters=4, pages=512, page_size=16,
                 max_position=8192, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s, scale=1.0: torch.randn(*s, generator=g, device="cuda") * scale   # noqa: E731
        self.hidden, self.q_heads, self.kv_heads, self.dim, self.page_size = hidden, q_heads, kv_heads, dim, page_size
        self.qkv_width, self.out_width = (q_heads + 2 * kv_heads) * dim, q_heads * dim
        self.w_qkv = fp8g.fp8_quantize_rowwise(rand(self.qkv_width, hidden, scale=hidden ** -0.5))
        self.w_out = fp8g.fp8_quantize_rowwise(rand(hidden, self.out_width, scale=self.out_width ** -0.5))

        def pair(k, n):
            return (rand(adapters, rank, k, scale=k ** -0.5).bfloat16(), rand(adapters, n, rank, scale=0.1).bfloat16())
        self.lora_qkv, self.lora_out = pair(hidden, self.qkv_width), pair(self.out_width, hidden)
        self.lora_scale = torch.ones(adapters, device="cuda")
        self.q_norm, self.k_norm = 1 + rand(dim, scale=0.1), 1 + rand(dim, scale=0.1)
        angle = torch.arange(max_position, device="cuda").double()[:, None] * \
            10000.0 ** (-torch.arange(dim // 2, device="cuda").double() / (dim // 2))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        self.cache = fp8g.kv4_cache(pages, kv_heads, page_size, dim, dim)

    def project(self, x, weight, lora, n, step):
        """x [T, k] bf16 through an FP8 projection and its adapters: [T, n] bf16."""
        codes, scale = fp8g.fp8_quantize_ex(x)
        y = fp8g.fp8_gemm_scaled(x.shape[0], n, x.shape[1], codes, weight[0], scale, weight[1])
        return fp8g.lora_add(y, x, lora[0], lora[1], self.lora_scale, step["q_start"], step["adapter"], out=y)

    def qkv(self, x, step):
        """Normed and rotated queries and keys, and values, [T, heads, dim] each."""
        T, (H, K, D) = x.shape[0], (self.q_heads, self.kv_heads, self.dim)
        rows = self.project(x, self.w_qkv, self.lora_qkv, self.qkv_width, step)
        q, k = rows[:, :H * D].unflatten(1, (H, D)), rows[:, H * D:(H + K) * D].unflatten(1, (K, D))
        # in place: the projection's own rows, values untouched
        fp8g.qk_norm_rope(q, k, self.q_norm, self.k_norm, step["positions"], self.cos_sin, q_out=q, k_out=k)
        return q, k, rows[:, (H + K) * D:].unflatten(1, (K, D))

    def attend(self, q, k, v, step):
        fp8g.kv4_append(self.cache, k, v, step["slots"])
        return fp8g.kv4_attention(q, self.cache, step["page_table"], step["q_start"], step["kv_len"])

    def __call__(self, x, step):
        q, k, v = self.qkv(x, step)
        out = self.attend(q, k, v, step).flatten(1)
        return self.project(out, self.w_out, self.lora_out, self.hidden, step)


def plan(block, lengths, new, adapters, page_table):
    """What a step hands to the operators: sequence b holds lengths[b] tokens and
    gets new[b] more; adapters[b] is its adapter (negative: none)."""
    ints = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device="cuda")   # noqa: E731
    starts, positions, slots = [0], [], []
    for b, (have, n) in enumerate(zip(lengths, new)):
        starts.append(starts[-1] + n)
        for p in range(have, have + n):
            positions.append(p)
            slots.append(page_table[b][p // block.page_size] * block.page_size + p % block.page_size)
    return {"q_start": ints(starts), "kv_len": ints([h + n for h, n in zip(lengths, new)]), "positions": ints(positions),
            "slots": ints(slots, torch.int64), "adapter": ints(adapters), "page_table": ints(page_table)}


def main():
    block = AttentionBlock()
    lengths, adapters = [0, 0, 0], [2, -1, 0]
    table = [list(range(b * 128, b * 128 + 128)) for b in range(3)]
    for name, new in (("prompts", [700, 33, 1201]), ("one token each", [1, 1, 1]), ("a prompt beside two tokens", [1, 300, 1])):
        step = plan(block, lengths, new, adapters, table)
        x = torch.randn(sum(new), block.hidden, device="cuda").bfloat16()
        block(x, step)
        torch.cuda.synchronize()
        t = time.perf_counter()
        y = block(x, step)                  # the same rows again: same slots, same result
        torch.cuda.synchronize()
        print("%-28s %5d tokens  %8.1f us  |y| %.4f" % (name, sum(new), 1e6 * (time.perf_counter() - t), y.float().norm() / y.numel() ** 0.5))
        lengths = [a + b for a, b in zip(lengths, new)]


if __name__ == "__main__":
    main()
