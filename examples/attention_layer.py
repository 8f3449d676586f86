"""One attention layer served from packed weights, with adapters and a paged
8-bit key/value cache: prompts first, then generation steps.

Every operator of the layer is the library's: the block tables and slot maps
(kv_plan), the projections decoded inside their products
(matmul_packed_batched, matmul_packed), each request's low-rank adapter beside
them (lora_add), the append to the cache (kv_append) and the attention over it
(attention_kv8).  A layer may rotate its heads by position, after their norms
(qk_norm_rope), take its inputs from a packed embedding table (embed_packed) and
serve requests behind one shared prompt (attention_prefix_kv8).  Lengths, tables
and slots stay on the GPU.  Weights are synthetic.

    python examples/attention_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_weight_block_gb300 as ndq  # noqa: E402
import synth  # noqa: E402


class AttentionLayer:
    """q, k, v and output projections of one layer in a packed format, stacked
    adapters of the q, k, v and output projections, and the layer's cache."""

    def __init__(self, fmt="gguf:q8_0", hidden=1024, q_heads=8, kv_heads=2, head_dim=128, adapters=3, rank=8,
                 num_blocks=64, block_size=16, code=torch.float8_e4m3fn, device="cuda", seed=0, rotate=False, vocab=0):
        self.fmt, self.hidden, self.q_heads, self.kv_heads, self.head_dim = fmt, hidden, q_heads, kv_heads, head_dim
        self.sizes = {"q": q_heads * head_dim, "k": kv_heads * head_dim, "v": kv_heads * head_dim, "o": hidden}
        inner = {"q": hidden, "k": hidden, "v": hidden, "o": q_heads * head_dim}
        self.payload = {n: synth.payload(fmt, (rows, inner[n]), seed=seed + i) for i, (n, rows) in enumerate(self.sizes.items())}
        self.w = {n: torch.from_numpy(p).to(device) for n, p in self.payload.items()}
        g = torch.Generator(device=device).manual_seed(seed)
        self.lora = {n: ((torch.randn(adapters, rank, inner[n], device=device, generator=g) / inner[n] ** 0.5).to(torch.bfloat16),
                         (torch.randn(adapters, rows, rank, device=device, generator=g) * 0.1).to(torch.bfloat16))
                     for n, rows in self.sizes.items()}
        self.ranks = torch.tensor([rank - i % 2 for i in range(adapters)], dtype=torch.int32, device=device)
        self.scales = torch.linspace(0.5, 1.5, adapters, device=device)
        self.cache = ndq.KvCache.empty(num_blocks, kv_heads, block_size, head_dim, code, device)
        self.workspace = ndq.attention_workspace(0, 0, q_heads, self.cache)
        self.shared_workspace, self.shared_tokens = None, -1  # made for the largest step so far
        # rotation by position after the norms of the query and key heads
        self.inv_freq = None
        if rotate:
            self.inv_freq = 10000.0 ** (-torch.arange(0, head_dim, 2, device=device) / head_dim)
            self.q_norm, self.k_norm = (1 + 0.1 * torch.randn(head_dim, device=device, generator=g) for _ in range(2))
        # the packed embedding table
        self.vocab = vocab
        if vocab:
            self.table = torch.from_numpy(synth.payload(fmt, (vocab, hidden), seed=seed + 9)).to(device)

    def embed(self, ids):
        """ids [T]: [T, hidden] bfloat16."""
        return ndq.embed_packed(self.fmt, self.table, self.vocab, self.hidden, ids)

    def project(self, name, y, x, adapter):
        a, b = self.lora[name]
        return ndq.lora_add(x, a, b, self.ranks, self.scales, adapter, y, out=y)

    def __call__(self, x, adapter, plan, block_table, max_q, shared=None):
        """x [T, hidden] bfloat16, adapter [T] int32 (-1: none), shared None or
        (group_start, prefix_len) of requests that share prefixes: [T, hidden] float32."""
        names = ("q", "k", "v")
        ys = ndq.matmul_packed_batched([(self.fmt, self.w[n], self.sizes[n]) for n in names], self.hidden, x,
                                       out_dtype=torch.bfloat16)
        q, k, v = (self.project(n, y, x, adapter) for n, y in zip(names, ys))
        q, k, v = (y.unflatten(1, (-1, self.head_dim)) for y in (q, k, v))
        if self.inv_freq is not None:
            ndq.qk_norm_rope(q, k, plan.positions, self.inv_freq, self.q_norm, self.k_norm, q_out=q, k_out=k)
        ndq.kv_append(self.cache, k, v, plan.slots)
        if shared is None:
            o = ndq.attention_kv8(q, self.cache, block_table, plan.kv_len, q_start=plan.q_start, max_q=max_q,
                                  workspace=self.workspace).flatten(1)
        else:
            if q.shape[0] > self.shared_tokens:
                self.shared_workspace = ndq.attention_prefix_workspace(self.cache, q.shape[0], self.q_heads)
                self.shared_tokens = q.shape[0]
            o = ndq.attention_prefix_kv8(q, self.cache, block_table, plan.kv_len, *shared, q_start=plan.q_start, max_q=max_q,
                                         workspace=self.shared_workspace).flatten(1)
        y = ndq.matmul_packed(self.fmt, self.w["o"], self.hidden, self.q_heads * self.head_dim, o)
        return self.project("o", y, o, adapter)


class Requests:
    """What a server keeps of its requests: lengths, block tables, free blocks."""

    def __init__(self, n, num_blocks, width, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.cached = torch.zeros(n, **i32)
        self.table = torch.full((n, width), -1, **i32)
        self.free = torch.arange(num_blocks - 1, -1, -1, **i32)
        self.count = torch.tensor([num_blocks], **i32)

    def plan(self, fresh, block_size):
        """Blocks and slots for the next `fresh[r]` tokens of every request."""
        new = torch.tensor(fresh, dtype=torch.int32, device=self.cached.device)
        plan = ndq.kv_plan(self.cached, new, block_size, self.free, self.count, self.table, n_tokens=sum(fresh))
        self.cached, self.count = plan.kv_len, plan.free_left
        return plan

    def share(self, tokens, block_size):
        """Every request goes on from the first one's first `tokens` tokens, a
        multiple of block_size; what attention_prefix_kv8 is to know of it."""
        assert tokens % block_size == 0
        self.table[1:] = -1
        self.table[1:, :tokens // block_size] = self.table[0, :tokens // block_size]
        self.cached[1:] = tokens
        i32 = dict(dtype=torch.int32, device=self.table.device)
        return torch.tensor([0, len(self.cached)], **i32), torch.tensor([tokens], **i32)


def main():
    torch.manual_seed(0)
    layer = AttentionLayer()
    prompts = [45, 7, 130]
    reqs = Requests(len(prompts), layer.cache.num_blocks, 16)
    adapter_of = torch.tensor([0, -1, 2], dtype=torch.int32, device="cuda")
    for fresh in [prompts] + [[1] * len(prompts)] * 4:
        plan = reqs.plan(fresh, layer.cache.block_size)
        x = torch.randn(sum(fresh), layer.hidden, device="cuda").to(torch.bfloat16)
        adapter = torch.repeat_interleave(adapter_of, torch.tensor(fresh, device="cuda"))
        y = layer(x, adapter, plan, reqs.table, max(fresh))
        print(f"{sum(fresh):4d} tokens -> {tuple(y.shape)}, |y| {y.abs().mean().item():.4f}, cached {reqs.cached.tolist()}, "
              f"free blocks {reqs.count.item()}")
    # three answers to one prompt, rotated heads, tokens by their ids
    layer = AttentionLayer(rotate=True, vocab=5000)
    reqs = Requests(3, layer.cache.num_blocks, 16)
    shared = None
    for fresh in [[128, 0, 0]] + [[1, 1, 1]] * 4:
        plan = reqs.plan(fresh, layer.cache.block_size)
        x = layer.embed(torch.randint(0, layer.vocab, (sum(fresh),), device="cuda"))
        y = layer(x, torch.full((sum(fresh),), -1, dtype=torch.int32, device="cuda"), plan, reqs.table, max(fresh), shared)
        if shared is None:
            shared = reqs.share(128, layer.cache.block_size)
        print(f"{sum(fresh):4d} tokens -> {tuple(y.shape)}, |y| {y.abs().mean().item():.4f}, cached {reqs.cached.tolist()}")
    if ndq.get_device_fault():
        raise SystemExit("device fault word set")


if __name__ == "__main__":
    main()
