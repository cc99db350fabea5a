"""One attention block of a model with 4-bit weights and a 4-bit cache, as a server runs it:

    projection of the hidden states to queries, keys and values     bitmm_qmm
    RMS norm of each query and key head, and the position rotation  bitmm_qk_norm_rope
    keys and values quantized into the cache's pages                bitmm_kv_append
    attention over the cache                                        bitmm_kv_attention
    projection back                                                 bitmm_qmm

Three prompts of different lengths go through it in chunks, then all three sequences decode
together, a token each a step, the step captured once into a HIP graph.

    python examples/attention_block.py
"""

import os
import sys
import time
from dataclasses import dataclass

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import bit_matmul_amd as bm


@dataclass
class Batch:
    """New tokens of some sequences, side by side, and what the block has to know of them."""
    positions: torch.Tensor   # int32 [T]
    slots: torch.Tensor       # int64 [T]: where the tokens' keys and values go
    page_table: torch.Tensor  # int32 [B, pages]
    kv_lens: torch.Tensor     # int32 [B], the new tokens included
    cu_q: torch.Tensor        # int32 [B + 1]
    max_q: int
    max_kv: int

    def take(self, other):
        """Another batch of the same shapes, into these tensors (those of a captured graph)."""
        for name in ("positions", "slots", "page_table", "kv_lens", "cu_q"):
            getattr(self, name).copy_(getattr(other, name))


class Pages:
    """Which pages of a cache each of `batch` sequences has. Lives on the host."""

    def __init__(self, cache, batch, max_tokens):
        self.size, self.device, self.max_tokens = cache.page_size, cache.device, max_tokens
        self.free = list(range(cache.num_pages))[::-1]
        self.table = torch.zeros(batch, -(-max_tokens // self.size), dtype=torch.int32)
        self.lens, self.held = [0] * batch, [0] * batch

    def extend(self, counts, bound=None):
        """Room for counts[b] more tokens of each sequence: the Batch of them. bound: of the
        lengths, where a graph is to be replayed at lengths to come."""
        positions, slots, cu = [], [], [0]
        for b, n in enumerate(counts):
            first, self.lens[b] = self.lens[b], self.lens[b] + n
            if self.lens[b] > self.max_tokens:
                raise ValueError(f"sequence {b} passes {self.max_tokens} tokens")
            while self.held[b] * self.size < self.lens[b]:
                self.table[b, self.held[b]] = self.free.pop()
                self.held[b] += 1
            at = torch.arange(first, self.lens[b])
            positions.append(at)
            slots.append(self.table[b].long()[at // self.size] * self.size + at % self.size)
            cu.append(cu[-1] + n)
        there = lambda t, dtype: t.to(dtype).to(self.device)
        return Batch(there(torch.cat(positions), torch.int32), there(torch.cat(slots), torch.int64),
                     self.table.to(self.device), there(torch.tensor(self.lens), torch.int32),
                     there(torch.tensor(cu), torch.int32), max(counts), bound or max(self.lens))


class AttentionBlock:
    """qkv, out: (words, scales, biases) of 4-bit projections, [(q_heads + 2 kv_heads) * D, hidden]
    and [hidden, q_heads * D]; q_norm, k_norm: [D]; rope: (inv_freq, rope_scale)."""

    def __init__(self, qkv, out, q_norm, k_norm, rope, q_heads, cache, window=0, sinks=0):
        self.qkv, self.out, self.q_norm, self.k_norm = qkv, out, q_norm, k_norm
        self.inv_freq, self.rope_scale = rope
        self.q_heads, self.cache, self.window, self.sinks = q_heads, cache, window, sinks
        # Set by the library if a slot, page or length is out of range.
        self.status = torch.zeros(1, dtype=torch.int32, device=cache.device)

    def __call__(self, x, batch):
        tokens, hq, hk = x.shape[0], self.q_heads, self.cache.kv_heads
        heads = bm.qmm(x, *self.qkv, 4).view(tokens, hq + 2 * hk, self.cache.head_dim)
        q, k, v = heads[:, :hq], heads[:, hq:hq + hk], heads[:, hq + hk:]
        q, k = bm.qk_norm_rope(q, k, self.q_norm, self.k_norm, batch.positions, self.inv_freq, rope_scale=self.rope_scale)
        bm.bitmm_kv_append(k, v, batch.slots, self.cache, status=self.status)
        y = bm.kv_attention(q, self.cache, batch.page_table, batch.kv_lens, batch.cu_q, max_q=batch.max_q,
                            max_kv=batch.max_kv, window=self.window, sinks=self.sinks, status=self.status)
        return bm.qmm(y.view(tokens, -1), *self.out, 4)


class DecodeGraph:
    """The block's step of one token a sequence, captured. `batch` serves as the graph's own
    tensors; its max_kv bounds the lengths of all replays."""

    def __init__(self, block, x, batch):
        self.x, self.batch = x.clone(), batch
        block(self.x, batch)  # what loads at a first call, loads outside the capture
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = block(self.x, batch)

    def __call__(self, x, batch):
        self.x.copy_(x)
        self.batch.take(batch)
        self.graph.replay()
        return self.y


def random_projection(rows, columns, generator, device):
    """A 4-bit projection of a size that keeps the variance of its input, in groups of 64."""
    words = torch.randint(-2 ** 31, 2 ** 31, (rows, columns // 8), generator=generator).to(torch.int32)
    scales = ((0.5 + torch.rand(rows, columns // 64, generator=generator)) / (4.6 * columns ** 0.5)).bfloat16()
    return words.to(device), scales.to(device), (-7.5 * scales.float()).bfloat16().to(device)


def random_block(hidden, q_heads, kv_heads, head_dim, num_pages, page_size=64, theta=1e6, device="cuda", seed=0, **kw):
    g = torch.Generator().manual_seed(seed)
    cache = bm.KVCache.empty(num_pages, page_size, kv_heads, head_dim, device=device)
    norms = [(1 + 0.1 * torch.randn(head_dim, generator=g)).bfloat16().to(device) for _ in range(2)]
    return AttentionBlock(random_projection((q_heads + 2 * kv_heads) * head_dim, hidden, g, device),
                          random_projection(hidden, q_heads * head_dim, g, device), *norms,
                          bm.rope_frequencies(head_dim, theta, device=device), q_heads, cache, **kw)


def serve(block, prompts, steps, chunk, max_tokens, graph=True):
    """Takes prompts [n_b, hidden] through the block, `chunk` tokens of each at a time, then
    decodes steps[i] [B, hidden] one after the other. Returns the block's outputs of each
    sequence's tokens."""
    pages = Pages(block.cache, len(prompts), max_tokens)
    outputs = [[] for _ in prompts]

    def keep(y, counts):
        for b, part in enumerate(y.split(counts)):
            outputs[b].append(part.clone())

    for at in range(0, max(len(p) for p in prompts), chunk):
        parts = [p[at:at + chunk] for p in prompts]
        counts = [len(p) for p in parts]
        keep(block(torch.cat(parts), pages.extend(counts)), counts)
    step = None
    for x in steps:
        batch = pages.extend([1] * len(prompts), bound=max_tokens)
        if step is None:
            step = DecodeGraph(block, x, batch) if graph else block
        keep(step(x, batch), [1] * len(prompts))
    return [torch.cat(y) for y in outputs]


def main():
    hidden, lens, count, limit = 5120, (600, 1451, 77), 64, 2048
    block = random_block(hidden, 40, 8, 128, num_pages=3 * limit // 64)
    prompts = [torch.randn(n, hidden, device="cuda").bfloat16() for n in lens]
    steps = torch.randn(count, len(lens), hidden, device="cuda").bfloat16()
    serve(block, prompts, steps[:2], 512, limit)  # loads kernels
    results = {}
    for name, graph in (("step by step", False), ("captured steps", True)):
        torch.cuda.synchronize()
        start = time.perf_counter()
        results[name] = serve(block, prompts, steps, 512, limit, graph)
        torch.cuda.synchronize()
        print(f"{name}: prompts of {lens} tokens and {count} steps in {1e3 * (time.perf_counter() - start):.1f} ms")
    same = all(torch.equal(a, b) for a, b in zip(*results.values()))
    print(f"the same outputs: {same}; out of range: {bool(block.status.item())}")
    return 0 if same and not block.status.item() else 1


if __name__ == "__main__":
    sys.exit(main())
