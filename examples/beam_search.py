"""Beam search over a small model with 4-bit weights and a 4-bit cache:

    head norms, rotation and append in one call        bitmm_qk_norm_rope_append
    attention, the prompt shared by all its beams      bitmm_kv_attention_shared
    the beams' best continuations                      bitmm_beam_select
    their cached states, full pages shared             bitmm_kv_beam_reorder

and the projections of bitmm_qmm between them. Prompts go through the layers once, one after the other; then all
beams of all prompts decode together, a token each a step, the step captured once into a HIP graph.

    python examples/beam_search.py
"""

import math
import os
import sys
import time

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]

import torch

import bit_matmul_amd as bm
from attention_block import random_projection


class Model:
    """Layers of attention with a residual each, between an embedding and a 4-bit projection to the vocabulary."""

    def __init__(self, vocab, hidden, layers, q_heads, kv_heads, head_dim, num_pages, page_size, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.embedding = torch.randn(vocab, hidden, generator=g).bfloat16().to(device)
        self.head = random_projection(vocab, hidden, g, device)
        self.qkv = [random_projection((q_heads + 2 * kv_heads) * head_dim, hidden, g, device) for _ in range(layers)]
        self.out = [random_projection(hidden, q_heads * head_dim, g, device) for _ in range(layers)]
        self.norms = [[(1 + 0.1 * torch.randn(head_dim, generator=g)).bfloat16().to(device) for _ in range(2)] for _ in range(layers)]
        self.inv_freq, _ = bm.rope_frequencies(head_dim, 1e6, device=device)
        self.caches = bm.KVLayers([bm.KVCache.empty(num_pages, page_size, kv_heads, head_dim, device=device) for _ in range(layers)])
        self.status = torch.zeros(1, dtype=torch.int32, device=device)   # set by the library if an index is out of range

    def __call__(self, tokens, positions, slots, attend, last=None):
        """f32 logits of tokens (of those at the rows `last`). attend(q, cache): attention of a layer's queries."""
        x = self.embedding[tokens]
        n, hq, hk = len(x), self.q_heads, self.kv_heads
        for i, cache in enumerate(self.caches.caches):
            heads = bm.qmm(x, *self.qkv[i], 4).view(n, hq + 2 * hk, self.head_dim)
            q = bm.qk_norm_rope_append(heads[:, :hq], heads[:, hq:hq + hk], heads[:, hq + hk:], *self.norms[i], positions, self.inv_freq,
                                       slots, cache, status=self.status)
            x = x + bm.qmm(attend(q, cache).view(n, -1), *self.out[i], 4)
        x = (x if last is None else x[last]).float()
        x = 2.5 * x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)   # logits of a deviation of 2.5 or so
        return bm.qmm(x.bfloat16(), *self.head, 4, out_dtype=torch.float32)


class Search:
    """beams of each of some prompts, `steps` tokens long at most."""

    def __init__(self, model, prompts, beams, steps, end_token=-1):
        device, page, groups = model.embedding.device, model.caches.page_size, len(prompts)
        self.model, self.beams, self.steps, self.end_token, rows = model, beams, steps, end_token, groups * beams
        i32 = dict(dtype=torch.int32, device=device)
        self.lens = [len(p) for p in prompts]
        pages = [-(-n // page) for n in self.lens]
        first = sum(pages)                                   # the prompts' pages come first, then a pool of each group
        self.prefix_table = torch.zeros(groups, max(pages), **i32)
        for g, n in enumerate(pages):
            self.prefix_table[g, :n] = torch.arange(n, **i32) + sum(pages[:g])
        self.prefix_lens = torch.tensor(self.lens, **i32)
        self.cu_groups, self.cu_q = torch.arange(0, rows + 1, beams, **i32), torch.arange(rows + 1, **i32)
        width = -(-steps // page)
        self.first_page, self.pages_per_group = first, beams * width
        if first + groups * self.pages_per_group > model.caches.caches[0].num_pages:
            raise ValueError(f"{first + groups * self.pages_per_group} pages are needed")
        # What a step takes from the one before it. Each is also what the step leaves there.
        self.table, self.held = torch.zeros(rows, width, **i32), torch.zeros(rows, **i32)
        self.parents, self.tokens = torch.zeros(groups, beams, **i32), torch.zeros(groups, beams, **i32)
        self.scores = torch.full((groups, beams), -math.inf, device=device)
        self.finished = torch.zeros(groups, beams, dtype=torch.bool, device=device)
        self.slots = torch.empty(rows, dtype=torch.int64, device=device)
        self.offset = self.prefix_lens.repeat_interleave(beams) - 1
        self.select_ws = torch.empty(bm.bitmm_beam_select_workspace_bytes(groups, beams, model.embedding.shape[0], beams, torch.float32),
                                     dtype=torch.uint8, device=device)
        self.reorder_ws = torch.empty(bm.bitmm_kv_beam_reorder_workspace_bytes(groups, beams), dtype=torch.uint8, device=device)
        self.graph = None
        self.scores[:, 0] = 0                                # the first step goes on from one beam of each prompt
        self.select(torch.cat([self.read(p, g) for g, p in enumerate(prompts)]).repeat_interleave(beams, 0))

    def read(self, prompt, g):
        """A prompt through the layers: the logits of its last token."""
        n, page = len(prompt), self.model.caches.page_size
        table, kv, cu = self.prefix_table[g:g + 1].contiguous(), self.prefix_lens[g:g + 1], torch.tensor([0, n], dtype=torch.int32, device=prompt.device)
        at = torch.arange(n, device=prompt.device)
        return self.model(prompt, at.int(), table[0, at // page].long() * page + at % page,
                          lambda q, cache: bm.kv_attention(q, cache, table, kv, cu, max_q=n, max_kv=n, status=self.model.status),
                          last=slice(n - 1, n))

    def select(self, logits):
        bm.bitmm_beam_select(logits, self.scores.view(-1), self.scores, self.parents, self.tokens, self.select_ws, beams=self.beams,
                             finished=self.finished.view(-1), finished_out=self.finished, end_token=self.end_token, status=self.model.status)

    def step(self):
        """The chosen tokens through the layers, and the choice of the next ones."""
        bm.bitmm_kv_beam_reorder(self.model.caches, self.table, self.held, self.parents, self.table, self.held, self.slots, self.reorder_ws,
                                 first_page=self.first_page, pages_per_group=self.pages_per_group, status=self.model.status)
        attend = lambda q, cache: bm.kv_attention_shared(
            q, cache, self.prefix_table, self.prefix_lens, self.cu_groups, self.table, self.held, self.cu_q, max_group_q=self.beams,
            max_prefix=max(self.lens), max_q=1, max_kv=self.steps, status=self.model.status)
        self.select(self.model(self.tokens.view(-1), self.held + self.offset, self.slots, attend))

    def state(self):
        return [self.table, self.held, self.parents, self.tokens, self.scores, self.finished]

    def capture(self):
        """The step as a graph. What loads at a first call loads in a call before, whose effects are taken back; what that
        writes to the caches is written there again by the step itself."""
        before = [t.clone() for t in self.state()]
        self.step()
        for t, was in zip(self.state(), before):
            t.copy_(was)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.step()

    def run(self, graph=True):
        """(tokens [groups, beams, steps], scores [groups, beams], best first), the steps' choices put together."""
        chosen = [(self.parents.clone(), self.tokens.clone())]
        if graph and self.steps > 1:
            self.capture()
        for _ in range(self.steps - 1):
            self.graph.replay() if graph else self.step()
            chosen.append((self.parents.clone(), self.tokens.clone()))
        at = torch.arange(self.beams, device=self.tokens.device).expand_as(self.tokens)
        tokens = []
        for parents, chosen_tokens in reversed(chosen):
            tokens.append(chosen_tokens.gather(1, at))
            at = parents.gather(1, at).long()
        return torch.stack(tokens[::-1], -1), self.scores.clone()


def main():
    vocab, beams, steps = 32000, 4, 48
    model = Model(vocab, 5120, 4, 40, 8, 128, num_pages=64, page_size=64)
    prompts = [torch.randint(0, vocab, (n,), device="cuda") for n in (573, 77, 1200)]
    results = {}
    for name, graph in (("loading", False), ("step by step", False), ("captured steps", True)):
        search = Search(model, prompts, beams, steps)
        torch.cuda.synchronize()
        start = time.perf_counter()
        results[name] = search.run(graph)
        torch.cuda.synchronize()
        print(f"{name}: {steps} tokens of {beams} beams of {len(prompts)} prompts in {1e3 * (time.perf_counter() - start):.1f} ms")
    same = all(torch.equal(a, b) for a, b in zip(results["step by step"], results["captured steps"]))
    print(f"the same beams: {same}; out of range: {bool(model.status.item())}")
    return 0 if same and not model.status.item() else 1


if __name__ == "__main__":
    sys.exit(main())
