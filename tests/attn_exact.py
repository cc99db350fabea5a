"""Attention whose result can be counted. Queries are zero, so that every token that a row sees has the same weight;
token j's value is 1 in dim j / 32 + 7 head (modulo the dims) and 0 in the others. A row that sees n tokens gives how
many of them fall on each dim, over n, and an lse of log n: a token that is lost, doubled or taken from another
place shows, however long the context.

In f32 all of it is exact up to the last steps: probabilities are a power of two, values 0 and 1 in a unit that is one,
and sums are whole numbers below 2^24 of these. The output is one division and one product away: under 4 half steps.
The lse is ln 2 (m + log2 l), of magnitudes up to 32, where f32's step is 2^-19: two of those."""

import math

import torch

from tests import attn_util as U

STEP = 32          # tokens that share a dim: the least that a kernel goes over at a time
OUT = 4 * 2.0 ** -24
LSE = 2.0 ** -18


class Counted(U.Sequences):
    def __init__(self, lens, *, q_heads, kv_heads, head_dim, group=64, page=64, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.group, self.dtype = lens, page, group, torch.bfloat16
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        need = [-(-kv // page) for _, kv in lens]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g).to(torch.int32)
        self.table = torch.zeros(len(lens), max(need + [1]), dtype=torch.int32)
        shape = (pages, kv_heads, page, head_dim)
        ones = torch.ones(pages, kv_heads, page, head_dim // group)
        keys, values = torch.randint(0, 16, shape, generator=g), torch.full(shape, 9)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
            j = torch.arange(lens[b][1])
            for h in range(kv_heads):
                page_of, off = self.table[b].long()[j // page], j % page
                values[page_of, h, off] = 0
                values[page_of, h, off, (j // STEP + 7 * h) % head_dim] = 1
        self.sides = [(keys, ones, 0 * ones), (values, ones, 0 * ones)]
        self.cu = torch.tensor([0] + [sum(q for q, _ in lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)
        self.kv_lens = torch.tensor([kv for _, kv in lens], dtype=torch.int32)
        self.q = torch.zeros(int(self.cu[-1]), q_heads, head_dim, dtype=torch.bfloat16)

    def counts(self, b, window=0, sinks=0, lost=None):
        """(tokens on each run of STEP [queries, runs], tokens [queries]) that sequence b's queries see, without
        the run `lost`."""
        nq, kv = self.lens[b]
        j = torch.arange(kv)[None]
        pos = torch.arange(kv - nq, kv)[:, None]
        see = j <= pos
        if window:
            see = see & ((j > pos - window) | (j < sinks))
        if lost is not None:
            see = see & (j // STEP != lost)
        runs = torch.nn.functional.pad(see, (0, -kv % STEP)).view(nq, -(-kv // STEP), STEP).sum(-1)
        return runs.double(), see.sum(-1).double()

    def expected(self, b, head, runs, total):
        """(out [queries, dims], lse [queries]) of a kv head."""
        out = torch.zeros(runs.shape[0], self.head_dim, dtype=torch.float64)
        out.index_add_(1, (torch.arange(runs.shape[1]) + 7 * head) % self.head_dim, runs)
        return out / total.clamp(min=1)[:, None], total.log()


# (queries, tokens) of sequences, query heads, kv heads, dims: split over workgroups, shared out by length, many
# rows with their last tiles split, and more sequences than can be shared out
CASES = {
    "split": ([(1, 20000)], 8, 1, 128),
    "split, two": ([(1, 9000), (1, 4001)], 40, 8, 128),
    "guesses": ([(4, 7777)], 4, 2, 256),
    "narrow": ([(1, 30000)], 2, 2, 64),
    "long": ([(1, 131072), (1, 99991)], 4, 1, 64),
    "chunk": ([(300, 900)], 10, 2, 128),
    "chunks": ([(130, 4100), (257, 257)], 3, 1, 64),
    "wide": ([(200, 2000)], 8, 1, 256),
    "chunks, split": ([(70, 2300), (700, 700)], 48, 6, 128),
    "one long": ([(1, 40), (1, 9000), (0, 500), (1, 0), (1, 1), (1, 700)], 8, 1, 128),
    "uneven guesses": ([(2, 5000), (1, 33), (0, 0), (2, 2), (2, 1)], 6, 2, 256),
    "64 of them": ([(1, 17 * i) for i in range(63)] + [(1, 20000)], 3, 3, 64),
    "100 of them": ([(1, 31 * i) for i in range(99)] + [(1, 8000)], 3, 3, 64),
}
WINDOWS = [(0, 0), (1000, 4), (600, 70), (33, 0)]


def case(name):
    lens, hq, hk, D = CASES[name]
    return Counted(lens, q_heads=hq, kv_heads=hk, head_dim=D, seed=len(name))
