"""The attention block's operators in 64 bits, on the CPU, and how far binary16 operands, one
rounding of the result and 32-bit sums may be from them."""

import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def quantise(x, group):
    """(codes int64 [..., D], scale, bias f64 [..., D / group]) as the cache stores x."""
    g = x.float().unflatten(-1, (-1, group))
    low, high = g.amin(-1), g.amax(-1)
    scale = ((high - low) / 15).to(torch.bfloat16)
    bias = low.to(torch.bfloat16)
    s = scale.double().unsqueeze(-1)
    codes = torch.round((g.double() - bias.double().unsqueeze(-1)) / torch.where(s > 0, s, torch.ones_like(s)))
    codes = codes.clamp(0, 15) * (s > 0)
    return codes.flatten(-2).long(), scale.double(), bias.double()


def pack(codes):
    """int32 words of codes [..., D]: eight a word, lowest bits first."""
    w = (codes.unflatten(-1, (-1, 8)) << torch.arange(0, 32, 4)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def values(codes, scale, bias):
    group = codes.shape[-1] // scale.shape[-1]
    s, b = scale.repeat_interleave(group, -1), bias.repeat_interleave(group, -1)
    return s * codes + b


def centre(scale, bias, group):
    """|bias + 8 scale| of each dim: what enters a value's second rounding."""
    return (bias + 8 * scale).abs().repeat_interleave(group, -1)


class Sequences:
    """Random sequences in a cache of scattered pages. lens: (queries, tokens) of each."""

    def __init__(self, lens, *, q_heads, kv_heads, head_dim, group, page, dtype, seed=0, spare=2, kv_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.group, self.dtype = lens, page, group, dtype
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        need = [-(-kv // page) for _, kv in lens]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).to(torch.int32)
        self.table = torch.zeros(len(lens), max(need + [1]), dtype=torch.int32)
        self.spare = order[sum(need):]
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (pages, kv_heads, page, head_dim)
        self.sides = []
        for _ in range(2):
            x = torch.randn(shape, generator=g)
            x[..., ::16] *= 3
            self.sides.append(quantise((x * kv_scale).to(torch.bfloat16), group))
        total = sum(q for q, _ in lens)
        self.q = (1.5 * torch.randn(total, q_heads, head_dim, generator=g)).to(dtype)
        self.cu = torch.tensor([0] + [sum(q for q, _ in lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)
        self.kv_lens = torch.tensor([kv for _, kv in lens], dtype=torch.int32)

    def cache(self, device):
        import bit_matmul_amd as bm
        t = []
        for codes, scale, bias in self.sides:
            t += [pack(codes).to(device), torch.stack([scale, bias], -1).to(torch.bfloat16).to(device)]
        return bm.KVCache(*t)

    def tokens(self, side, b, kv):
        """(values, |centres|) f64 [kv, kv_heads, head_dim] of sequence b."""
        codes, scale, bias = self.sides[side]
        j = torch.arange(kv)
        page, off = self.table[b].long()[j // self.page], j % self.page
        return (values(codes[page, :, off], scale[page, :, off], bias[page, :, off]),
                centre(scale[page, :, off], bias[page, :, off], self.group))

    def reference(self, out_dtype, scale, window=0, sinks=0, hide=None):
        """(out, lse, tolerance of out, of lse) in f64. hide(b, tokens): tokens nobody sees."""
        share = self.q_heads // self.kv_heads
        out = torch.zeros(self.q.shape, dtype=torch.float64)
        lse = torch.full(self.q.shape[:2], -math.inf, dtype=torch.float64)
        tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
        h16, f32 = 2.0 ** -11, 2.0 ** -24
        for b, (nq, kv) in enumerate(self.lens):
            if not nq or not kv:
                continue
            r = slice(int(self.cu[b]), int(self.cu[b + 1]))
            (k, kc), (v, vc) = self.tokens(0, b, kv), self.tokens(1, b, kv)
            pos = torch.arange(kv - nq, kv)[:, None]
            j = torch.arange(kv)[None]
            see = j <= pos
            if window:
                see = see & ((j > pos - window) | (j < sinks))
            if hide is not None:
                see = see & ~hide(b, torch.arange(kv))[None]
            for h in range(self.q_heads):
                kh = h // share
                q = self.q[r, h].double()
                x = (q @ k[:, kh].T) * scale
                # keys: the centre and the sum with it are rounded to binary16
                dx = abs(scale) * h16 * (q.abs() @ (k[:, kh].abs() + kc[:, kh]).T)
                # products and sums in f32: one rounding each of up to head_dim + 8 terms
                dx += abs(scale) * f32 * (self.head_dim + 8) * (q.abs() @ k[:, kh].abs().T) + 4 * f32 * x.abs()
                x = x.masked_fill(~see, -math.inf)
                any_seen = see.any(-1)
                lse[r, h] = torch.logsumexp(x, -1)
                p = torch.where(any_seen[:, None], torch.softmax(x, -1), torch.zeros_like(x))
                o = p @ v[:, kh]
                out[r, h] = o
                d = torch.where(see, dx, torch.zeros_like(dx)).amax(-1, keepdim=True)
                size = p @ v[:, kh].abs()
                n = see.sum(-1, keepdim=True)
                e = torch.expm1(2 * d) + h16 + f32 * (n + 64)       # probabilities, and 32-bit sums of n terms
                t = size * e + h16 * (p @ (v[:, kh].abs() + vc[:, kh]))
                t += 2.0 ** -25 * (see.double() @ v[:, kh].abs())   # probabilities below binary16's normal range
                tol[r, h] = 1.01 * t + HALF_STEP[out_dtype] * (o.abs() + t) + (2.0 ** -25 if out_dtype == torch.float16 else 1e-37)
                tol_lse[r, h] = (d[:, 0] + f32 * (n[:, 0] + 64) + 4 * f32 * lse[r, h].abs()).nan_to_num(0, 0, 0)
        return out, lse, tol, tol_lse


def rope_reference(x, weight, positions, inv_freq, *, interleaved, eps, weight_offset=0.0, rope_scale=1.0):
    """(y, tolerance before the last rounding) in f64."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (weight_offset + weight.double())
    n = inv_freq.numel()
    t = torch.outer(positions.double(), inv_freq.double())[:, None]
    c, s = rope_scale * t.cos(), rope_scale * t.sin()
    i = torch.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    y, size = x.clone(), x.abs()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    both = abs(rope_scale) * (size[..., a] + size[..., b])
    size[..., a] = both
    size[..., b] = both
    # sum of squares, root, weight, sine and cosine of an angle rounded to 2^-24 of a turn,
    # products and sum: fewer than 48 half steps of f32
    return y, 48 * 2.0 ** -24 * size
