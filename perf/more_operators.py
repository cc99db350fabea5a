"""Decoding several continuations of one prompt, operator by operator: head norms, rotation and the append to the 4-bit
paged cache in one call, attention of sequences that share a long prefix, beam search's selection, and the reordering of
the cached states after it.

The cache is four tensors. Tokens live in pages; slot s is place s % page_size of page s // page_size:
    k_codes, v_codes    int32 [pages, kv_heads, page_size, head_dim / 8]   eight 4-bit codes a word, lowest bits first
    k_scales, v_scales  bf16  [pages, kv_heads, page_size, head_dim / group, 2]   (scale, bias) of each group of dims
and a value is scale * code + bias.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    append = dict(op="append", q_heads=40, kv_heads=8, head_dim=128, group=64, page=64, rot_dim=128, interleaved=False,
                  dtype="bf16")
    shared = dict(op="shared", q_heads=40, kv_heads=8, head_dim=128, group=64, page=64, ragged=False, dtype="bf16")
    reorder = dict(op="reorder", kv_heads=8, head_dim=128, group=64, page=64, ragged=False)
    return [
        # one step of a few beams at hidden size 5120 (40 heads of 128): only latency counts
        dict(append, name="append_step", tokens=8, span=4096),
        # one step of a large batch, wide heads, a quarter of them rotated in neighbouring pairs
        dict(append, name="append_batch", tokens=500, span=1 << 17, q_heads=16, kv_heads=2, head_dim=256, group=32, page=16,
             rot_dim=64, interleaved=True, dtype="f16"),
        # a long chunk of a prompt
        dict(append, name="append_chunk", tokens=8191, span=32768),
        # four beams right after a prompt of 573 tokens: latency
        dict(shared, name="shared_beams_4", groups=1, beams=4, q=1, prefix=573, own=29),
        # a serving batch: eight prompts of ragged lengths with four beams each
        dict(shared, name="shared_batch", groups=8, beams=4, q=1, prefix=4096, own=200, ragged=True),
        # many samples of one long prompt
        dict(shared, name="shared_samples_64", groups=1, beams=64, q=1, prefix=32768, own=512, ragged=True),
        # ragged new requests that start with one of two system prompts, narrow heads, small pages
        dict(shared, name="shared_chunks", groups=2, beams=6, q=301, prefix=6000, own=301, ragged=True, q_heads=32, head_dim=64,
             group=32, page=16, dtype="f16"),
        # four beams of one prompt, logits in f32: latency
        dict(op="select", name="select_4", groups=1, beams=4, vocab=32000, k=4, finished=False, dtype="f32"),
        # odd sizes, twice as many candidates as beams
        dict(op="select", name="select_odd", groups=13, beams=5, vocab=50001, k=10, finished=False, dtype="bf16"),
        # a large batch over a large vocabulary, some beams at their end
        dict(op="select", name="select_large", groups=32, beams=8, vocab=131072, k=8, finished=True, dtype="bf16"),
        # four beams of one prompt through the layers of a model: latency
        dict(reorder, name="reorder_4", groups=1, beams=4, layers=40, own=41),
        # a batch of prompts with eight beams each
        dict(reorder, name="reorder_batch", groups=16, beams=8, layers=24, own=300, page=32, ragged=True),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "shared", "shared", "select", "reorder"])
    head_dim = rng.choice([64, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if g <= head_dim])
    kv_heads = rng.choice([1, 2, 4, 8])
    share = rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    cache = dict(kv_heads=kv_heads, head_dim=head_dim, group=group, page=page)
    dtype = rng.choice(["bf16", "f16"])
    if op == "append":
        return dict(cache, op=op, tokens=_spread(rng, 1, 4096), q_heads=kv_heads * min(share, 5), rot_dim=head_dim // rng.choice([1, 1, 2, 4]),
                    interleaved=rng.random() < 0.5, span=_spread(rng, 64, 1 << 17), dtype=dtype)
    if op == "select":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
        vocab = _spread(rng, 100, 200000)
        groups = max(1, min(_spread(rng, 1, 64), (1 << 24) // (vocab * beams)))
        return dict(op=op, groups=groups, beams=beams, vocab=vocab, k=rng.choice([beams, 2 * beams]), finished=rng.random() < 0.4,
                    dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "reorder":
        beams = rng.choice([1, 2, 3, 4, 8, 16])
        return dict(cache, op=op, groups=_spread(rng, 1, 48 // beams), beams=beams, layers=_spread(rng, 1, 24), own=_spread(rng, 1, 400),
                    ragged=rng.random() < 0.5)
    if rng.random() < 0.7:   # decoding: one token a sequence, or a few that were guessed ahead
        groups, beams = rng.choice([1, 1, 2, 5, 8]), rng.choice([2, 3, 4, 8, 16, 32])
        q, own_tokens = rng.choice([1, 1, 1, 2, 5]), _spread(rng, 1, 1024)
    else:                    # prefill behind a shared prompt
        groups, beams, q = rng.choice([1, 1, 2, 3]), rng.choice([2, 3, 6]), _spread(rng, 16, 400)
        own_tokens = q + rng.choice([0, _spread(rng, 1, 500)])
    case = dict(cache, op=op, groups=groups, beams=beams, q=q, prefix=_spread(rng, 16, 32768), own=max(q, own_tokens),
                ragged=rng.random() < 0.5, q_heads=kv_heads * share, dtype=dtype)
    while work(case)["flops"] > 3e10:   # no larger than the listed ones
        case["prefix"] = max(1, case["prefix"] // 2)
        case["q"], case["own"] = max(1, case["q"] // 2), max(1, case["own"] // 2)
    return case


def _part(case, i):
    return 1.0 if not case["ragged"] or i == 0 else 0.3 + 0.7 * ((i * 0.6180339887) % 1.0)


def _lengths(case):
    """Prefix tokens of each group, and (query tokens, own tokens) of each sequence; own ones hold the queries'."""
    prefixes = [max(1, int(case["prefix"] * _part(case, g))) for g in range(case["groups"])]
    rows = []
    for i in range(case["groups"] * case["beams"]):
        part = _part(case, i)
        q = max(1, int(case["q"] * part))
        rows.append((q, max(q, int(case["own"] * part))))
    return prefixes, rows


def _own_lens(case):
    """Own tokens of each beam: those of one prompt are of one length, as a search leaves them."""
    return [max(1, int(case["own"] * _part(case, i // case["beams"]))) for i in range(case["groups"] * case["beams"])]


def work(case):
    if case["op"] == "select":
        n = case["groups"] * case["beams"] * case["vocab"]
        return {"bytes": (4 if case["dtype"] == "f32" else 2) * n + 5 * case["groups"] * case["beams"] + 12 * case["groups"] * case["k"],
                "flops": 4 * n}
    d = case["head_dim"]
    stored = case["kv_heads"] * (d // 2 + 4 * d // case["group"])   # bytes of a token's keys, or values
    if case["op"] == "append":
        n = case["tokens"] * d
        # written once, and once more read and returned
        return {"bytes": 4 * n * case["q_heads"] + 4 * n * case["kv_heads"] + 4 * case["tokens"] * stored + 4 * n * case["kv_heads"]
                + 12 * case["tokens"], "flops": 10 * n * (case["q_heads"] + 2 * case["kv_heads"])}
    if case["op"] == "reorder":
        # of a group's beams, all but the parent's first child copy what the last page holds
        moved = sum(n % case["page"] for i, n in enumerate(_own_lens(case)) if i % case["beams"] >= (case["beams"] + 1) // 2)
        rows = case["groups"] * case["beams"]
        pages = -(-case["own"] // case["page"]) + 2
        return {"bytes": 2 * 2 * moved * stored * case["layers"] + 8 * rows * pages + 20 * rows, "flops": 0}
    prefixes, rows = _lengths(case)
    pairs = sum(q * prefixes[i // case["beams"]] + q * n - q * (q - 1) // 2 for i, (q, n) in enumerate(rows))
    tokens = sum(prefixes) + sum(n for _, n in rows)
    return {"bytes": 2 * tokens * stored + 4 * sum(q for q, _ in rows) * case["q_heads"] * d,
            "flops": 4 * d * pairs * case["q_heads"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _codes(x, group):
    """(codes as int32 words, (scale, bias) pairs) of x [..., head_dim], in x's precision."""
    g = x.unflatten(-1, (-1, group))
    low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    bias = low.to(torch.bfloat16)
    scale = ((high - low) / 15).to(torch.bfloat16)
    # 64 bits: a value next to the border of two codes must fall on its own side
    step = torch.where(scale == 0, torch.ones_like(scale), scale).double()
    codes = torch.round((g.double() - bias.double()) / step).clamp_(0, 15).mul_(scale != 0).to(torch.int32)
    codes = codes.flatten(-2).unflatten(-1, (-1, 8))
    words = (codes << torch.arange(0, 32, 4, device=x.device, dtype=torch.int32)).sum(-1, dtype=torch.int32)
    return words, torch.cat([scale, bias], -1)


def _values(words, scales):
    """f32 values of code words [..., head_dim / 8] and their (scale, bias) pairs [..., groups, 2]."""
    codes = (words.unsqueeze(-1) >> torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)) & 15
    codes = codes.flatten(-2).unflatten(-1, (scales.shape[-2], -1)).float()
    s, b = scales.float().split(1, -1)
    return (codes * s + b).flatten(-2)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 29)
    return {"append": _inputs_append, "shared": _inputs_shared, "select": _inputs_select, "reorder": _inputs_reorder}[case["op"]](
        case, gen, dev)


def _pool(case, pages, dev):
    shape, d = (pages, case["kv_heads"], case["page"]), case["head_dim"]
    sides = []
    for _ in range(2):
        sides += [torch.zeros(shape + (d // 8,), dtype=torch.int32, device=dev),
                  torch.zeros(shape + (d // case["group"], 2), dtype=torch.bfloat16, device=dev)]
    return sides


def _filled_pool(case, pages, gen, dev):
    cache, d = _pool(case, pages, dev), case["head_dim"]
    each = max(1, (1 << 26) // (case["kv_heads"] * case["page"] * d))   # a bounded part of the pool at a time
    for side in (0, 2):
        for a in range(0, pages, each):
            b = min(pages, a + each)
            x = torch.randn((b - a, case["kv_heads"], case["page"], d), generator=gen, device=dev)
            x[..., ::16] *= 3   # some dims of keys and values are larger than the rest
            cache[side][a:b], cache[side + 1][a:b] = _codes(x, case["group"])
    return cache


def _inputs_append(case, gen, dev):
    # the projections' output holds queries, keys and values of a token side by side
    tokens, hq, hk, d, page = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    dtype = DTYPES[case["dtype"]]
    qkv = torch.randn((tokens, hq + 2 * hk, d), generator=gen, device=dev)
    qkv[..., ::16] *= 4
    qkv = qkv.to(dtype)
    half = case["rot_dim"] // 2
    freq = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
    pos = torch.randint(0, case["span"], (tokens,), generator=gen, device=dev).to(torch.int32)
    pages = -(-tokens // page) * 2 + 2
    slots = torch.randperm(pages * page, generator=gen, device=dev)[:tokens].contiguous()
    weights = [(1 + 0.2 * torch.randn(d, generator=gen, device=dev)).to(dtype) for _ in range(2)]
    return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], q_weight=weights[0], k_weight=weights[1],
                positions=pos, inv_freq=freq.float(), slots=slots, cache=_pool(case, pages, dev), eps=1e-6,
                interleaved=case["interleaved"])


def _inputs_shared(case, gen, dev):
    prefixes, rows = _lengths(case)
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    need = [-(-n // page) for n in prefixes] + [-(-n // page) for _, n in rows]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    tables = torch.zeros(len(need), max(need), dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = order[at:at + n]
        at += n
    groups = case["groups"]
    cu = [0]
    for q, _ in rows:
        cu.append(cu[-1] + q)
    qkv = torch.randn((cu[-1], case["q_heads"] + 2 * hk, d), generator=gen, device=dev).to(DTYPES[case["dtype"]])
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    cu_groups = list(range(0, len(rows) + 1, case["beams"]))
    seq = torch.repeat_interleave(torch.arange(len(rows)), torch.tensor([q for q, _ in rows]))
    place = torch.arange(cu[-1]) - torch.tensor(cu)[seq]
    return dict(case=case, q=qkv[:, :case["q_heads"]], cache=_filled_pool(case, pages, gen, dev),
                prefix_table=tables[:groups, :max(need[:groups])].contiguous(), prefix_lens=ints(prefixes),
                cu_groups=ints(cu_groups), page_table=tables[groups:, :max(need[groups:])].contiguous(),
                kv_lens=ints([n for _, n in rows]), cu_q=ints(cu), max_q=max(q for q, _ in rows), max_kv=max(n for _, n in rows),
                max_prefix=max(prefixes), max_group_q=max(cu[b] - cu[a] for a, b in zip(cu_groups, cu_groups[1:])),
                scale=1.0 / math.sqrt(d),
                # where each query token stands: its sequence and its place among that sequence's queries
                seq=seq.to(dev), place=place.to(dev))


def _inputs_select(case, gen, dev):
    rows, vocab = case["groups"] * case["beams"], case["vocab"]
    x = 2.5 * torch.randn((rows, vocab), generator=gen, device=dev)
    for _ in range(4):   # a few likely tokens
        at = torch.randint(0, vocab, (rows, 1), generator=gen, device=dev)
        x.scatter_add_(1, at, 4 + 4 * torch.rand((rows, 1), generator=gen, device=dev))
    x[:, torch.randint(0, vocab, (max(1, vocab // 1000),), generator=gen, device=dev)] = -math.inf   # forbidden ones
    scores = -8 * torch.rand(rows, generator=gen, device=dev) - 0.5
    finished = torch.rand(rows, generator=gen, device=dev) < 0.2 if case["finished"] else None
    return dict(case=case, logits=x.to(DTYPES[case["dtype"]]), scores=scores, finished=finished, end_token=vocab // 3)


def _inputs_reorder(case, gen, dev):
    groups, beams, page, layers, d = case["groups"], case["beams"], case["page"], case["layers"], case["head_dim"]
    lens = _own_lens(case)
    width = -(-case["own"] // page) + 1
    each = beams * (width + 2)     # pages of a group's pool
    first = 3                      # the prompts' pages come first
    # A search's beams: their early pages are shared, the last ones their own.
    table = torch.zeros(groups * beams, width, dtype=torch.int32, device=dev)
    order = torch.stack([torch.randperm(each, generator=gen, device=dev) for _ in range(groups)]).to(torch.int32)
    for i in range(groups * beams):
        g, n = i // beams, -(-lens[i] // page)
        old = max(0, n - 2)
        take = order[g] + (first + g * each)
        table[i, :old] = take[:old]
        table[i, old:n] = take[width + 2 * (i % beams):][:n - old]
    # the better half of the beams goes on, the best ones twice
    parents = (torch.arange(beams, device=dev) % ((beams + 1) // 2)).repeat(groups, 1)
    shuffle = torch.rand((groups, beams), generator=gen, device=dev).argsort(1)
    parents = shuffle.gather(1, parents).to(torch.int32)
    pages = first + groups * each
    shape = (layers, pages, case["kv_heads"], page)
    cache = []
    for _ in range(2):
        cache += [torch.randint(-(1 << 31), 1 << 31, shape + (d // 8,), generator=gen, device=dev, dtype=torch.int32),
                  torch.randint(1, 200, shape + (d // case["group"], 2), generator=gen, device=dev, dtype=torch.int16).to(torch.bfloat16)]
    return dict(case=case, cache=cache, page_table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev), parents=parents,
                first_page=first, pages_per_group=each)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"append": _plain_append, "shared": _plain_shared, "select": _plain_select, "reorder": _plain_reorder}[op](state)
    import bit_matmul_amd as bm
    if op == "select":
        scores, parents, tokens, finished = bm.beam_select(state["logits"], state["scores"], state["case"]["k"],
                                                           beams=state["case"]["beams"], finished=state["finished"],
                                                           end_token=state["end_token"])
        return {"scores": scores, "parents": parents, "tokens": tokens, "finished": finished}
    if op == "reorder":
        if "handle" not in state:   # a program makes the handles of its layers' caches once
            state["handle"] = bm.KVLayers([bm.KVCache(*(t[i] for t in state["cache"])) for i in range(state["case"]["layers"])])
        table, lens, slots = bm.kv_beam_reorder(state["handle"], state["page_table"], state["lens"], state["parents"],
                                                first_page=state["first_page"], pages_per_group=state["pages_per_group"])
        return {"table": table, "lens": lens, "slots": slots, "cache": state["cache"]}
    if "handle" not in state:
        state["handle"] = bm.KVCache(*state["cache"])
    if op == "append":
        q = bm.qk_norm_rope_append(state["q"], state["k"], state["v"], state["q_weight"], state["k_weight"], state["positions"],
                                   state["inv_freq"], state["slots"], state["handle"], interleaved=state["interleaved"],
                                   eps=state["eps"])
        k, v = bm.kv_read(state["handle"], state["slots"], dtype=state["k"].dtype)
        return {"q": q, "k": k, "v": v}
    return {"out": bm.kv_attention_shared(state["q"], state["handle"], state["prefix_table"], state["prefix_lens"],
                                          state["cu_groups"], state["page_table"], state["kv_lens"], state["cu_q"],
                                          max_group_q=state["max_group_q"], max_prefix=state["max_prefix"], max_q=state["max_q"],
                                          max_kv=state["max_kv"], scale=state["scale"])}


def _plain_append(state):
    case, cache, half = state["case"], state["cache"], state["inv_freq"].numel()
    # 64 bits: at far positions a 32-bit angle has lost the fraction of its last turn
    angle = state["positions"].double()[:, None] * state["inv_freq"].double()

    def turned(x, weight):   # in x's precision
        cos, sin = (t.to(x.dtype)[:, None] for t in (angle.cos(), angle.sin()))
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + state["eps"]) * weight.to(x.dtype)
        first, rest = x[..., :2 * half], x[..., 2 * half:]
        if state["interleaved"]:
            a, b = first[..., 0::2], first[..., 1::2]
            first = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = first[..., :half], first[..., half:]
            first = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([first, rest], -1)

    dtype = state["q"].dtype
    at, off = state["slots"] // case["page"], state["slots"] % case["page"]
    # 64 bits: keys next to the border of two codes, values whose scale lies next to that of two 16-bit numbers
    cache[0][at, :, off], cache[1][at, :, off] = _codes(turned(state["k"].double(), state["k_weight"]), case["group"])
    cache[2][at, :, off], cache[3][at, :, off] = _codes(state["v"].double(), case["group"])
    return {"q": turned(state["q"].float(), state["q_weight"]).to(dtype),
            "k": _values(cache[0][at, :, off], cache[1][at, :, off]).to(dtype),
            "v": _values(cache[2][at, :, off], cache[3][at, :, off]).to(dtype)}


def _plain_shared(state):
    case, cache, q = state["case"], state["cache"], state["q"]
    dev, page, hk, d = q.device, case["page"], case["kv_heads"], case["head_dim"]
    groups, beams, max_q = case["groups"], case["beams"], state["max_q"]

    def sides(table, longest):   # [rows of the table, kv_heads, longest, head_dim] of keys and of values
        token = torch.arange(longest, device=dev)
        at, off = table[:, token // page].long(), token % page
        return [_values(cache[i][at, :, off], cache[i + 1][at, :, off]).transpose(1, 2) for i in (0, 2)]

    cu = state["cu_q"].long()
    count, lens = cu[1:] - cu[:-1], state["kv_lens"].long()
    place = torch.arange(max_q, device=dev)
    rows = (cu[:-1, None] + place).clamp(max=q.shape[0] - 1)
    x = q[rows].float().unflatten(2, (hk, -1)).permute(0, 2, 3, 1, 4)            # [sequences, kv_heads, share, max_q, head_dim]
    share = x.shape[2]
    by_seq = x.flatten(2, 3)                                                     # [sequences, kv_heads, share * max_q, head_dim]
    by_group = by_seq.unflatten(0, (groups, beams)).transpose(1, 2).flatten(2, 3)   # the prefix is read once for its group

    k, v = sides(state["prefix_table"], state["max_prefix"])
    first = torch.matmul(by_group, k.transpose(-1, -2)) * state["scale"]
    token = torch.arange(state["max_prefix"], device=dev)
    first.masked_fill_((token >= state["prefix_lens"].long()[:, None])[:, None, None], -math.inf)
    k2, v2 = sides(state["page_table"], state["max_kv"])
    second = torch.matmul(by_seq, k2.transpose(-1, -2)) * state["scale"]
    pos = (lens - count)[:, None] + place                                        # [sequences, max_q]
    token = torch.arange(state["max_kv"], device=dev)
    seen = (token <= pos[..., None]) & (token < lens[:, None, None])
    second = second.unflatten(2, (share, max_q)).masked_fill_(~seen[:, None, None], -math.inf).flatten(2, 3)

    def per_seq(t):   # the group's rows as the sequences'
        return t.unflatten(2, (beams, -1)).transpose(1, 2).flatten(0, 1)

    def per_group(t):
        return t.unflatten(0, (groups, beams)).transpose(1, 2).flatten(2, 3)

    top = torch.maximum(per_seq(first.amax(-1, keepdim=True)), second.amax(-1, keepdim=True))
    first = (first - per_group(top)).exp_()
    second = (second - top).exp_()
    total = per_seq(first.sum(-1, keepdim=True)) + second.sum(-1, keepdim=True)
    out = (per_seq(torch.matmul(first, v)) + torch.matmul(second, v2)) / total
    out = out.unflatten(2, (share, max_q)).permute(0, 3, 1, 2, 4).flatten(2, 3)
    return {"out": out[state["seq"], state["place"]].to(q.dtype)}


def _plain_select(state):
    case = state["case"]
    groups, beams, vocab, k = case["groups"], case["beams"], case["vocab"], case["k"]
    # 64 bits: candidates of two beams that are next to each other
    x = state["logits"].double()
    top = x.amax(-1, keepdim=True)
    log_sum = top + (x - top).exp_().sum(-1, keepdim=True).log_()
    total = x.sub_(log_sum).add_(state["scores"].double()[:, None])
    if state["finished"] is not None:   # these go on with their end alone
        done = state["finished"][:, None]
        only = torch.where(torch.arange(vocab, device=x.device) == state["end_token"], state["scores"].double()[:, None], -math.inf)
        total = torch.where(done, only, total)
    total = total.view(groups, beams * vocab)
    best = torch.sort(total, dim=-1, descending=True, stable=True)
    score, at = best.values[:, :k], best.indices[:, :k]
    parents, tokens = at // vocab, at % vocab
    ended = tokens == state["end_token"]
    if state["finished"] is not None:
        ended |= state["finished"].view(groups, beams).gather(1, parents)
    none = score == -math.inf   # fewer candidates than places
    return {"scores": score.float(), "parents": parents.masked_fill(none, -1).to(torch.int32),
            "tokens": tokens.masked_fill(none, -1).to(torch.int32), "finished": ended.masked_fill(none, False)}


def _plain_reorder(state):
    case, cache, page = state["case"], state["cache"], state["case"]["page"]
    groups, beams, each, first = case["groups"], case["beams"], state["pages_per_group"], state["first_page"]
    table = state["page_table"].view(groups, beams, -1).long()
    parents = state["parents"].long()
    dev, width = table.device, table.shape[2]
    lens = state["lens"].view(groups, beams).long().gather(1, parents)
    column = torch.arange(width, device=dev)
    held = column < ((lens + page - 1) // page)[..., None]
    new = torch.where(held, table.gather(1, parents[..., None].expand(-1, -1, width)), table)
    # the lowest pages of the group's pool that no row holds
    base = first + each * torch.arange(groups, device=dev)[:, None]
    taken = torch.zeros(groups, each + 1, dtype=torch.int64, device=dev)
    taken.scatter_(1, torch.where(held.flatten(1), new.flatten(1) - base, each), 1)
    free = torch.sort(taken[:, :each], dim=1, stable=True).indices
    earlier = torch.tril(torch.ones(beams, beams, dtype=torch.bool, device=dev), -1)
    again = ((parents[:, :, None] == parents[:, None, :]) & earlier).any(-1)   # another child keeps the parent's page
    part = lens % page
    fresh = (part == 0) | again
    page_of = base + free.gather(1, (fresh.long().cumsum(1) - 1).clamp(min=0))
    last = (lens // page)[..., None]
    was = new.gather(2, last)
    new = new.scatter(2, last, torch.where(fresh[..., None], page_of[..., None], was))
    copied = fresh & (part > 0)
    src, dst = was[..., 0][copied], page_of[copied]
    live = torch.arange(page, device=dev) < part[copied][:, None]
    for t in cache:
        mask = live.view(1, src.numel(), 1, page, *[1] * (t.dim() - 4))
        t[:, dst] = torch.where(mask, t[:, src], t[:, dst])
    slots = new.gather(2, last)[..., 0] * page + part
    return {"table": new.flatten(0, 1).to(torch.int32), "lens": (lens + 1).flatten().to(torch.int32), "slots": slots.flatten(),
            "cache": cache}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "reorder":
        return None   # nothing is computed: whole numbers are moved
    state = prepare(case, seed)
    return {"append": _exact_append, "shared": _exact_shared, "select": _exact_select}[case["op"]](state)


def _exact_append(state):
    n, group = state["inv_freq"].numel(), state["case"]["group"]
    turn = torch.polar(torch.ones((state["positions"].numel(), n), dtype=torch.float64, device="cuda"),
                       torch.outer(state["positions"].double(), state["inv_freq"].double()))
    out = {}
    for name in ("q", "k"):
        x = state[name].double()
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + state["eps"]) * state[name + "_weight"].double()
        first = torch.arange(n, device=x.device) * (2 if state["interleaved"] else 1)
        second = first + (1 if state["interleaved"] else n)
        z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        x[..., first], x[..., second] = z.real, z.imag
        out[name] = x
    for name, x in (("k", out["k"]), ("v", state["v"].double())):
        g = x.reshape(x.shape[:-1] + (-1, group))
        least = g.min(-1, keepdim=True).values
        scale = ((g.max(-1, keepdim=True).values - least) / 15).bfloat16().double()
        bias = least.bfloat16().double()
        level = torch.where(scale > 0, (g - bias) / scale, torch.zeros_like(g)).round().clamp(0, 15)
        out[name] = (scale * level + bias).reshape(x.shape)
    return out


def _exact_shared(state):
    case, cache = state["case"], state["cache"]
    page, d, hk = case["page"], case["head_dim"], case["kv_heads"]
    share = case["q_heads"] // hk
    prefixes, rows = _lengths(case)
    shifts = 4 * torch.arange(8, device="cuda")

    def held(row, tokens, h):
        pages = row[:-(-tokens // page)].long()
        sides = []
        for side in (0, 2):
            words, pair = cache[side][pages, h].reshape(-1, d // 8)[:tokens], cache[side + 1][pages, h].double()
            pair = pair.reshape(-1, d // case["group"], 2)[:tokens]
            level = torch.bitwise_and(words[..., None].long() >> shifts, 15).double().reshape(tokens, -1, case["group"])
            sides.append((level * pair[..., :1] + pair[..., 1:]).reshape(tokens, d))
        return sides

    out = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    for h in range(hk):
        start = 0
        for g, n_prefix in enumerate(prefixes):
            shared = held(state["prefix_table"][g], n_prefix, h)
            for b in range(g * case["beams"], (g + 1) * case["beams"]):
                nq, n = rows[b]
                mine = held(state["page_table"][b], n, h)
                keys, values = (torch.cat(p) for p in zip(shared, mine))
                hidden = torch.arange(n_prefix + n, device="cuda")[None] > torch.arange(n - nq, n, device="cuda")[:, None] + n_prefix
                x = state["q"][start:start + nq, h * share:(h + 1) * share].double().transpose(0, 1)
                s = (torch.matmul(x, keys.T) * state["scale"]).masked_fill(hidden, -math.inf)
                out[start:start + nq, h * share:(h + 1) * share] = torch.matmul(torch.softmax(s, -1), values).transpose(0, 1)
                start += nq
    return {"out": out}


def _exact_select(state):
    case = state["case"]
    beams, vocab, k = case["beams"], case["vocab"], case["k"]
    scores, parents, tokens, ended = [], [], [], []
    for g in range(case["groups"]):
        part = slice(g * beams, (g + 1) * beams)
        total = torch.log_softmax(state["logits"][part].double(), -1) + state["scores"][part].double()[:, None]
        done = state["finished"][part] if state["finished"] is not None else torch.zeros(beams, dtype=torch.bool, device="cuda")
        for b in done.nonzero().flatten().tolist():
            total[b] = -math.inf
            total[b, state["end_token"]] = state["scores"][part][b].double()
        # each beam's best ones are enough
        few = min(k, vocab)
        value, token = torch.sort(total, dim=-1, descending=True, stable=True)
        value, token = value[:, :few].flatten(), token[:, :few].flatten()
        order = torch.sort(value, descending=True, stable=True).indices[:k]
        value, token, beam = value[order], token[order], order // few
        none = value == -math.inf
        end = (token == state["end_token"]) | done[beam]
        scores.append(value)
        parents.append(torch.where(none, -1, beam))
        tokens.append(torch.where(none, -1, token))
        ended.append(end & ~none)
    return {"scores": torch.stack(scores), "parents": torch.stack(parents).int(), "tokens": torch.stack(tokens).int(),
            "finished": torch.stack(ended)}
