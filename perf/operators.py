"""The attention block's operators on their own workloads: head norms with the position rotation, the 4-bit paged
key/value cache (append and read back), and attention over that cache.

The cache is four tensors. Tokens live in pages; slot s is place s % page_size of page s // page_size:
    k_codes, v_codes    int32 [pages, kv_heads, page_size, head_dim / 8]   eight 4-bit codes a word, lowest bits first
    k_scales, v_scales  bf16  [pages, kv_heads, page_size, head_dim / group, 2]   (scale, bias) of each group of dims
and a value is scale * code + bias.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    rope = dict(op="rope", q_heads=40, kv_heads=8, head_dim=128, rot_dim=128, interleaved=False, scaled=True, dtype="bf16")
    append = dict(op="append", kv_heads=8, head_dim=128, group=64, page=64, dtype="bf16")
    attend = dict(op="attend", q_heads=40, kv_heads=8, head_dim=128, group=64, page=64, window=0, sinks=0,
                  ragged=False, dtype="bf16")
    return [
        # one decode step of a few sequences at hidden size 5120 (40 heads of 128): only latency counts
        dict(rope, name="rope_decode", tokens=8, span=131072),
        # a prompt of 600 tokens
        dict(rope, name="rope_prefill_600", tokens=600, span=600),
        # a long chunk far into a context, a quarter of each wide head rotated in neighbouring pairs
        dict(rope, name="rope_long_partial", tokens=8191, span=1 << 20, q_heads=16, kv_heads=2, head_dim=256, rot_dim=64,
             interleaved=True, scaled=False, dtype="f16"),
        # one decode step of 32 sequences: 32 tokens scattered over the pages
        dict(append, name="append_decode", tokens=32),
        # a prefill chunk written and read back
        dict(append, name="append_prefill", tokens=8192),
        # one sequence right after its 573-token prompt: latency
        dict(attend, name="attend_decode_1", batch=1, q=1, kv=573),
        # a serving batch of ragged contexts
        dict(attend, name="attend_decode_32", batch=32, q=1, kv=4096, ragged=True),
        # few sequences with very long contexts: the work has to be split along them
        dict(attend, name="attend_decode_long", batch=4, q=1, kv=131072),
        # wide heads with a sliding window and four first tokens that stay visible, small pages
        dict(attend, name="attend_decode_window", batch=64, q=1, kv=16384, ragged=True, window=4096, sinks=4, q_heads=16,
             kv_heads=2, head_dim=256, group=32, page=16, dtype="f16"),
        # a prompt of 600 tokens
        dict(attend, name="attend_prefill_600", batch=1, q=600, kv=600),
        # ragged chunks of several sequences under a window, narrow heads
        dict(attend, name="attend_prefill_window", batch=6, q=1021, kv=8000, ragged=True, window=1024, sinks=4,
             q_heads=32, head_dim=64, group=32, page=16, dtype="f16"),
        # the last chunk of a long prompt
        dict(attend, name="attend_prefill_long", batch=1, q=4096, kv=16384),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend"])
    head_dim = rng.choice([64, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if g <= head_dim])
    kv_heads = rng.choice([1, 2, 4, 8])
    share = rng.choice([1, 2, 3, 4, 5, 7, 8])
    dtype = rng.choice(["bf16", "f16"])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        return dict(op=op, tokens=_spread(rng, 1, 8192), q_heads=kv_heads * share, kv_heads=kv_heads, head_dim=head_dim,
                    rot_dim=head_dim // rng.choice([1, 1, 2, 4]), interleaved=rng.random() < 0.5, scaled=rng.random() < 0.5,
                    span=_spread(rng, 64, 1 << 20), dtype=dtype)
    if op == "append":
        return dict(op=op, tokens=_spread(rng, 1, 8192), kv_heads=kv_heads, head_dim=head_dim, group=group, page=page,
                    dtype=dtype)
    if rng.random() < 0.5:   # decode: one token a sequence, or a few that were guessed ahead
        q, batch = rng.choice([1, 1, 1, 2, 5]), _spread(rng, 1, 64)
        kv = _spread(rng, 16, min(131072, (1 << 19) // batch))
    else:                    # prefill chunks
        q = _spread(rng, 16, 2048)
        kv = q + rng.choice([0, _spread(rng, 1, 8192)])
        batch = rng.choice([1, 1, 2, 3])
    window = rng.choice([0, 0, _spread(rng, 16, 4096)])
    case = dict(op=op, batch=batch, q=q, kv=kv, ragged=rng.random() < 0.5, q_heads=kv_heads * share, kv_heads=kv_heads,
                head_dim=head_dim, group=group, page=page, window=window, sinks=rng.choice([0, 1, 4]) if window else 0,
                dtype=dtype)
    while work(case)["flops"] > 1e12:   # no larger than the listed ones
        case["q"], case["kv"] = case["q"] // 2, case["kv"] // 2
    return case


def _lengths(case):
    """(query tokens, cached tokens) of each sequence; the cached ones hold the queries' own."""
    out = []
    for i in range(case["batch"]):
        part = 1.0 if not case["ragged"] or i == 0 else 0.25 + 0.75 * ((i * 0.6180339887) % 1.0)
        q = max(1, int(case["q"] * part))
        out.append((q, max(q, int(case["kv"] * part))))
    return out


def _seen(case):
    """(visible query-key pairs, cached tokens that any query sees) over all sequences, for one head."""
    pairs = tokens = 0
    window, sinks = case["window"], case["sinks"]
    for q, kv in _lengths(case):
        first = kv - q
        for p in range(first, kv):
            pairs += p + 1 if not window else min(p + 1, window) + min(sinks, max(0, p + 1 - window))
        low = max(0, first - window + 1) if window else 0
        tokens += kv - low + min(sinks, low)
    return pairs, tokens


def work(case):
    d = case["head_dim"]
    if case["op"] == "rope":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * d
        return {"bytes": 4 * n + 4 * case["tokens"] + 4 * d + 2 * case["rot_dim"], "flops": 8 * n}
    if case["op"] == "append":
        n = 2 * case["tokens"] * case["kv_heads"] * d   # keys and values
        stored = n // 2 + 4 * n // case["group"]
        return {"bytes": 2 * n + stored + stored + 2 * n + 16 * case["tokens"], "flops": 10 * n}
    pairs, tokens = _seen(case)
    rows = sum(q for q, _ in _lengths(case)) * case["q_heads"]
    stored = 2 * tokens * case["kv_heads"] * (d // 2 + 4 * d // case["group"])
    return {"bytes": stored + 4 * rows * d, "flops": 4 * d * pairs * case["q_heads"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _quantise(x, group):
    """(codes as int32 words, (scale, bias) pairs) of x [..., head_dim]."""
    g = x.float().unflatten(-1, (-1, group))
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
    gen.manual_seed(int(seed) * 1000003 + 17)
    dtype = DTYPES[case["dtype"]]
    d = case["head_dim"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if case["op"] == "rope":
        # the projections' output holds queries, keys and values of a token side by side
        tokens, hq, hk = case["tokens"], case["q_heads"], case["kv_heads"]
        qkv = (3 * normal(tokens, hq + 2 * hk, d)).to(dtype)
        half = case["rot_dim"] // 2
        freq = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        if case["scaled"]:   # long contexts: slow rotations at a quarter of their speed, fast ones as they were
            freq = torch.where(freq < 2 * math.pi / 4096, freq / 4, freq)
        if tokens * 2 > case["span"]:
            pos = torch.arange(tokens, device=dev) % case["span"]
        else:
            pos = torch.randint(0, case["span"], (tokens,), generator=gen, device=dev)
        return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hk], q_weight=(1 + 0.2 * normal(d)).to(dtype),
                    k_weight=(1 + 0.2 * normal(d)).to(dtype), positions=pos.to(torch.int32), inv_freq=freq.float(),
                    rope_scale=1.1386 if case["scaled"] else 1.0, eps=1e-6, interleaved=case["interleaved"])

    hk, page = case["kv_heads"], case["page"]

    def pool(pages):
        shape = (pages, hk, page)
        sides = []
        for _ in range(2):
            sides += [torch.zeros(shape + (d // 8,), dtype=torch.int32, device=dev),
                      torch.zeros(shape + (d // case["group"], 2), dtype=torch.bfloat16, device=dev)]
        return sides

    if case["op"] == "append":
        tokens = case["tokens"]
        pages = -(-tokens // page) * 2 + 2
        qkv = normal(tokens, 3 * hk, d)
        qkv[..., ::16] *= 4   # some dims of keys and values are larger than the rest
        qkv = qkv.to(dtype)
        slots = torch.randperm(pages * page, generator=gen, device=dev)[:tokens].contiguous()
        return dict(case=case, k=qkv[:, hk:2 * hk], v=qkv[:, 2 * hk:], slots=slots, cache=pool(pages))

    lengths = _lengths(case)
    need = [-(-kv // page) for _, kv in lengths]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(len(lengths), max(need), dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    cache = pool(pages)
    for side in (0, 2):
        for a in range(0, pages, max(1, (1 << 27) // (hk * page * d))):   # a bounded part of the pool at a time
            b = min(pages, a + max(1, (1 << 27) // (hk * page * d)))
            x = normal(b - a, hk, page, d)
            x[..., ::16] *= 3
            cache[side][a:b], cache[side + 1][a:b] = _quantise(x, case["group"])
    q_lens = [q for q, _ in lengths]
    total = sum(q_lens)
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    qkv = normal(total, case["q_heads"] + 2 * hk, d).to(dtype)
    seq = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(q_lens))
    return dict(case=case, q=qkv[:, :case["q_heads"]], cache=cache, page_table=table,
                kv_lens=torch.tensor([kv for _, kv in lengths], dtype=torch.int32, device=dev),
                cu_q=torch.tensor(cu, dtype=torch.int32, device=dev), max_q=max(q_lens), max_kv=max(kv for _, kv in lengths),
                window=case["window"], sinks=case["sinks"], scale=1.0 / math.sqrt(d),
                # where each query token stands: its sequence and its place among that sequence's queries
                seq=seq.to(dev), place=(torch.arange(total) - torch.tensor(cu)[seq]).to(dev))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[op](state)
    import bit_matmul_amd as bm
    if op == "rope":
        q, k = bm.qk_norm_rope(state["q"], state["k"], state["q_weight"], state["k_weight"], state["positions"],
                               state["inv_freq"], interleaved=state["interleaved"], eps=state["eps"],
                               rope_scale=state["rope_scale"])
        return {"q": q, "k": k}
    if "handle" not in state:   # a program makes the handle of its cache once
        state["handle"] = bm.KVCache(*state["cache"])
    if op == "append":
        bm.bitmm_kv_append(state["k"], state["v"], state["slots"], state["handle"])
        k, v = bm.kv_read(state["handle"], state["slots"], dtype=state["k"].dtype)
        return {"k": k, "v": v}
    return {"out": bm.kv_attention(state["q"], state["handle"], state["page_table"], state["kv_lens"], state["cu_q"],
                                   max_q=state["max_q"], max_kv=state["max_kv"], scale=state["scale"],
                                   window=state["window"], sinks=state["sinks"])}


def _plain_rope(state):
    half = state["inv_freq"].numel()
    # 64 bits: at far positions a 32-bit angle has lost the fraction of its last turn
    angle = state["positions"].double()[:, None] * state["inv_freq"].double()
    cos = (angle.cos() * state["rope_scale"]).float()[:, None]
    sin = (angle.sin() * state["rope_scale"]).float()[:, None]

    def one(x, weight):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + state["eps"]) * weight.float()
        turned, rest = y[..., :2 * half], y[..., 2 * half:]
        if state["interleaved"]:
            a, b = turned[..., 0::2], turned[..., 1::2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = turned[..., :half], turned[..., half:]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([turned, rest], -1).to(x.dtype)

    return {"q": one(state["q"], state["q_weight"]), "k": one(state["k"], state["k_weight"])}


def _plain_append(state):
    cache, group, page = state["cache"], state["case"]["group"], state["case"]["page"]
    at, off = state["slots"] // page, state["slots"] % page
    cache[0][at, :, off], cache[1][at, :, off] = _quantise(state["k"], group)
    cache[2][at, :, off], cache[3][at, :, off] = _quantise(state["v"], group)
    dtype = state["k"].dtype
    return {"k": _values(cache[0][at, :, off], cache[1][at, :, off]).to(dtype),
            "v": _values(cache[2][at, :, off], cache[3][at, :, off]).to(dtype)}


def _plain_attend(state):
    case, cache, q = state["case"], state["cache"], state["q"]
    dev, page, hk, d = q.device, case["page"], case["kv_heads"], case["head_dim"]
    batch, max_q, max_kv = case["batch"], state["max_q"], state["max_kv"]
    token = torch.arange(max_kv, device=dev)
    at, off = state["page_table"][:, token // page].long(), token % page
    k = _values(cache[0][at, :, off], cache[1][at, :, off]).transpose(1, 2)      # [batch, kv_heads, max_kv, head_dim]
    v = _values(cache[2][at, :, off], cache[3][at, :, off]).transpose(1, 2)
    cu = state["cu_q"].long()
    count, lens = cu[1:] - cu[:-1], state["kv_lens"].long()
    place = torch.arange(max_q, device=dev)
    rows = (cu[:-1, None] + place).clamp(max=q.shape[0] - 1)
    x = q[rows].float().unflatten(2, (hk, -1)).permute(0, 2, 3, 1, 4)            # [batch, kv_heads, share, max_q, head_dim]
    scores = torch.matmul(x.flatten(2, 3), k.transpose(-1, -2)) * state["scale"]
    pos = (lens - count)[:, None] + place                                        # [batch, max_q]
    seen = (token <= pos[..., None]) & (token < lens[:, None, None])
    if state["window"]:
        seen &= (token > pos[..., None] - state["window"]) | (token < state["sinks"])
    scores = scores.unflatten(2, (-1, max_q)).masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_(min=-3e38)                        # finite where nothing is visible
    p = (scores - top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), v).unflatten(2, (-1, max_q)) / total.clamp_(min=1e-37)
    return {"out": out.permute(0, 3, 1, 2, 4).flatten(2, 3)[state["seq"], state["place"]].to(q.dtype)}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend}[case["op"]](state)


def _exact_rope(state):
    n = state["inv_freq"].numel()
    turn = torch.polar(torch.full((state["positions"].numel(), n), state["rope_scale"], dtype=torch.float64, device="cuda"),
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
    return out


def _exact_append(state):
    out = {}
    for name in ("k", "v"):
        x = state[name].double()
        g = x.reshape(x.shape[:-1] + (-1, state["case"]["group"]))
        least = g.min(-1, keepdim=True).values
        scale = ((g.max(-1, keepdim=True).values - least) / 15).bfloat16().double()
        bias = least.bfloat16().double()
        level = torch.where(scale > 0, (g - bias) / scale, torch.zeros_like(g)).round().clamp(0, 15)
        out[name] = (scale * level + bias).reshape(x.shape)
    return out


def _exact_attend(state):
    case, cache = state["case"], state["cache"]
    hk, page, d = case["kv_heads"], case["page"], case["head_dim"]
    share = case["q_heads"] // hk
    shifts = 4 * torch.arange(8, device="cuda")
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    start = 0
    for i, (nq, kv) in enumerate(_lengths(case)):
        pages = state["page_table"][i, :-(-kv // page)].long()
        where = torch.arange(kv - nq, kv, device="cuda")[:, None]
        key = torch.arange(kv, device="cuda")[None]
        hidden = key > where
        if case["window"]:
            hidden = hidden | ((where - key >= case["window"]) & (key >= case["sinks"]))
        for h in range(hk):
            sides = []
            for side in (0, 2):
                words, pair = cache[side][pages, h].reshape(-1, d // 8)[:kv], cache[side + 1][pages, h].double()
                pair = pair.reshape(-1, d // case["group"], 2)[:kv]
                level = torch.bitwise_and(words[..., None].long() >> shifts, 15).double().reshape(kv, -1, case["group"])
                sides.append((level * pair[..., :1] + pair[..., 1:]).reshape(kv, d))
            for j in range(share):
                head = h * share + j
                x = state["q"][start:start + nq, head].double() @ sides[0].T * state["scale"]
                out[start:start + nq, head] = torch.softmax(x.masked_fill_(hidden, -math.inf), -1) @ sides[1]
        start += nq
    return {"out": out}
