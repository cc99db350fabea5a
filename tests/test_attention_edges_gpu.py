"""The attention block where it can go wrong: tiny groups, other streams, wide windows, evicted pages,
tokens of extreme size beside the ones a row sees, weight that sits on one token, and each token of long
contexts counted. Against 64 bits; tests/attn_util.py derives the tolerances that are not derived here."""

import math

import pytest
import torch

import bit_matmul_amd as bm
from tests import attn_exact as X
from tests import attn_util as U
from tests import test_attention_gpu as T
from tests.test_attention_gpu import BF16, F16, F32, dev, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("spread", [1e-35, 1e-37, 3e-38, 1e-38, 1e-39, 2e-40])
@pytest.mark.parametrize("group", [32, 64])
def test_append_of_tiny_groups(spread, group):
    """Groups whose scale is at the end of the f32 range or below its normal numbers."""
    g = torch.Generator().manual_seed(group)
    k, v = (spread * (2 * torch.rand(9, 2, 64, generator=g, dtype=torch.float64) - 1) for _ in range(2))
    k, v = k.to(BF16), v.to(BF16)
    cache = bm.KVCache.empty(1, 16, 2, 64, group)
    bm.bitmm_kv_append(dev(k), dev(v), torch.arange(9, device="cuda:0"), cache)
    for x, codes, scales in ((k, cache.k_codes, cache.k_scales), (v, cache.v_codes, cache.v_scales)):
        c, s, b = U.quantise(x, group)
        if spread >= 1e-39:  # below, scales round to 0
            assert (s > 0).all() and c.unique().numel() == 16
        pairs = scales.cpu()[0, :, :9].transpose(0, 1).double()
        assert torch.equal(pairs[..., 0], s) and torch.equal(pairs[..., 1], b)
        assert torch.equal(codes.cpu()[0, :, :9].transpose(0, 1), U.pack(c))


# ---------------------------------------------------------------------------
# streams
# ---------------------------------------------------------------------------

def test_memory_of_a_call_on_another_stream(monkeypatch):
    """What a form allocates for a call on `stream` is not handed to the current stream when it is dropped
    (the call may still be at work on it), nor taken from what the current stream has dropped."""
    seq = U.Sequences([(1, 9000), (1, 4001)], q_heads=8, kv_heads=2, head_dim=128, group=64, page=64, dtype=BF16)
    cache = seq.cache("cuda:0")
    t = [dev(x) for x in (seq.q, seq.table, seq.kv_lens, seq.cu)]
    at = []
    inner = bm.attention.bitmm_kv_attention

    def noting(*args, **kw):
        at.append(args[6].data_ptr())
        return inner(*args, **kw)

    monkeypatch.setattr(bm.attention, "bitmm_kv_attention", noting)
    need = bm.bitmm_kv_attention_workspace_bytes(2, 2, 1, 9000, 8, 2, 128)
    assert need > 0
    good = bm.kv_attention(t[0], cache, t[1], t[2], t[3], max_q=1, max_kv=9000)
    slots = torch.arange(70, device="cuda:0")
    freq = dev(bm.rope_frequencies(128)[0])
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        at.clear()
        dropped = [torch.empty(need, dtype=torch.uint8, device="cuda:0") for _ in range(4)]
        before = [x.data_ptr() for x in dropped]
        del dropped
        side.wait_stream(torch.cuda.current_stream())
        y = bm.kv_attention(t[0], cache, t[1], t[2], t[3], max_q=1, max_kv=9000, stream=stream)
        after = [torch.empty(need, dtype=torch.uint8, device="cuda:0") for _ in range(4)]
        assert len(at) == 1 and at[0] not in before and at[0] not in [x.data_ptr() for x in after]
        for make in (lambda: bm.kv_attention(t[0], cache, t[1], t[2], t[3], max_q=1, max_kv=9000, stream=stream),
                     lambda: bm.kv_read(cache, slots, stream=stream)[0],
                     lambda: bm.qk_norm_rope(t[0], None, None, None, t[2], freq, stream=stream)[0]):
            x = make()
            shape, dtype, p = x.shape, x.dtype, x.data_ptr()
            del x
            assert p not in [torch.empty(shape, dtype=dtype, device="cuda:0").data_ptr() for _ in range(4)]
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, good)
        side.synchronize()


def test_memory_of_a_product_on_another_stream():
    x = torch.randn(600, 512, device="cuda:0").to(BF16)
    w = torch.randint(-2 ** 31, 2 ** 31, (256, 64), device="cuda:0").to(torch.int32)
    s, b = (torch.rand(256, 8, device="cuda:0").to(BF16) for _ in range(2))
    side = torch.cuda.Stream()
    good = bm.qmm(x, w, s, b, 4)
    side.wait_stream(torch.cuda.current_stream())
    y = bm.qmm(x, w, s, b, 4, stream=side)
    z = bm.qmm(x, w, s, b, 4, stream=side)
    p = z.data_ptr()
    del z
    assert p not in [torch.empty_like(good).data_ptr() for _ in range(4)]
    ids = torch.zeros(600, dtype=torch.int32, device="cuda:0")
    side.wait_stream(torch.cuda.current_stream())
    z, ws = bm.gather_qmm(x, w[None], s[None], b[None], ids, 4, stream=side)
    p, size = ws.data_ptr(), ws.numel()
    del ws
    assert p not in [torch.empty(size, dtype=torch.uint8, device="cuda:0").data_ptr() for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, good) and (z.float() - good.float()).norm() <= 2.0 ** -7 * good.float().norm()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

# The host's bounds of the lengths choose the kernel: these send small sizes through the one for many rows,
# with a row tile's tokens in one piece or split over workgroups.
KERNELS = {"rows": {}, "tiles": dict(max_q=8192, max_kv=2047), "tiles, split": dict(max_q=130, max_kv=65536)}


def bounds(kernel, seq):
    b = KERNELS[kernel]
    return {} if not b else dict(max_q=max(b["max_q"], max(q for q, _ in seq.lens)),
                                 max_kv=max(b["max_kv"], max(kv for _, kv in seq.lens)))


def ran(kernel):
    assert bm.bitmm_last_launches()[0].startswith(f"attention_{kernel.split(',')[0]}_kernel<")


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30])
@pytest.mark.parametrize("sinks", [0, 2 ** 31 - 1])
def test_widest_windows(kernel, window, sinks):
    """More queries than tokens under windows at the end of their range: the queries that see tokens see them all."""
    seq = U.Sequences([(9, 4), (1, 50), (40, 3)], q_heads=4, kv_heads=2, head_dim=64, group=32, page=16, dtype=BF16)
    got = T.check(seq, window=window, sinks=sinks, **bounds(kernel, seq))
    ran(kernel)
    assert (got[:5] == 0).all() and (got[5:9] != 0).any(-1).all()


@pytest.mark.parametrize("kernel", ["rows", "tiles"])
@pytest.mark.parametrize("nq", [1, 3, 70])
@pytest.mark.parametrize("page", [16, 32])
def test_evicted_pages(kernel, nq, page):
    """Pages that no query sees any token of may be gone from the table, wherever the window begins in a step
    or tile of the kernels; one that a query sees a token of is reported, and its tokens are seen by nobody."""
    window, sinks = 100, 5
    word = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    evicted = 0
    for kv in (nq + 150, nq + 187, nq + 222, nq + 255, nq + 300, nq + 333):
        seq = U.Sequences([(nq, kv), (1, 90)], q_heads=2, kv_heads=1, head_dim=64, group=32, page=page, dtype=BF16)
        low = max(0, kv - nq - window + 1)                       # the first token that a query's window holds
        want, _, tol, _ = seq.reference(BF16, 0.125, window, sinks)
        cache, keep = seq.cache("cuda:0"), seq.table.clone()
        for j in range(-(-kv // page)):
            if (j + 1) * page <= low and j * page >= sinks:
                keep[0, j] = (-1, cache.num_pages, 2 ** 31 - 1)[j % 3]
                evicted += 1
        whole, seq.table = seq.table, keep
        word.zero_()
        got, _ = T.attend(seq, cache, BF16, scale=0.125, window=window, sinks=sinks, status=word, **bounds(kernel, seq))
        ran(kernel)
        near(got, want, tol)
        assert word.item() == 0, kv
        for j in {0, low // page, (kv - 1) // page}:             # the pages at each end of what is seen
            seq.table = whole
            want2, _, tol2, _ = seq.reference(BF16, 0.125, window, sinks, hide=lambda b, t: (t // page == j) & (b == 0))
            seq.table = keep.clone()
            seq.table[0, j] = -1
            word.zero_()
            got, _ = T.attend(seq, cache, BF16, scale=0.125, window=window, sinks=sinks, status=word, **bounds(kernel, seq))
            near(got, want2, tol2)
            assert word.item() == 1, (kv, j)
    assert evicted > 10


def one_heavy_token(lens, D, at, bits, seed=1):
    """Keys that are codes and queries of one dim, so that scores are whole numbers of bits: token `at` of each
    sequence scores `bits` more than the others do on the average, and its value is zero; the others' are 1 to 2."""
    seq = U.Sequences(lens, q_heads=4, kv_heads=2, head_dim=D, group=64, page=32, dtype=BF16, seed=seed)
    g = torch.Generator().manual_seed(seed)
    for side, (codes, scale, bias) in enumerate(seq.sides):
        codes = torch.randint(1, 4, codes.shape, generator=g) if side == 0 else codes
        scale, bias = torch.ones_like(scale), torch.zeros_like(bias)
        if side == 1:
            scale, bias = scale / 16, bias + 1
        for b in range(len(lens)):
            page, off = seq.table[b, at // 32].long(), at % 32
            if side == 0:
                codes[page, :, off, 0] = 15
            else:
                scale[page, :, off], bias[page, :, off] = 0, 0
        seq.sides[side] = (codes, scale, bias)
    seq.q = torch.zeros_like(seq.q)
    seq.q[..., 0] = bits / 13          # 15 against 1, 2 or 3
    return seq


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("at", [0, 40])
@pytest.mark.parametrize("bits", [13, 26, 39])
@pytest.mark.parametrize("sinks", [0, 50])
def test_weight_on_one_token(kernel, D, at, bits, sinks):
    """A token that takes all but 2^-3 to 2^-29 of the weight and has nothing to give: the output is what the rest
    add up to, and its probabilities keep their bits.

    Scores are exact. A probability is rounded to 2^-11 of itself, or, where it is small beside the others of
    its step or half tile, to no more than 2^-25 of 2^-9 at least: 2^-11 of the part's weight for 32 of them. Where
    the heavy token is in the part itself, that is 64 * 2^-29 of its weight."""
    window = 200 if sinks else 0
    if window and kernel == "tiles, split":
        pytest.skip("a window is not split")
    seq = one_heavy_token([(3, 573), (40, 900)], D, at, bits)
    got, lse = T.attend(seq, seq.cache("cuda:0"), F32, scale=math.log(2), window=window, sinks=sinks, **bounds(kernel, seq))
    ran(kernel)
    h16, f32 = 2.0 ** -11, 2.0 ** -24
    for b, (nq, kv) in enumerate(seq.lens):
        r = slice(int(seq.cu[b]), int(seq.cu[b + 1]))
        (k, _), (v, vc) = seq.tokens(0, b, kv), seq.tokens(1, b, kv)
        pos, j = torch.arange(kv - nq, kv)[:, None], torch.arange(kv)[None]
        see = (j <= pos) & ((j > pos - window) | (j < sinks)) if window else j <= pos
        for h in range(4):
            x = (seq.q[r, h].double() @ k[:, h // 2].T).masked_fill(~see, -math.inf) * math.log(2)
            p, n = torch.softmax(x, -1), see.sum(-1, keepdim=True)
            off = 4 * f32 * x.masked_fill(~see, 0).abs().amax(-1, keepdim=True)
            rest = p.clone()
            rest[:, at] = 0
            want = p @ v[:, h // 2]
            tol = want * (torch.expm1(2 * off) + h16 + f32 * (n + 64)) + h16 * (p @ (v + vc)[:, h // 2])
            tol += 2 * (h16 * rest.sum(-1, keepdim=True) + 64 * 2.0 ** -29 * p[:, at:at + 1])
            near(got[r, h], want, 1.01 * tol, f"head {h} of sequence {b}")
            total = torch.logsumexp(x, -1)
            near(lse[r, h], total, off[:, 0] + f32 * (n[:, 0] + 64) + 8 * f32 * total.abs(), "lse")


def times(seq, side, tokens, factor):
    """The keys (side 0) or values of those tokens of each sequence times a power of two."""
    _, scale, bias = seq.sides[side]
    for b, (_, kv) in enumerate(seq.lens):
        for t in tokens:
            if t < kv:
                page, off = seq.table[b, t // seq.page].long(), t % seq.page
                scale[page, :, off] *= factor
                bias[page, :, off] *= factor


def compare(seq, kernel, out=F32, only=None, window=0, sinks=0):
    """Rows that `only` (of position and sequence) names, all without it, against 64 bits."""
    scale = 1 / math.sqrt(seq.head_dim)
    want, lse, tol, tol_lse = seq.reference(out, scale, window, sinks)
    got, rows = T.attend(seq, seq.cache("cuda:0"), out, scale=scale, window=window, sinks=sinks, **bounds(kernel, seq))
    ran(kernel)
    keep = torch.ones(len(seq.q), dtype=torch.bool)
    if only is not None:
        for b, (nq, kv) in enumerate(seq.lens):
            keep[int(seq.cu[b]):int(seq.cu[b + 1])] = only(torch.arange(kv - nq, kv))
    assert keep.any()
    near(got[keep], want[keep], tol[keep])
    near(rows[keep], lse[keep], tol_lse[keep], "lse")


EXTREMES = [2.0 ** 40, 2.0 ** 100, 2.0 ** -40, 2.0 ** -100]


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("D, group", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("factor", EXTREMES, ids=str)
def test_extreme_token_after_a_query(kernel, D, group, factor):
    """A row's result does not depend on a token behind it, whatever finite values that has."""
    for first in (0, 150):
        seq = U.Sequences([(45, first + 45), (1, 30)], q_heads=4, kv_heads=2, head_dim=D, group=group, page=16, dtype=BF16, seed=D)
        at = first + 30
        for side in range(2):
            times(seq, side, [at, at + 5], factor)
        compare(seq, kernel, only=lambda pos: pos < at)


@pytest.mark.parametrize("kernel", ["rows", "tiles"])
@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("factor", EXTREMES, ids=str)
def test_extreme_token_before_the_window(kernel, nq, factor):
    seq = U.Sequences([(nq, 400), (nq, 345)], q_heads=4, kv_heads=2, head_dim=128, group=64, page=32, dtype=BF16, seed=nq)
    gone = [0, 1, 5, 283, 284, 230, 231, 232]
    for side in range(2):
        times(seq, side, gone, factor)
    sees = lambda pos: ((torch.tensor(gone)[None] > pos[:, None] - 60)).any(-1)  # noqa: E731
    compare(seq, kernel, only=lambda pos: ~sees(pos), window=60)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("lens", [[(1, 700), (1, 40), (2, 3)], [(80, 300), (70, 70)]], ids=str)
@pytest.mark.parametrize("factor", [2.0 ** 20, 2.0 ** 45, 2.0 ** 100, 2.0 ** -20, 2.0 ** -45, 2.0 ** -100], ids=str)
@pytest.mark.parametrize("tokens", ["first", "one", "every other", "later half"])
def test_values_of_many_sizes(kernel, lens, factor, tokens):
    """Values of very different sizes that are seen: each as exact as its own size allows."""
    seq = U.Sequences(lens, q_heads=4, kv_heads=2, head_dim=128, group=64, page=32, dtype=BF16, seed=2)
    times(seq, 1, {"first": range(1), "one": [45], "every other": range(0, 800, 2), "later half": range(150, 800)}[tokens],
          factor)
    compare(seq, kernel)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("lens", [[(1, 700), (1, 40), (2, 3)], [(80, 300), (70, 70)]], ids=str)
@pytest.mark.parametrize("factor", [2.0 ** -12, 2.0 ** -20, 2.0 ** -60, 2.0 ** -100], ids=str)
def test_keys_of_many_sizes(kernel, lens, factor):
    """Small keys among large ones: every other token's, those of the first half, and one alone the larger."""
    for tokens in (range(0, 800, 2), range(0, 150), [t for t in range(800) if t != 45]):
        seq = U.Sequences(lens, q_heads=4, kv_heads=2, head_dim=64, group=64, page=32, dtype=BF16, seed=2)
        times(seq, 0, tokens, factor)
        compare(seq, kernel)


@pytest.mark.parametrize("window, sinks", X.WINDOWS)
@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("name", list(X.CASES))
def test_each_token_counts(name, kernel, window, sinks):
    """tests/attn_exact.py; the rule's own kernel ("rows" stands for it) and the one for many rows."""
    if window and kernel == "tiles, split":
        pytest.skip("a window is not split")
    seq = X.case(name)
    got, lse = T.attend(seq, seq.cache("cuda:0"), F32, window=window, sinks=sinks, **bounds(kernel, seq))
    if kernel != "rows":
        ran(kernel)
    got, lse = got.double().cpu(), lse.double().cpu()
    for b, (nq, kv) in enumerate(seq.lens):
        r = slice(int(seq.cu[b]), int(seq.cu[b + 1]))
        runs, total = seq.counts(b, window, sinks)
        for h in range(seq.q_heads):
            want, want_lse = seq.expected(b, h * seq.kv_heads // seq.q_heads, runs, total)
            assert ((got[r, h] - want).abs() <= X.OUT * want).all(), (b, h)
            seen = total > 0
            assert (lse[r, h][~seen] == -math.inf).all()
            assert ((lse[r, h] - want_lse)[seen].abs() <= X.LSE).all(), (b, h)


@pytest.mark.parametrize("kernel", ["rows", "tiles"])
@pytest.mark.parametrize("D, group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)])
def test_error_of_binary16_results(kernel, D, group):
    """Over all, at most twice what the rounding of the result gives alone. A value has two roundings and its
    probability one, each of which is in the mean, token by token, what the result's is relative to the same sum: three
    and the result's own add up to sqrt(4) of it. Scores add nothing: their roundings have to be far below."""
    seq = U.Sequences([(100, 700)] if kernel == "tiles" else [(4, 700), (1, 550)], q_heads=4, kv_heads=2, head_dim=D, group=group,
                      page=16, dtype=F16, seed=D + group)
    want, _, _, _ = seq.reference(F16, 1 / math.sqrt(D))
    got, _ = T.attend(seq, seq.cache("cuda:0"), F16, scale=1 / math.sqrt(D), **bounds(kernel, seq))
    ran(kernel)
    off = (got.double().cpu() - want).norm()
    assert off <= 2 * (want.to(F16).double() - want).norm(), (off / want.norm()).item()
