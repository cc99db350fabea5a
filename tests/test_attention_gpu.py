"""The attention block on the GPU against the same operators in 64 bits: head norms with the
rotation, the 4-bit cache, attention over it. Tolerances are worst cases of the roundings the
header names (tests/attn_util.py derives them)."""

import math

import pytest
import torch

import bit_matmul_amd as bm
from tests import attn_util as U

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bm.lib()
    yield
    torch.cuda.synchronize()


def dev(t):
    return t.to("cuda:0")


def near(got, want, tol, what=""):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    off = (got - want).abs() - tol
    worst = int(off.argmax())
    assert off.flatten()[worst] <= 0, (
        f"{what}: {got.flatten()[worst].item()} for {want.flatten()[worst].item()}, allowed {tol.flatten()[worst].item()}")


# ---------------------------------------------------------------------------
# norms and rotation
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T, hq, hk, D, rot, il", [
    (1, 1, 1, 64, 64, False), (3, 5, 2, 128, 128, False), (2, 8, 1, 256, 256, True), (7, 40, 8, 128, 128, False),
    (5, 3, 3, 128, 64, True), (4, 9, 2, 256, 64, False), (9, 6, 2, 64, 8, False), (6, 7, 1, 64, 24, True),
    (4, 4, 4, 128, 0, False), (601, 16, 2, 128, 32, False), (2500, 5, 1, 64, 64, True),
])
def test_norm_and_rotation(dtype, T, hq, hk, D, rot, il):
    g = torch.Generator().manual_seed(T + D)
    qkv = (2 * torch.randn(T, hq + 2 * hk, D, generator=g)).to(dtype)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).to(dtype) for _ in range(2))
    pos = torch.randint(-50, 1 << 20, (T,), generator=g, dtype=torch.int32)
    freq, scale = bm.rope_frequencies(rot, factor=8.0, scaling="by_parts", original_context=4096)
    opts = dict(interleaved=il, eps=1e-5, rope_scale=scale)
    gpu = dev(qkv)
    yq, yk = bm.qk_norm_rope(gpu[:, :hq], gpu[:, hq:hq + hk], dev(wq), dev(wk), dev(pos), dev(freq), **opts)
    for name, got, x, w in (("q", yq, q, wq), ("k", yk, k, wk)):
        want, tol = U.rope_reference(x, w, pos, freq, **opts)
        near(got, want, tol + U.HALF_STEP[dtype] * (want.abs() + tol) + 2.0 ** -25, name)


def test_rotation_variants():
    """No weights (rotation alone), one weight, an offset to the weights, one side alone, and in place."""
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn(11, h, 128, generator=g).to(BF16) for h in (6, 2))
    w = (0.2 * torch.randn(128, generator=g)).to(BF16)
    pos = torch.arange(11, dtype=torch.int32)
    freq, _ = bm.rope_frequencies(128)

    def check(got, x, weight, **kw):
        want, tol = U.rope_reference(x, weight, pos, freq, interleaved=False, eps=1e-6, **kw)
        near(got, want, tol + U.HALF_STEP[BF16] * (want.abs() + tol))

    p, f = dev(pos), dev(freq)
    yq, yk = bm.qk_norm_rope(dev(q), dev(k), None, dev(w), p, f, weight_offset=1.0)
    check(yq, q, None)
    check(yk, k, w, weight_offset=1.0)
    yq, none = bm.qk_norm_rope(dev(q), None, dev(w), None, p, f)
    assert none is None
    check(yq, q, w)
    none, yk = bm.qk_norm_rope(None, dev(k), None, None, p, f)
    check(yk, k, None)
    both = dev(torch.cat([q, k], 1))
    a, b = both[:, :6], both[:, 6:]
    bm.bitmm_qk_norm_rope(a, b, dev(w), dev(w), p, f, a, b)
    check(a, q, w)
    check(b, k, w)
    # zero heads stay zero, a NaN or infinity stays in its own head
    bad = q.clone()
    bad[0, 0] = 0
    bad[1, 1, 5], bad[2, 2, 7] = math.nan, math.inf
    y, _ = bm.qk_norm_rope(dev(bad), None, dev(w), None, p, f)
    y = y.float().cpu()
    assert (y[0, 0] == 0).all() and y[1, 1].isnan().all()
    y[1, 1], y[2, 2] = 0, 0
    assert y.isfinite().all()


def test_rotation_of_far_positions():
    """At position 2^31 - 1 an angle is reduced without loss: against 64 bits, at f32 size."""
    q = torch.ones(4, 1, 64, dtype=F16)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 16777217, 123456789], dtype=torch.int32)
    freq, _ = bm.rope_frequencies(64)
    y, _ = bm.qk_norm_rope(dev(q), None, None, None, dev(pos), dev(freq))
    want, tol = U.rope_reference(q, None, pos, freq, interleaved=False, eps=0.0)
    # 64 bits lose 2^-22 radians at 2^31 themselves
    near(y, want, tol + 2.0 ** -20 + U.HALF_STEP[F16] * want.abs())


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T, hk, D, group, page", [
    (1, 1, 64, 32, 16), (3, 2, 64, 64, 32), (70, 8, 128, 64, 64), (17, 3, 128, 32, 16), (33, 1, 128, 128, 128),
    (5, 2, 256, 128, 16), (130, 5, 256, 32, 256), (1000, 4, 128, 64, 16),
])
def test_append_and_read(dtype, T, hk, D, group, page):
    g = torch.Generator().manual_seed(T * D + group)
    kv = torch.randn(T, 2 * hk + 1, D, generator=g)
    kv[..., ::16] *= 6
    kv = kv.to(dtype)
    kv[0, 0, :group] = 1.5                         # a constant group: scale 0
    kv[T // 2, hk, :] = 0                          # zeros
    kv[T - 1, 0, :group] = (torch.arange(group) % 31 * 0.5).to(dtype)   # every border: 0.5, 1.5, ... of scale 1
    k, v = kv[:, :hk], kv[:, hk:2 * hk]
    pages = -(-T // page) + 3
    slots = torch.randperm(pages * page, generator=g)[:T]
    cache = bm.KVCache.empty(pages, page, hk, D, group)
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(-1)
    for t in (cache.k_scales, cache.v_scales):
        t.fill_(7)
    word = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    gpu = dev(kv)
    bm.bitmm_kv_append(gpu[:, :hk], gpu[:, hk:2 * hk], dev(slots), cache, status=word)
    yk, yv = bm.kv_read(cache, dev(slots), dtype=dtype, status=word)
    assert word.item() == 0
    at, off = slots // page, slots % page
    for x, codes, scales, y in ((k, cache.k_codes, cache.k_scales, yk), (v, cache.v_codes, cache.v_scales, yv)):
        c, s, b = U.quantise(x, group)
        assert torch.equal(codes.cpu()[at, :, off], U.pack(c))
        pairs = scales.cpu()[at, :, off].double()
        assert torch.equal(pairs[..., 0], s) and torch.equal(pairs[..., 1], b)
        want = U.values(c, s, b)
        # one f32 and one final rounding
        near(y, want, (U.HALF_STEP[dtype] + 2.0 ** -23) * want.abs() + 2.0 ** -25)
        mask = torch.ones(pages * page, dtype=torch.bool)
        mask[slots] = False                        # nothing else was written
        rest = codes.cpu().transpose(1, 2).reshape(pages * page, -1)[mask]
        assert (rest == -1).all()
        assert (scales.cpu().transpose(1, 2).reshape(pages * page, -1)[mask] == 7).all()


def test_slots_outside_the_cache():
    """-1 is padding; any other slot outside is skipped and reported; reads give zeros."""
    cache = bm.KVCache.empty(2, 16, 2, 64, 32)
    for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales):
        t.fill_(3)
    before = [t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    k = torch.randn(3, 2, 64, device="cuda:0").to(BF16)
    word = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    pad = torch.tensor([-1, -1, -1], device="cuda:0")
    bm.bitmm_kv_append(k, k, pad, cache, status=word)
    y, _ = bm.kv_read(cache, pad, status=word)
    assert word.item() == 0 and (y == 0).all()
    out = torch.tensor([32, -2, 1 << 40], device="cuda:0")
    bm.bitmm_kv_append(k, k, out, cache, status=word)
    assert word.item() == 1
    word.zero_()
    y, z = bm.kv_read(cache, out, dtype=F16, status=word)
    assert word.item() == 1 and (y == 0).all() and (z == 0).all()
    bm.bitmm_kv_append(k, k, out, cache)           # without a status word
    for a, b in zip(before, (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)):
        assert torch.equal(a, b)
    only = torch.empty(1, 2, 64, dtype=BF16, device="cuda:0")
    bm.bitmm_kv_read(cache, out[:1] * 0 + 5, None, only)
    assert (only != 0).all()


def test_append_not_finite():
    cache = bm.KVCache.empty(1, 16, 1, 64, 32)
    k = torch.ones(2, 1, 64, dtype=BF16, device="cuda:0")
    k[0, 0, 3], k[1, 0, 40] = math.inf, math.nan
    bm.bitmm_kv_append(k, k, torch.arange(2, device="cuda:0"), cache)
    y, _ = bm.kv_read(cache, torch.arange(2, device="cuda:0"))
    assert y[0, 0, :32].isnan().all() and (y[0, 0, 32:] == 1).all()
    assert y[1, 0, 32:].isnan().all() and (y[1, 0, :32] == 1).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def attend(seq, cache, out_dtype, *, lse=True, workspace=None, **kw):
    t = {n: dev(x) for n, x in (("q", seq.q), ("table", seq.table), ("lens", seq.kv_lens), ("cu", seq.cu))}
    rows = torch.full(seq.q.shape[:2], 9.0, device="cuda:0") if lse else None
    kw.setdefault("max_q", max(q for q, _ in seq.lens))
    kw.setdefault("max_kv", max(kv for _, kv in seq.lens))
    out = bm.kv_attention(t["q"], cache, t["table"], t["lens"], t["cu"], out_dtype=out_dtype, lse=rows, **kw)
    return out, rows


def check(seq, out_dtype=None, scale=None, window=0, sinks=0, **kw):
    out_dtype = out_dtype or seq.dtype
    scale = 1 / math.sqrt(seq.head_dim) if scale is None else scale
    want, lse, tol, tol_lse = seq.reference(out_dtype, scale, window, sinks, kw.pop("hide", None))
    got, rows = attend(seq, kw.pop("cache", None) or seq.cache("cuda:0"), out_dtype, scale=scale, window=window,
                       sinks=sinks, **kw)
    near(got, want, tol, f"lens {seq.lens}")
    none = lse == -math.inf
    rows = rows.double().cpu()
    assert torch.equal(rows == -math.inf, none)
    if not none.all():
        near(rows[~none], lse[~none], tol_lse[~none], "lse")
    return got


SHAPES = [  # q_heads, kv_heads, head_dim, group, page
    (1, 1, 64, 32, 16), (4, 4, 64, 64, 64), (5, 1, 128, 64, 64), (16, 2, 128, 32, 16), (10, 2, 128, 128, 32),
    (14, 2, 256, 64, 16), (8, 1, 256, 32, 128), (6, 3, 256, 128, 256),
]
LENGTHS = {
    "one token": [(1, 1)],
    "decode": [(1, 31), (1, 32), (1, 33), (1, 700), (1, 2)],
    "prompt": [(37, 37)],
    "guesses": [(5, 300), (2, 17), (0, 40), (3, 3)],
    "chunks": [(70, 515), (1, 129), (40, 40)],
}


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("lens", list(LENGTHS), ids=str)
def test_attention(dtype, shape, lens):
    hq, hk, D, group, page = shape
    seq = U.Sequences(LENGTHS[lens], q_heads=hq, kv_heads=hk, head_dim=D, group=group, page=page, dtype=dtype, seed=D)
    check(seq)


@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (16, 4), (33, 70), (64, 0), (200, 5), (5000, 3)])
@pytest.mark.parametrize("lens", ["decode", "chunks"], ids=str)
def test_window_and_first_tokens(out, window, sinks, lens):
    seq = U.Sequences(LENGTHS[lens], q_heads=6, kv_heads=2, head_dim=128, group=64, page=32, dtype=BF16, seed=window)
    check(seq, out, window=window, sinks=sinks)


@pytest.mark.parametrize("lens, hq, hk, D", [
    ([(1, 20000)], 8, 1, 128), ([(1, 9000), (1, 4001)], 40, 8, 128), ([(4, 7777)], 4, 2, 256), ([(1, 30000)], 2, 2, 64),
    ([(300, 900)], 10, 2, 128), ([(130, 4100), (257, 257)], 3, 1, 64), ([(200, 2000)], 8, 1, 256),
])
def test_long(lens, hq, hk, D):
    """Long enough to be split over workgroups, and many query rows."""
    seq = U.Sequences(lens, q_heads=hq, kv_heads=hk, head_dim=D, group=64, page=64, dtype=BF16, seed=len(lens))
    check(seq)
    check(seq, F32, window=1000, sinks=4)


UNEVEN = {
    "one long": [(1, 40), (1, 9000), (0, 500), (1, 0), (1, 1), (1, 700)],
    "none": [(0, 90), (1, 0)],
    "guesses": [(2, 5000), (1, 33), (0, 0), (2, 2), (2, 1)],
    "64 of them": [(1, 17 * i) for i in range(63)] + [(1, 20000)],
}


@pytest.mark.parametrize("hq, hk, D", [(8, 1, 128), (6, 2, 256), (3, 3, 64)])
@pytest.mark.parametrize("lens", list(UNEVEN), ids=str)
def test_uneven_lengths(lens, hq, hk, D):
    """Workgroups shared out by length, also to sequences without tokens or without queries."""
    seq = U.Sequences(UNEVEN[lens], q_heads=hq, kv_heads=hk, head_dim=D, group=64, page=64, dtype=BF16, seed=3)
    check(seq)
    check(seq, F32, window=600, sinks=70)


@pytest.mark.parametrize("lens, hq, hk, D, name, groups", [
    ([(1, 300)], 2, 2, 64, "rows_kernel<64, 64, 0, 8>", 2),
    ([(1, 300)] * 80, 4, 4, 64, "rows_kernel<64, 64, 0, 8>", 320),
    ([(1, 1500)] * 65, 4, 4, 64, "rows_kernel<64, 64, 0, 4>", 260 * 3),
    ([(1, 300)] * 65, 2, 1, 128, "rows_kernel<128, 64, 0, 8>", 65),
    ([(65, 100)], 1, 1, 128, "rows_kernel<128, 64, 0, 8>", 5),
    ([(300, 600)] * 2, 40, 8, 128, "tiles_kernel<128, 64, 0, 8, 4>", 16 * 12),
    ([(1024, 1024)], 64, 64, 64, "tiles_kernel<64, 64, 0, 8, 8>", 256),
    ([(300, 300)] * 16, 32, 16, 64, "tiles_kernel<64, 64, 0, 8, 8>", 3 * 256),
    ([(1, 40), (300, 301), (33, 600), (0, 5), (290, 290)] * 13, 8, 4, 128, "tiles_kernel<128, 64, 0, 8, 8>", 3 * 260),
    ([(100, 700)] * 3, 33, 1, 256, "rows_kernel<256, 64, 0, 4>", 3 * (170 + 37 * 4)),
    ([(70, 2300)], 64, 1, 256, "tiles_kernel<256, 64, 0, 4, 4>", 35 * 4),
    ([(70, 2300), (700, 700)], 48, 6, 128, "tiles_kernel<128, 64, 0, 8, 8>", 12 * (21 + 4)),
])
def test_variants(lens, hq, hk, D, name, groups):
    """Each kernel and way to split, and that the rule takes the one meant here."""
    seq = U.Sequences(lens, q_heads=hq, kv_heads=hk, head_dim=D, group=64, page=64, dtype=BF16, seed=5)
    attend(seq, seq.cache("cuda:0"), BF16)
    assert bm.bitmm_last_launches()[0].startswith(f"attention_{name} grid={groups}x1 ")
    check(seq)


@pytest.mark.parametrize("lens", [[(1, 700), (2, 90)], [(90, 700)], [(90, 100), (70, 3000)]], ids=str)
@pytest.mark.parametrize("D, power", [(64, 8), (128, 8), (256, 12), (128, -10)])
def test_scores_of_millions(lens, D, power):
    """Integer keys and queries, and scale = 2^power ln 2: a step of a score is a factor of
    2^(2^power), so that a row is the mean of the values at its largest score, or for a negative
    power a softmax whose exponents are exact. Both products are exact in any order: only the
    values, the probabilities and the sums are rounded."""
    seq = U.Sequences(lens, q_heads=4, kv_heads=2, head_dim=D, group=64, page=16, dtype=F16, seed=power)
    codes, scale, bias = seq.sides[0]
    seq.sides[0] = (codes, torch.ones_like(scale), torch.zeros_like(bias))
    seq.q = torch.randint(-3, 4, seq.q.shape, generator=torch.Generator().manual_seed(D)).to(F16)
    factor = 2.0 ** power * math.log(2.0)
    got, lse = attend(seq, seq.cache("cuda:0"), F32, scale=factor)
    h16, f32 = 2.0 ** -11, 2.0 ** -24
    for b, (nq, kv) in enumerate(seq.lens):
        r = slice(int(seq.cu[b]), int(seq.cu[b + 1]))
        (k, _), (v, vc) = seq.tokens(0, b, kv), seq.tokens(1, b, kv)
        see = torch.arange(kv)[None] <= torch.arange(kv - nq, kv)[:, None]
        for h in range(4):
            x = (seq.q[r, h].double() @ k[:, h // 2].T).masked_fill(~see, -math.inf) * factor
            p, n = torch.softmax(x, -1), see.sum(-1, keepdim=True)
            off = 4 * f32 * x.masked_fill(~see, 0).abs().amax(-1, keepdim=True)  # factor and exponents in f32
            if power > 0:  # the same for scores that are the same, and nothing beside them
                off = off * 0
            e = torch.expm1(2 * off) + h16 + f32 * (n + 64)
            va = v[:, h // 2].abs()
            tol = (p @ va) * e + h16 * (p @ (va + vc[:, h // 2])) + 2.0 ** -25 * (see.double() @ va)
            near(got[r, h], p @ v[:, h // 2], 1.01 * tol + f32 * (p @ va), f"head {h} of sequence {b}")
            want = torch.logsumexp(x, -1)
            near(lse[r, h], want, off[:, 0] + f32 * (n[:, 0] + 64) + 8 * f32 * want.abs(), "lse")


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales_of_scores(scale):
    seq = U.Sequences([(3, 90), (40, 200)], q_heads=4, kv_heads=2, head_dim=64, group=32, page=16, dtype=F16)
    check(seq, scale=scale)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 300.0, 1e6, 1e30])
@pytest.mark.parametrize("lens", [[(1, 500)], [(80, 200)]], ids=str)
def test_ranges_beyond_binary16(size, lens):
    """Keys and values far outside binary16's range (values; the keys' size is taken off the
    scale of the scores)."""
    seq = U.Sequences(lens, q_heads=4, kv_heads=1, head_dim=128, group=64, page=64, dtype=BF16, kv_scale=size)
    check(seq, F32, scale=0.05 / size)


def test_growing_range():
    """Later tokens a million times larger than the first, and then small again."""
    seq = U.Sequences([(1, 900), (64, 900)], q_heads=4, kv_heads=1, head_dim=64, group=32, page=64, dtype=BF16)
    for side in range(2):
        codes, scale, bias = seq.sides[side]
        for b in range(2):
            for page in (2, 7):
                scale[seq.table[b, page]] *= 2.0 ** 20
                bias[seq.table[b, page]] *= 2.0 ** 20
    check(seq, F32, scale=2.0 ** -22)


@pytest.mark.parametrize("lens", [[(1, 75), (1, 0), (1, 40)], [(50, 75), (50, 50)]], ids=str)
@pytest.mark.parametrize("window", [0, 20])
def test_stale_slots_do_not_matter(lens, window):
    """Slots past the sequences' ends hold NaN and infinite scales."""
    lens = [x for x in lens if x[1]]
    seq = U.Sequences(lens, q_heads=4, kv_heads=2, head_dim=64, group=64, page=32, dtype=BF16)
    cache = seq.cache("cuda:0")
    live = torch.zeros(cache.num_pages, 32, dtype=torch.bool)
    for b, (_, kv) in enumerate(lens):
        j = torch.arange(kv)
        live[seq.table[b].long()[j // 32], j % 32] = True
    for t in (cache.k_scales, cache.v_scales):
        x = t.cpu()
        x.transpose(1, 2)[~live] = torch.tensor([math.nan, math.inf], dtype=BF16)
        t.copy_(x)
    check(seq, window=window, cache=cache)


@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("lens", [[(1, 200)], [(100, 200)]], ids=str)
def test_not_finite_where_masked_and_where_seen(side, lens):
    """A token with a NaN (or infinite) scale makes NaN of the queries that see it and of no other."""
    seq = U.Sequences(lens, q_heads=4, kv_heads=1, head_dim=64, group=32, page=16, dtype=BF16)
    cache = seq.cache("cuda:0")
    t = cache.k_scales if side == "k" else cache.v_scales
    hidden, window = 130, 40        # seen by queries at 130 .. 169 alone
    t[seq.table[0, hidden // 16], 0, hidden % 16, 1, 0] = math.inf
    want, _, tol, _ = seq.reference(BF16, 0.125, window, 2)
    got, lse = attend(seq, cache, BF16, scale=0.125, window=window, sinks=2)
    got, lse = got.cpu(), lse.cpu()
    pos = torch.arange(200 - lens[0][0], 200)
    sees = (pos >= hidden) & (pos < hidden + window)
    assert got[sees].isnan().all() and lse[sees].isnan().all()
    near(got[~sees], want[~sees], tol[~sees])
    # and as one of the first tokens it is seen by all
    t[seq.table[0, 0], 0, 1, 0, 1] = math.nan
    got, _ = attend(seq, cache, BF16, scale=0.125, window=window, sinks=2)
    assert got.isnan().all()
    q = seq.q
    q[0, 1] = math.nan              # a NaN query is its own affair
    got, _ = attend(seq, seq.cache("cuda:0"), BF16, scale=0.125)
    assert got[0, 1].isnan().all() and got[0, 0].isfinite().all() and got[1:].isfinite().all()


def test_rows_that_see_nothing():
    """More queries than tokens, or none: zeros and -infinity; rows of no sequence are left alone."""
    seq = U.Sequences([(6, 4), (2, 0), (1, 50)], q_heads=3, kv_heads=1, head_dim=64, group=32, page=16, dtype=BF16)
    # the reference takes queries at positions kv - nq ..: the first two see nothing
    got = check(seq)
    assert (got[:2] == 0).all() and (got[6:8] == 0).all()
    seq.cu[0] = 1                   # row 0 belongs to nobody now
    out = torch.full(seq.q.shape, 5.0, device="cuda:0")
    lse = torch.full(seq.q.shape[:2], 5.0, device="cuda:0")
    bm.bitmm_kv_attention(dev(seq.q), seq.cache("cuda:0"), dev(seq.table), dev(seq.kv_lens), dev(seq.cu), out, None,
                          max_q=6, max_kv=50, lse=lse)
    assert (out[0] == 5).all() and (lse[0] == 5).all() and (out[1] == 0).all()


@pytest.mark.parametrize("lens", [[(1, 100), (1, 100)], [(60, 100), (33, 100)]], ids=str)
def test_bad_pages(lens):
    """Tokens on a page outside the cache are seen by nobody; the status word tells."""
    seq = U.Sequences(lens, q_heads=4, kv_heads=2, head_dim=64, group=32, page=32, dtype=BF16)
    cache = seq.cache("cuda:0")
    word = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    good = attend(seq, cache, BF16, status=word)[0]
    assert word.item() == 0
    keep = seq.table.clone()
    for bad in (-1, cache.num_pages, 2 ** 31 - 1):
        seq.table = keep.clone()
        seq.table[0, 1] = bad
        word.zero_()
        hide = lambda b, j: (j // 32 == 1) if b == 0 else j < 0  # noqa: E731
        bad_table, seq.table = seq.table, keep          # the reference reads no bad page
        want, _, tol, _ = seq.reference(BF16, 0.125, hide=hide)
        seq.table = bad_table
        got, _ = attend(seq, cache, BF16, scale=0.125, status=word)
        assert word.item() == 1
        near(got, want, tol)
    n = int(seq.cu[1])
    assert torch.equal(got[n:], good[n:])


def test_lengths_are_cut_to_bounds():
    """Lengths and offsets that pass what the host was told are cut and reported."""
    seq = U.Sequences([(1, 90), (1, 60)], q_heads=2, kv_heads=1, head_dim=64, group=32, page=16, dtype=BF16)
    cache = seq.cache("cuda:0")
    word = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    good = attend(seq, cache, BF16, status=word)[0]
    assert word.item() == 0
    for change, rows in [(dict(lens=[90, 2 ** 31 - 1]), 1), (dict(lens=[90, -5]), 1), (dict(cu=[0, 1, 7]), 2),
                         (dict(cu=[0, 1, -3]), 1), (dict(cu=[-4, 1, 2]), 2), (dict(cu=[0, 1, 0]), 1)]:
        t = dict(lens=seq.kv_lens.tolist(), cu=seq.cu.tolist())
        t.update(change)
        word.zero_()
        out = bm.kv_attention(dev(seq.q), cache, dev(seq.table), dev(torch.tensor(t["lens"], dtype=torch.int32)),
                              dev(torch.tensor(t["cu"], dtype=torch.int32)), max_q=1, max_kv=90, status=word)
        assert word.item() == 1, change
        assert torch.equal(out[:rows], good[:rows]), change


def test_strides_and_streams():
    """Queries and outputs as slices of wider rows, on a stream of its own."""
    seq = U.Sequences([(1, 400), (60, 60)], q_heads=6, kv_heads=2, head_dim=128, group=64, page=64, dtype=BF16)
    cache = seq.cache("cuda:0")
    good, _ = attend(seq, cache, BF16)
    T = seq.q.shape[0]
    wide = torch.zeros(T, 11, 128, dtype=BF16, device="cuda:0")
    wide[:, 2:8] = dev(seq.q)
    out = torch.full((T, 9, 128), 3.0, dtype=BF16, device="cuda:0")
    args = [dev(t) for t in (seq.table, seq.kv_lens, seq.cu)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    need = bm.bitmm_kv_attention_workspace_bytes(T, 2, 60, 400, 6, 2, 128)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda:0")
    bm.bitmm_kv_attention(wide[:, 2:8], cache, *args, out[:, 1:7], ws, max_q=60, max_kv=400, stream=side)
    side.synchronize()
    assert torch.equal(out[:, 1:7], good) and (out[:, 0] == 3).all() and (out[:, 7:] == 3).all()


def test_results_are_the_same_every_time():
    seq = U.Sequences([(1, 20000), (1, 7000)], q_heads=8, kv_heads=2, head_dim=128, group=64, page=64, dtype=BF16)
    cache = seq.cache("cuda:0")
    a, la = attend(seq, cache, F32)
    for _ in range(3):
        b, lb = attend(seq, cache, F32)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_offsets_past_32_bits():
    """Pages whose codes lie past 2^32 bytes and 2^31 words."""
    pages, page, hk, D, group = 33500, 256, 8, 256, 128
    cache = bm.KVCache.empty(pages, page, hk, D, group)
    assert cache.k_codes.numel() > 2 ** 31
    seq = U.Sequences([(1, 600), (20, 300)], q_heads=8, kv_heads=hk, head_dim=D, group=group, page=page, dtype=BF16)
    for t, (codes, scale, bias) in zip(((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)), seq.sides):
        n = codes.shape[0]
        t[0][pages - n:] = dev(U.pack(codes))
        t[1][pages - n:] = dev(torch.stack([scale, bias], -1).to(BF16))
    want, _, tol, _ = seq.reference(BF16, 1 / 16)
    got = bm.kv_attention(dev(seq.q), cache, dev(seq.table) + (pages - seq.sides[0][0].shape[0]), dev(seq.kv_lens),
                          dev(seq.cu), max_q=20, max_kv=600)
    near(got, want, tol)
    k = torch.randn(2, hk, D, device="cuda:0").to(BF16)
    slots = torch.tensor([pages * page - 1, pages * page - 300], device="cuda:0")
    bm.bitmm_kv_append(k, k, slots, cache)
    y, z = bm.kv_read(cache, slots)
    c, s, b = U.quantise(k.cpu(), group)
    want = U.values(c, s, b)
    near(y, want, 2.0 ** -7 * want.abs())
    assert torch.equal(y, z)


def test_graph_replays():
    """A decoding step (norms and rotation, append, attention) captured and replayed with other inputs."""
    hq, hk, D = 8, 2, 128
    seq = U.Sequences([(1, 3000), (1, 1200)], q_heads=hq, kv_heads=hk, head_dim=D, group=64, page=64, dtype=BF16)
    cache = seq.cache("cuda:0")
    table, lens, cu = (dev(t) for t in (seq.table, seq.kv_lens, seq.cu))
    qkv = torch.randn(2, hq + 2 * hk, D, device="cuda:0").to(BF16)
    w = torch.ones(D, dtype=BF16, device="cuda:0")
    freq = dev(bm.rope_frequencies(D)[0])
    slots = torch.stack([seq.table[b, (int(n) - 1) // 64].long() * 64 + (int(n) - 1) % 64
                         for b, n in enumerate(seq.kv_lens)]).cuda()
    q, k = torch.empty(2, hq, D, dtype=BF16, device="cuda:0"), torch.empty(2, hk, D, dtype=BF16, device="cuda:0")
    out = torch.empty_like(q)
    ws = torch.empty(bm.bitmm_kv_attention_workspace_bytes(2, 2, 1, 3000, hq, hk, D) + 1, dtype=torch.uint8,
                     device="cuda:0")

    def step():
        bm.bitmm_qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hk], w, w, lens, freq, q, k)
        bm.bitmm_kv_append(k, qkv[:, hq + hk:], slots, cache)
        bm.bitmm_kv_attention(q, cache, table, lens, cu, out, ws, max_q=1, max_kv=3000)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(4):
        qkv.copy_(torch.randn(qkv.shape, device="cuda:0"))
        step()
        torch.cuda.synchronize()
        eager = out.clone()
        out.fill_(99)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i
        _ = (qkv.float() * 2).sum().item()
    del graph
