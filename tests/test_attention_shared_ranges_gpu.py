"""Attention over shared and own tokens whose sizes are far apart, or not finite: between the two, within each, in every
kernel that the call may take, against 64 bits."""

import math

import pytest
import torch

import bit_matmul_amd as bm
from tests.test_attention_shared_gpu import BF, F16, F32, Groups, beams

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bm.lib()
    yield
    torch.cuda.synchronize()


# Bounds of the lengths choose the kernels: (bounds, what the passes are called)
FORMS = {
    "one launch": ({}, ["rows both"]),
    "rows": (dict(max_prefix=3000), ["rows prefix", "rows own"]),
    "rows, joined": (dict(max_prefix=3000, max_kv=3000), ["rows prefix", "rows own", "join"]),
    "tiles": (dict(max_group_q=8192, max_prefix=2047, max_q=8192, max_kv=2047), ["tiles prefix", "tiles own"]),
    "tiles, split": (dict(max_group_q=200, max_prefix=65536, max_q=8192, max_kv=2047), ["tiles prefix", "tiles own"]),
    "tiles, joined": (dict(max_group_q=200, max_prefix=65536, max_q=130, max_kv=65536), ["tiles prefix", "tiles own", "join"]),
}
SHAPES = {
    "decode": [(300, beams(3, 1, 40)), (150, [(1, 5), (2, 90)])],
    "chunks": [(200, [(80, 120), (30, 30)]), (90, [(70, 70)])],
}
forms = pytest.mark.parametrize("form", list(FORMS))
shapes = pytest.mark.parametrize("shape", list(SHAPES))


def groups_of(shape, D=128, group=64, dtype=BF, seed=2):
    return Groups(SHAPES[shape], q_heads=4, kv_heads=2, head_dim=D, group=group, page=32, dtype=dtype, seed=seed)


def run(s, form, **kw):
    b = {k: max(v, s.bounds()[k]) for k, v in FORMS[form][0].items()}
    out, lse, status = s.run(out_dtype=F32, **b, **kw)
    names = [line.replace("attention_", "").split("<")[0].replace("_shared_kernel", "").replace("_kernel", "") for line in bm.bitmm_last_launches()]
    passes = [line.split(">")[0].split(", ")[-1] for line in bm.bitmm_last_launches()]
    got = [n if n == "join" else f"{n} {p}" for n, p in zip(names, passes)]
    assert got == FORMS[form][1] and status == 0
    return out, lse


def times(s, side, part, tokens, factor):
    """The keys (side 0) or values of those shared or own tokens times a power of two."""
    _, scale, bias = s.sides[side]
    tables = zip(s.prefix_table, s.shared) if part == "shared" else zip(s.page_table, [n for _, n in s.own])
    for table, n in tables:
        for t in tokens:
            if t < n:
                page, off = table[t // s.page].long(), t % s.page
                scale[page, :, off] *= factor
                bias[page, :, off] *= factor


def compare(s, form, scale=None, only=None):
    scale = 1 / math.sqrt(s.head_dim) if scale is None else scale
    out, lse = run(s, form, scale=scale)
    want, want_lse, tol, tol_lse = s.reference(F32, scale)
    keep = torch.ones(len(s.q), dtype=torch.bool) if only is None else only
    assert keep.any()
    assert ((out - want).abs() <= tol)[keep].all()
    assert ((lse == want_lse) | ((lse - want_lse).abs() <= tol_lse))[keep].all()


@forms
@shapes
@pytest.mark.parametrize("dtype", [BF, F16], ids=str)
@pytest.mark.parametrize("D, group", [(64, 32), (128, 128), (256, 64)])
def test_ordinary(form, shape, dtype, D, group):
    compare(groups_of(shape, D, group, dtype), form)


@forms
@shapes
@pytest.mark.parametrize("factor", [2.0 ** 20, 2.0 ** 45, 2.0 ** 100, 2.0 ** -20, 2.0 ** -45, 2.0 ** -100], ids=str)
@pytest.mark.parametrize("part", ["shared", "own"])
@pytest.mark.parametrize("tokens", ["all", "one", "every other", "later half"])
def test_values_of_many_sizes(form, shape, factor, part, tokens):
    """Shared values far larger or smaller than the own ones, and some among either: each as exact as its size allows."""
    s = groups_of(shape)
    times(s, 1, part, {"all": range(500), "one": [35], "every other": range(0, 500, 2), "later half": range(45, 500)}[tokens], factor)
    compare(s, form)


@forms
@shapes
@pytest.mark.parametrize("factor", [2.0 ** -12, 2.0 ** -20, 2.0 ** -60, 2.0 ** -100], ids=str)
@pytest.mark.parametrize("part", ["shared", "own"])
@pytest.mark.parametrize("D, group", [(64, 64), (128, 32), (256, 128)])
def test_keys_of_many_sizes(form, shape, factor, part, D, group):
    for tokens in (range(500), range(0, 500, 2), range(0, 45), [t for t in range(500) if t != 35]):
        s = groups_of(shape, D, group, F16)
        times(s, 0, part, tokens, factor)
        compare(s, form)


@forms
@shapes
@pytest.mark.parametrize("D, group", [(64, 32), (128, 64), (256, 64)])
def test_growing_range(form, shape, D, group):
    """Shared tokens a million times larger than the first ones, in keys and values, then small again; and own ones."""
    for part, tokens in (("shared", range(64, 96)), ("shared", range(0, 200)), ("own", range(20, 60))):
        s = groups_of(shape, D, group)
        for side in range(2):
            times(s, side, part, tokens, 2.0 ** 20)
        compare(s, form, scale=2.0 ** -22)


@forms
@pytest.mark.parametrize("factor", [2.0 ** 40, 2.0 ** 100, 2.0 ** -40, 2.0 ** -100], ids=str)
def test_extreme_token_after_a_query(form, factor):
    """A row's result does not depend on an own token behind it, whatever finite values that has."""
    s = groups_of("chunks")
    for side in range(2):
        times(s, side, "own", [25, 29], factor)
    position = torch.cat([torch.arange(n - q, n) for q, n in s.own])
    compare(s, form, only=position < 25)


@forms
@shapes
@pytest.mark.parametrize("bits", [13, 26, 39])
@pytest.mark.parametrize("part", ["shared", "own"])
def test_weight_on_one_token(form, shape, bits, part):
    """A token, the first shared or own one, that takes all but 2^-3 to 2^-29 of the weight and has nothing to give: the
    rest keep their bits on both sides of it. Scores are whole numbers of bits; a probability is rounded to 2^-11 of itself or,
    where it is small beside the others of its step or half tile, to 2^-25 of 2^-9 at least: 2^-11 of the part's weight
    for 32 of them, and where the heavy token is in the part, 64 * 2^-29 of its weight."""
    s = groups_of(shape)
    g = torch.Generator().manual_seed(bits)
    for side, (codes, scale, bias) in enumerate(s.sides):
        codes = torch.randint(1, 4, codes.shape, generator=g) if side == 0 else codes
        scale, bias = torch.ones_like(scale), torch.zeros_like(bias)
        if side == 1:
            scale, bias = scale / 16, bias + 1
        for table in s.prefix_table if part == "shared" else s.page_table:
            page = table[0].long()
            if side == 0:
                codes[page, :, 0, 0] = 15
            else:
                scale[page, :, 0], bias[page, :, 0] = 0, 0
        s.sides[side] = (codes, scale, bias)
    s.q = torch.zeros_like(s.q)
    s.q[..., 0] = bits / 13          # 15 against 1, 2 or 3
    out, lse = run(s, form, scale=math.log(2))
    h16, f32 = 2.0 ** -11, 2.0 ** -24
    for b, (nq, kv) in enumerate(s.lens):
        r = slice(int(s.cu[b]), int(s.cu[b + 1]))
        (k, _), (v, vc) = s.tokens(0, b, kv), s.tokens(1, b, kv)
        at = 0 if part == "shared" else s.shared[s.prefix_of[b]]
        see = torch.arange(kv)[None] <= torch.arange(kv - nq, kv)[:, None]
        for h in range(4):
            x = (s.q[r, h].double() @ k[:, h // 2].T).masked_fill(~see, -math.inf) * math.log(2)
            p, n = torch.softmax(x, -1), see.sum(-1, keepdim=True)
            off = 4 * f32 * x.masked_fill(~see, 0).abs().amax(-1, keepdim=True)
            rest = p.clone()
            rest[:, at] = 0
            want = p @ v[:, h // 2]
            tol = want * (torch.expm1(2 * off) + h16 + f32 * (n + 64)) + h16 * (p @ (v + vc)[:, h // 2])
            tol += 2 * (h16 * rest.sum(-1, keepdim=True) + 64 * 2.0 ** -29 * p[:, at:at + 1])
            assert ((out[r, h] - want).abs() <= 1.01 * tol).all()
            total = torch.logsumexp(x, -1)
            assert ((lse[r, h] - total).abs() <= off[:, 0] + f32 * (n[:, 0] + 64) + 8 * f32 * total.abs()).all()


@forms
@shapes
@pytest.mark.parametrize("part", ["shared", "own"])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("side", [0, 1])
def test_what_is_not_finite(form, shape, part, value, side):
    """A scale that is not finite makes NaN of the rows that see its token, and of no others."""
    s = groups_of(shape)
    clean, _ = run(s, form)
    if part == "shared":       # token 33 of the first group, second kv head
        page, off = s.prefix_table[0, 1].long(), 1
        hit = torch.tensor([p == 0 for (q, _), p in zip(s.own, s.prefix_of) for _ in range(q)])
    else:                      # own token 3 of the last sequence
        page, off = s.page_table[-1, 0].long(), 3
        hit = torch.zeros(len(s.q), dtype=torch.bool)
        q, n = s.own[-1]
        hit[len(s.q) - q:] = torch.arange(n - q, n) >= 3
    s.sides[side][1][page, 1, off] = value
    out, _ = run(s, form)
    assert out[hit][:, 2:].isnan().all()
    # others are as they were, but for a second attempt's units
    want, _, tol, _ = Groups.reference(groups_of(shape), F32, 1 / math.sqrt(128))
    off = (out - want).abs() <= tol
    assert off[~hit].all() and off[:, :2].all() and clean.isfinite().all()
