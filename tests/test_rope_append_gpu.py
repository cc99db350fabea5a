"""Norm, rotation and append in one call, on the GPU: queries are those of the call without the append, values'
codes those of kv_append, and keys' codes the nearest ones in 64 bits."""

import pytest
import torch

import bit_matmul_amd as bm
from tests import attn_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bm.lib()
    yield
    torch.cuda.synchronize()


def filled(pages, page, heads, D, group):
    """A cache whose every word is known, so that one written by mistake shows."""
    c = bm.KVCache.empty(pages, page, heads, D, group)
    for t, v in ((c.k_codes, 0x12345678), (c.v_codes, 0x31415926), (c.k_scales, 3.5), (c.v_scales, -2.25)):
        t.fill_(v)
    return c


def tensors(c):
    return [c.k_codes, c.k_scales, c.v_codes, c.v_scales]


def unpack(words):
    w = words.cpu().long()
    return ((w.unsqueeze(-1) >> torch.arange(0, 32, 4)) & 15).flatten(-2)


def held(c, slots, side):
    """(codes [T, heads, D], scales, biases f64 [T, heads, groups]) of slots >= 0."""
    s = slots.cpu()
    at, off = s // c.page_size, s % c.page_size
    codes, pairs = tensors(c)[2 * side:2 * side + 2]
    pairs = pairs.cpu()[at, :, off].double()
    return unpack(codes.cpu()[at, :, off]), pairs[..., 0], pairs[..., 1]


def check_keys(got, k64, group):
    """Scale and bias are the group's, rounded once, and each code the nearest, to 2^-30 of a code."""
    codes, scale, bias = got
    g = k64.unflatten(-1, (-1, group))
    low, high = g.amin(-1), g.amax(-1)
    assert torch.equal(bias, low.bfloat16().double())
    assert torch.equal(scale, ((high - low) / 15).bfloat16().double())
    s = torch.where(scale > 0, scale, torch.ones_like(scale))
    t = ((g - bias[..., None]) / s[..., None]).clamp(0, 15) * (scale > 0)[..., None]
    off = (t - codes.unflatten(-1, (-1, group))).abs()
    assert off.max() <= 0.5 + 2.0 ** -30


def inputs(T, hq, hk, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, hq + 2 * hk + 1, D, generator=g)
    qkv[..., ::16] *= 4
    qkv = qkv.to(dtype).cuda()
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2)]
    pos = torch.randint(-5, 1 << 17, (T,), generator=g).to(torch.int32).cuda()
    return qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:hq + 2 * hk], w[0], w[1], pos


CASES = [  # tokens, query heads, kv heads, dims, group, page, rotated dims, interleaved, type
    (1, 5, 1, 64, 32, 16, 64, False, torch.bfloat16), (3, 8, 2, 64, 64, 32, 8, False, torch.float16),
    (7, 0, 3, 64, 64, 64, 64, True, torch.bfloat16), (33, 40, 8, 128, 64, 64, 128, False, torch.bfloat16),
    (16, 6, 3, 128, 32, 16, 24, False, torch.float16), (5, 7, 7, 128, 128, 128, 40, True, torch.bfloat16),
    (9, 4, 1, 128, 128, 256, 0, False, torch.float16), (600, 10, 5, 128, 64, 64, 64, False, torch.float16),
    (11, 16, 2, 256, 32, 16, 64, True, torch.float16), (2, 2, 2, 256, 64, 16, 256, False, torch.bfloat16),
    (301, 3, 1, 256, 128, 32, 120, False, torch.bfloat16), (2100, 8, 8, 64, 32, 16, 48, False, torch.bfloat16),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c).replace("torch.", ""))
def test_against_64_bits(case):
    T, hq, hk, D, group, page, rot, interleaved, dtype = case
    q, k, v, qw, kw, pos = inputs(T, hq, hk, D, dtype, seed=T)
    freq, _ = bm.rope_frequencies(rot, 10000.0, device="cuda") if rot else (None, None)
    pages = -(-T // page) + 2
    c, plain = (filled(pages, page, hk, D, group) for _ in range(2))
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(T))[:T].cuda()
    options = dict(interleaved=interleaved, eps=1e-5, weight_offset=0.25, rope_scale=1.25)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if hq:
        got = bm.qk_norm_rope_append(q, k, v, qw, kw, pos, freq, slots, c, status=status, **options)
        assert len(bm.bitmm_last_launches()) == 1
        want, _ = bm.qk_norm_rope(q, None, qw, None, pos, freq, **options)
        assert torch.equal(got, want)
    else:
        assert bm.bitmm_qk_norm_rope_append(None, k, v, None, kw, pos, freq, None, slots, c, status=status, **options) is None
    eps = float(torch.tensor(1e-5, dtype=torch.float32))   # as the C call takes it
    k64, _ = U.rope_reference(k.cpu(), kw.cpu(), pos.cpu(), torch.zeros(0) if freq is None else freq.cpu(),
                              interleaved=interleaved, eps=eps, weight_offset=0.25, rope_scale=1.25)
    check_keys(held(c, slots, 0), k64, group)
    bm.bitmm_kv_append(k, v, slots, plain)
    assert torch.equal(c.v_codes, plain.v_codes) and torch.equal(c.v_scales, plain.v_scales)
    other = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    other[slots] = False   # slots that were not given stay as they were
    other = other.view(pages, page)
    untouched = filled(pages, page, hk, D, group)
    for a, b in zip(tensors(c), tensors(untouched)):
        assert torch.equal(a.transpose(1, 2)[other], b.transpose(1, 2)[other])
    assert status.item() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D, group", [(64, 32), (128, 64), (256, 128)])
def test_without_norm_and_rotation_it_is_the_append(D, group, dtype):
    """Keys as they come are 16-bit numbers, many of them halfway between two codes."""
    T, hk = 500, 3
    g = torch.Generator().manual_seed(D)
    k = torch.randn(T, hk, D, generator=g)
    k[:100] = torch.randint(-7, 9, (100, hk, D), generator=g) * 0.5    # scales and codes that are whole numbers
    k[100] = 0
    k[101] = 3.25
    k[102] = torch.randint(0, 2, (hk, D), generator=g) * 1e-6
    k, v = k.to(dtype).cuda(), torch.randn(T, hk, D, generator=g).to(dtype).cuda()
    a, b = (filled(9, 64, hk, D, group) for _ in range(2))
    slots = torch.arange(T).cuda()
    bm.bitmm_qk_norm_rope_append(None, k, v, None, None, None, None, None, slots, a)
    bm.bitmm_kv_append(k, v, slots, b)
    for x, y in zip(tensors(a), tensors(b)):
        assert torch.equal(x, y)


def test_slots_that_store_nothing():
    q, k, v, qw, kw, pos = inputs(6, 4, 2, 128, torch.bfloat16, 1)
    freq, _ = bm.rope_frequencies(128, device="cuda")
    c = filled(4, 16, 2, 128, 64)
    want = [t.clone() for t in tensors(c)]
    for slots, flagged in (([-1] * 6, 0), ([-1, -1, 64, -1, -1, -1], 1), ([-2, -1, -1, -1, -1, -1], 1), ([2 ** 40] + [-1] * 5, 1),
                           ([-2 ** 62, -1, -1, -1, -1, 2 ** 62], 1)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = bm.qk_norm_rope_append(q, k, v, qw, kw, pos, freq, torch.tensor(slots).cuda(), c, status=status)
        assert torch.equal(got, bm.qk_norm_rope(q, None, qw, None, pos, freq)[0])
        assert status.item() == flagged
        assert all(torch.equal(a, b) for a, b in zip(tensors(c), want))


def test_in_place_and_other_stream():
    q, k, v, qw, kw, pos = inputs(40, 8, 2, 64, torch.float16, 2)
    freq, scale = bm.rope_frequencies(64, device="cuda")
    c, d = filled(4, 16, 2, 64, 32), filled(4, 16, 2, 64, 32)
    slots = torch.arange(40).cuda()
    want = bm.qk_norm_rope_append(q, k, v, qw, kw, pos, freq, slots, c)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    other = bm.qk_norm_rope_append(q, k, v, qw, kw, pos, freq, slots, d, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(want, other) and all(torch.equal(a, b) for a, b in zip(tensors(c), tensors(d)))
    bm.bitmm_qk_norm_rope_append(q, k, v, qw, kw, pos, freq, q, slots, d)
    assert torch.equal(want, q) and all(torch.equal(a, b) for a, b in zip(tensors(c), tensors(d)))


def test_what_is_not_finite_stays_in_its_group():
    """An infinity in a normed head makes its sum of squares infinite, and with it the head's values 0 or NaN."""
    D, group = 128, 32
    k = torch.randn(4, 2, D).bfloat16()
    k[1, 0, 5] = float("nan")
    k[2, 1, 40] = float("inf")
    k = k.cuda()
    for norm in (False, True):
        w = torch.ones(D, dtype=torch.bfloat16, device="cuda") if norm else None
        a, b = filled(1, 16, 2, D, group), filled(1, 16, 2, D, group)
        slots = torch.arange(4).cuda()
        bm.bitmm_qk_norm_rope_append(None, k, k, None, w, None, None, None, slots, a)
        sane = k.nan_to_num(0, 0, 0)
        bm.bitmm_qk_norm_rope_append(None, sane, sane, None, w, None, None, None, slots, b)
        x, y = a.k_scales[0, :, :4], b.k_scales[0, :, :4]
        touched = torch.zeros(2, 4, D // group, dtype=torch.bool)
        touched[0, 1, slice(None) if norm else 0] = True
        touched[1, 2, slice(None) if norm else 1] = True
        # finite values over an infinite root are zeros
        nans = x.isnan().all(-1).cpu()
        expect = touched.clone()
        if norm:
            expect[1, 2] = torch.tensor([False, True, False, False])
        assert torch.equal(nans, expect)
        assert torch.equal(x.cpu()[~touched], y.cpu()[~touched])
        assert torch.equal(a.k_codes[0, 1, 3], b.k_codes[0, 1, 3])


def test_captured():
    """A captured call, replayed over other tokens, gives what eager calls give."""
    T = 5
    q, k, v, qw, kw, pos = (t.clone() for t in inputs(T, 8, 2, 128, torch.bfloat16, 3))
    freq, _ = bm.rope_frequencies(128, device="cuda")
    c, d = filled(4, 16, 2, 128, 64), filled(4, 16, 2, 128, 64)
    slots = torch.arange(T).cuda()
    out = torch.empty_like(q)
    call = lambda cache, to: bm.bitmm_qk_norm_rope_append(q, k, v, qw, kw, pos, freq, to, slots, cache)
    call(c, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c, out)
    for i in range(4):
        new = inputs(T, 8, 2, 128, torch.bfloat16, 10 + i)
        for t, n in zip((q, k, v, qw, kw, pos), new):
            t.copy_(n)
        slots.copy_(torch.arange(T) + 7 * i)
        graph.replay()
        torch.cuda.synchronize()
        eager = torch.empty_like(q)
        call(d, eager)
        assert torch.equal(out, eager)
        at = slots
        assert all(torch.equal(a[at // 16, :, at % 16], b[at // 16, :, at % 16]) for a, b in zip(tensors(c), tensors(d)))
