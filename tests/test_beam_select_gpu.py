"""Beam search's selection on the GPU, against the definition in 64 bits: places are equal, scores are the
totals rounded once."""

import math

import pytest
import torch

import bit_matmul_amd as bm

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bm.lib()
    yield
    torch.cuda.synchronize()


def reference(logits, scores, k, beams, finished=None, end_token=-1):
    """(totals f64, parents, tokens, finished) on the CPU; within a beam the order is that of the logits."""
    x, s = logits.cpu().double(), scores.cpu().double()
    groups, vocab = x.shape[0] // beams, x.shape[1]
    done = torch.zeros(x.shape[0], dtype=torch.bool) if finished is None else finished.cpu()
    few = min(k, vocab)
    out = []
    for g in range(groups):
        found = []
        for b in range(beams):
            r = g * beams + b
            bad = not s[r] < math.inf or (not done[r] and not (x[r] < math.inf).all())
            if bad or s[r] == -math.inf:
                continue
            if done[r]:
                if 0 <= end_token < vocab:
                    found.append((-s[r].item(), b, 0, end_token))
                continue
            total = s[r] + (x[r] - torch.logsumexp(x[r], 0))
            value, token = torch.sort(x[r], descending=True, stable=True)
            found += [(-total[t].item(), b, i, t) for i, t in enumerate(token[:few].tolist()) if x[r, t] > -math.inf]
        best = sorted(found)[:k]
        best += [(math.inf, -1, 0, -1)] * (k - len(best))
        out.append([(-t, b, v, b >= 0 and (bool(done[g * beams + b]) or v == end_token)) for t, b, _, v in best])
    total, parents, tokens, ended = ([[c[i] for c in row] for row in out] for i in range(4))
    return torch.tensor(total, dtype=torch.float64), torch.tensor(parents), torch.tensor(tokens), torch.tensor(ended)


def check(logits, scores, k, beams, finished=None, end_token=-1, flagged=0, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = bm.beam_select(logits, scores, k, beams=beams, finished=finished, end_token=end_token, status=status, **kw)
    want = reference(logits, scores, k, beams, finished, end_token)
    assert [t.dtype for t in got] == [torch.float32, torch.int32, torch.int32, torch.bool]
    for a, b in zip(got[1:], want[1:]):
        assert torch.equal(a.cpu().to(b.dtype), b)
    none = want[0] == -math.inf
    assert torch.equal(got[0].cpu() == -math.inf, none)
    # one rounding to f32, and 2^-30 for the f64 sum's exponentials (4e-11 each) and logarithm
    off = (got[0].cpu().double() - want[0]).masked_fill(none, 0).abs()
    assert (off <= 2.0 ** -24 * want[0].masked_fill(none, 0).abs() + 2.0 ** -30).all()
    assert status.item() == flagged
    return got


def rows(n, vocab, dtype, seed, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn(n, vocab, generator=g)
    return x.to(dtype).cuda(), (-6 * torch.rand(n, generator=g)).cuda()


CASES = [  # groups, beams, vocabulary, k
    (1, 1, 1, 1), (2, 3, 1, 5), (1, 2, 2, 4), (3, 2, 7, 4), (1, 4, 8, 8), (2, 5, 9, 10), (1, 1, 63, 64), (4, 3, 100, 6),
    (1, 64, 64, 64), (2, 64, 1000, 64), (1, 2, 1023, 64), (3, 4, 1025, 8), (7, 4, 5000, 4), (1, 4, 32000, 8), (13, 5, 50001, 10),
    (1, 1, 200003, 16), (40, 8, 4099, 8), (300, 4, 1031, 4), (2, 33, 33333, 33), (1, 8, 262144, 64),
]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_64_bits(case, dtype):
    groups, beams, vocab, k = case
    x, s = rows(groups * beams, vocab, dtype, seed=vocab)
    check(x, s, k, beams)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_strides_and_offsets(dtype):
    """Rows that start at any element, and what lies between them is not looked at."""
    for vocab, stride, offset in ((1000, 1001, 0), (997, 1003, 1), (2048, 2053, 3), (5, 6, 5), (4096, 8192, 7)):
        x, s = rows(6, vocab, dtype, seed=stride)
        whole = torch.full((6 * stride + offset,), math.inf, dtype=dtype, device="cuda")
        view = whole[offset:].view(6, stride)[:, :vocab]
        view.copy_(x)
        got = check(view, s, 6, 3)
        assert all(torch.equal(a, b) for a, b in zip(got, check(x, s, 6, 3)))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("vocab", [70, 3001, 40007])
def test_ties(dtype, vocab):
    """Equal logits go to the lowest token, equal beams to the lowest beam, wherever their rows begin."""
    g = torch.Generator().manual_seed(vocab)
    s = torch.tensor([-1.0, -1.0, -0.5, -1.0], device="cuda")
    flat = torch.zeros(4, vocab, dtype=dtype, device="cuda")
    check(flat, s, 64, 4)
    check(flat, s, 5, 4)
    two = torch.randint(0, 2, (1, vocab), generator=g).to(dtype).cuda().expand(4, vocab).contiguous()
    check(two, s, 64, 4)
    check(two, s, 64, 2)
    few = torch.randint(-3, 3, (4, vocab), generator=g).to(dtype).cuda()
    few[2] = few[0]
    few[3] = few[0]
    check(few, s, 33, 4)
    signs = torch.where(torch.rand(4, vocab, generator=g) < 0.5, 0.0, -0.0).to(dtype).cuda()
    check(signs, s, 64, 4)
    one = flat.clone()
    one[:, -1] = 1
    one[:, 0] = 1
    check(one, s, 3, 4)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("vocab", [700, 60001])
def test_orders(dtype, vocab):
    """Logits that rise pass every threshold, those that fall none; both, and one of the two in blocks."""
    up = torch.linspace(-30, 30, vocab)
    s = torch.tensor([-0.1, -0.2, -0.3, -0.4], device="cuda")
    blocks = up.view(-1, 1).expand(-1, 1).clone()
    blocks[::3] = -blocks[::3]
    x = torch.stack([up, up.flip(0), blocks[:, 0], up * 0.5]).to(dtype).cuda()
    for k in (1, 8, 64):
        check(x, s, k, 4)
        check(x, s, k, 2)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_masked_logits(dtype):
    """-infinity is no candidate: rows with less than k others, with none at all, and with one at any place."""
    vocab = 5003
    x, s = rows(4, vocab, dtype, 3)
    x[0] = -math.inf
    x[1] = -math.inf
    x[1, 4097] = 2
    x[2, 100:] = -math.inf
    x[3, ::2] = -math.inf
    check(x, s, 8, 4)
    check(x, s, 64, 2)
    x[:] = -math.inf
    check(x, s, 3, 4)
    for at in (0, 1, 7, 8, 63, 511, 512, 1024, 5002):
        x[2] = -math.inf
        x[2, at] = -50
        check(x, s, 2, 4)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_far_apart(dtype):
    """Logits whose exponentials pass f32's range, upwards and downwards, and a jump late in the row."""
    big = 6e4 if dtype is torch.float16 else 3e38
    vocab = 9000
    x, s = rows(5, vocab, dtype, 4)
    x[0, :4000] = -1000
    x[0, 4000:] += 1000
    x[1] *= 100
    x[2, 8999] = big
    x[3] = -big
    x[3, 77] = -big * 0.5
    x[4, 5] = -big
    check(x, s, 10, 5)
    check(x, s, 10, 1)


def test_finished_beams():
    x, s = rows(12, 4000, torch.bfloat16, 5)
    done = torch.zeros(12, dtype=torch.bool, device="cuda")
    done[[1, 4, 5, 6, 7]] = True
    x[1] = math.nan        # not read
    s[6] = -0.01
    check(x, s, 4, 4, finished=done, end_token=17)
    check(x, s, 8, 4, finished=done, end_token=3999)
    check(x, s, 4, 4, finished=done, end_token=-1)      # finished beams that have no end
    check(x, s, 4, 4, finished=done, end_token=4000)
    x[3, 17] = 30          # a beam that ends now
    got = check(x, s, 4, 4, finished=done, end_token=17)
    assert got[3][0].any()
    check(x, s, 4, 4, finished=torch.ones_like(done), end_token=17)


def test_beams_that_do_not_count():
    x, s = rows(8, 3000, torch.float32, 6)
    s[1:4] = -math.inf     # a search's first step: one live beam
    check(x, s, 8, 4)
    s[:] = -math.inf
    check(x, s, 4, 4)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_what_is_not_a_number(dtype):
    """A row with a NaN or +infinity has no candidates, whatever its place and sign, and others are as without it."""
    for at, value in ((0, math.nan), (3999, math.nan), (2000, math.inf), (4001, math.nan), (7, math.inf)):
        x, s = rows(6, 4002, dtype, 7)
        x[1, at] = value
        check(x, s, 6, 3, flagged=1)
        x[1, at] = -math.nan if value != value else value
        if value != value:
            bits = x.view(torch.int32 if dtype is torch.float32 else torch.int16)
            bits[1, at] |= -(1 << 31) if dtype is torch.float32 else -(1 << 15)
        check(x, s, 6, 3, flagged=1)
        x[1] = value
        check(x, s, 6, 3, flagged=1)
    for value in (math.nan, math.inf):
        x, s = rows(6, 100, dtype, 8)
        s[4] = value
        check(x, s, 6, 3, flagged=1)
        check(x, s, 2, 3, finished=torch.ones(6, dtype=torch.bool, device="cuda"), end_token=5, flagged=1)


def test_in_place_and_other_stream():
    x, s = rows(12, 30011, torch.bfloat16, 9)
    done = torch.zeros(12, dtype=torch.bool, device="cuda")
    done[3] = True
    want = bm.beam_select(x, s, 4, beams=4, finished=done, end_token=9)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    other = bm.beam_select(x, s, 4, beams=4, finished=done, end_token=9, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    assert len(bm.bitmm_last_launches()) == 2
    parents, tokens = (torch.empty(3, 4, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.empty(bm.bitmm_beam_select_workspace_bytes(3, 4, 30011, 4, torch.bfloat16), dtype=torch.uint8, device="cuda")
    bm.bitmm_beam_select(x, s, s.view(3, 4), parents, tokens, ws, beams=4, finished=done, finished_out=done.view(3, 4), end_token=9)
    assert all(torch.equal(a, b) for a, b in zip(want, (s.view(3, 4), parents, tokens, done.view(3, 4))))


def test_captured():
    """Replays over new logits and a workspace that something else has written to."""
    x, s = rows(8, 20003, torch.bfloat16, 10)
    outs = [torch.empty(2, 4, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    ws = torch.empty(bm.bitmm_beam_select_workspace_bytes(2, 4, 20003, 4, torch.bfloat16), dtype=torch.uint8, device="cuda")
    call = lambda: bm.bitmm_beam_select(x, s, *outs, ws, beams=4)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        new, score = rows(8, 20003, torch.bfloat16, 20 + i)
        x.copy_(new)
        s.copy_(score)
        ws.fill_(255 * (i % 2))
        graph.replay()
        torch.cuda.synchronize()
        want = reference(x, s, 4, 4)
        assert torch.equal(outs[1].cpu().long(), want[1]) and torch.equal(outs[2].cpu().long(), want[2])
