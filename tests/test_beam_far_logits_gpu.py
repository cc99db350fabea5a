"""Beam search's selection over logits of any finite size: masks far below the rest, whole rows of one, and rows whose
every logit is large."""

import pytest
import torch

import bit_matmul_amd as bm
from tests import test_beam_select_gpu as S

pytestmark = pytest.mark.gpu

SIZES = [1e6, 1e8, 1e12, 1e18, 9e19, 1e20, 1e21, 1e22, 3.3e23, 2e25, 1e30, 1e37]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bm.lib()
    yield
    torch.cuda.synchronize()


def reference(x, scores, k, beams):
    """(totals f64, parents, tokens). The row's largest is taken off before the logarithm: that added to a large logit would
    take 2^-53 of the logit from the sum. Within a beam the order is that of the logits."""
    x, s, out = x.cpu().double(), scores.cpu().double(), []
    for g in range(x.shape[0] // beams):
        found = []
        for b in range(beams):
            r = g * beams + b
            top = x[r].max()
            total = s[r] + ((x[r] - top) - torch.exp(x[r] - top).sum().log())
            order = torch.sort(x[r], descending=True, stable=True)[1][:k].tolist()
            found += [(-total[t].item(), b, i, t) for i, t in enumerate(order)]
        out.append([(-t, b, v) for t, b, _, v in sorted(found)[:k]])
    total, parents, tokens = ([[c[i] for c in row] for row in out] for i in range(3))
    return torch.tensor(total, dtype=torch.float64), torch.tensor(parents), torch.tensor(tokens)


def check(x, s, k, beams):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = bm.beam_select(x, s, k, beams=beams, status=status)
    want = reference(x, s, k, beams)
    assert status.item() == 0
    assert torch.equal(got[1].cpu().long(), want[1]) and torch.equal(got[2].cpu().long(), want[2])
    assert not torch.isinf(got[0]).any()
    # one rounding to f32, and 2^-30 for the f64 sum's exponentials (4e-11 each, brought to another reference twice)
    # and logarithm
    off = (got[0].cpu().double() - want[0]).abs()
    assert (off <= 2.0 ** -24 * want[0].abs() + 2.0 ** -30).all()


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_masks_of_any_size(dtype, size):
    """Logits of -size at the start, in the middle and all but at the end of rows: they weigh nothing."""
    x, s = S.rows(5, 9001, dtype, 11)
    x[0, :1024] = -size
    x[1, :8500] = -size
    x[2, 2048:7000] = -size
    x[3, ::2] = -size
    x[4, -1] = -size
    check(x, s, 8, 5)
    check(x, s, 8, 1)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_rows_of_one_size(dtype, size):
    """Rows all of which is -size, or size: each logit weighs as much as any other."""
    for vocab in (5, 700, 9001):
        x, s = S.rows(4, vocab, dtype, 12)
        x[0] = -size
        x[2] = size
        check(x, s, 4, 4)
        check(x, s, 4, 1)
        x[1, vocab // 2] = -size
        x[3, vocab // 2] = size
        check(x, s, 4, 1)


@pytest.mark.parametrize("centre", [1e6, -1e6, 1e8, -1e8])
def test_differences_of_large_logits(centre):
    """Few steps of f32 apart: differences, and so totals, are as of small logits."""
    g = torch.Generator().manual_seed(13)
    step = 8.0 if abs(centre) > 1e7 else 0.0625
    x = (centre + step * torch.randint(-40, 3, (6, 20011), generator=g)).float().cuda()
    s = (-6 * torch.rand(6, generator=g)).cuda()
    check(x, s, 10, 3)
    check(x, s, 10, 1)


@pytest.mark.parametrize("size", [6e4, 1e4, 300.0])
def test_binary16(size):
    x, s = S.rows(4, 9001, torch.float16, 14)
    x[0, :5000] = -size
    x[1] = -size
    x[2] = size
    x[3, 100] = size
    for beams in (1, 4):
        check(x, s, 6, beams)
