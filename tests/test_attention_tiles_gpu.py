"""The attention kernel for many query rows at small sizes. The host's bounds of the lengths, not the
lengths, decide which kernel runs: wide ones send the checks of test_attention_gpu.py through it, with
a row tile's tokens in one piece or (where no window keeps them few) split over workgroups."""

import pytest
import torch

import bit_matmul_amd as bm
from tests import test_attention_gpu as T

pytestmark = pytest.mark.gpu

BOUNDS = {"whole": dict(max_q=8192, max_kv=2047), "split": dict(max_q=130, max_kv=65536)}


@pytest.fixture(params=list(BOUNDS), autouse=True)
def wide_bounds(request, monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    attend = T.attend

    def wide(seq, cache, out_dtype, **kw):
        bounds = BOUNDS["whole" if kw.get("window") else request.param]
        kw.setdefault("max_q", max(bounds["max_q"], max(q for q, _ in seq.lens)))
        kw.setdefault("max_kv", max(bounds["max_kv"], max(kv for _, kv in seq.lens)))
        y = attend(seq, cache, out_dtype, **kw)
        assert bm.bitmm_last_launches()[0].startswith("attention_tiles_kernel<")
        return y

    monkeypatch.setattr(T, "attend", wide)


@pytest.mark.parametrize("dtype", [T.BF16, T.F16])
@pytest.mark.parametrize("shape", T.SHAPES, ids=str)
@pytest.mark.parametrize("lens", list(T.LENGTHS), ids=str)
def test_attention(dtype, shape, lens):
    T.test_attention(dtype, shape, lens)


@pytest.mark.parametrize("out", [T.BF16, T.F16, T.F32])
@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (16, 4), (33, 70), (64, 0), (200, 5), (1900, 3)])
@pytest.mark.parametrize("lens", ["decode", "chunks"], ids=str)
def test_window_and_first_tokens(out, window, sinks, lens):
    T.test_window_and_first_tokens(out, window, sinks, lens)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales_of_scores(scale):
    T.test_scales_of_scores(scale)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 300.0, 1e6, 1e30])
@pytest.mark.parametrize("lens", [[(1, 500)], [(80, 200)]], ids=str)
def test_ranges_beyond_binary16(size, lens):
    T.test_ranges_beyond_binary16(size, lens)


def test_growing_range():
    T.test_growing_range()


@pytest.mark.parametrize("lens", [[(1, 75), (1, 0), (1, 40)], [(50, 75), (50, 50)]], ids=str)
@pytest.mark.parametrize("window", [0, 20])
def test_stale_slots_do_not_matter(lens, window):
    T.test_stale_slots_do_not_matter(lens, window)


@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("lens", [[(1, 200)], [(100, 200)]], ids=str)
def test_not_finite_where_masked_and_where_seen(side, lens):
    T.test_not_finite_where_masked_and_where_seen(side, lens)


def test_rows_that_see_nothing():
    T.test_rows_that_see_nothing()


@pytest.mark.parametrize("lens", [[(1, 100), (1, 100)], [(60, 100), (33, 100)]], ids=str)
def test_bad_pages(lens):
    T.test_bad_pages(lens)


@pytest.mark.parametrize("lens", [[(1, 700), (2, 90)], [(90, 700)], [(90, 100), (70, 3000)]], ids=str)
@pytest.mark.parametrize("D, power", [(64, 8), (128, 8), (256, 12), (128, -10)])
def test_scores_of_millions(lens, D, power):
    T.test_scores_of_millions(lens, D, power)
