"""The attention block where it can go wrong: tiny groups, other streams, wide windows, evicted pages,
tokens of extreme size beside the ones a row sees, weight that sits on one token, and each token of long
contexts counted. Against 64 bits; tests/attn_util.py derives the tolerances that are not derived here."""

import math

import pytest
import torch

import bit_matmul_amd as bm
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
