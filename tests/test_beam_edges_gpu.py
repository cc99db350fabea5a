"""The calls of include/bitmm_beam.h at the edges of what their bindings take, on the GPU."""

import pytest
import torch

import bit_matmul_amd as bm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bm.lib()
    yield
    torch.cuda.synchronize()


def test_keys_alone_in_the_allocating_form():
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(20, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    slots = torch.randperm(48, generator=g)[:20].cuda()
    a, b = (bm.KVCache(*(torch.zeros_like(t) for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)))
            for c in [bm.KVCache.empty(3, 16, 2, 64, 32)] for _ in range(2))
    assert bm.qk_norm_rope_append(None, k, v, None, None, None, None, slots, a) is None
    bm.bitmm_qk_norm_rope_append(None, k, v, None, None, None, None, None, slots, b)
    for side in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a, side), getattr(b, side)) and getattr(a, side).any()
