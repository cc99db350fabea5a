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


def test_shared_attention_without_a_workspace():
    """None is taken where the call needs none, and refused where it does."""
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(2)
    c = bm.KVCache.empty(5, 16, 2, 64, 32)
    k, v = (torch.randn(80, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    bm.bitmm_kv_append(k, v, torch.arange(80, device="cuda"), c)
    q = torch.randn(2, 4, 64, generator=g).bfloat16().cuda()
    there = (torch.tensor([[2, 0, 1]], **i32), torch.tensor([40], **i32), torch.tensor([0, 2], **i32),
             torch.tensor([[3], [4]], **i32), torch.tensor([5, 9], **i32), torch.arange(3, **i32))
    sizes = dict(max_group_q=2, max_prefix=48, max_q=1, max_kv=16)
    want = bm.kv_attention_shared(q, c, *there, **sizes)
    out = torch.empty_like(q)
    assert bm.bitmm_kv_attention_shared_workspace_bytes(2, 2, 1, *sizes.values(), 4, 2, 64) == 0
    assert bm.bitmm_kv_attention_shared(q, c, *there, out, None, **sizes) is out and torch.equal(out, want)
    with pytest.raises(bm.BitmmError):
        bm.bitmm_kv_attention_shared(q, c, *there, out, None, **{**sizes, "max_prefix": 4096})
