"""The calls of include/bitmm_beam.h where their bindings can go wrong, without a GPU."""

import pytest
import torch

import bit_matmul_amd as bm

BF = dict(dtype=torch.bfloat16)
I32 = dict(dtype=torch.int32)


def test_keys_alone_in_the_allocating_form():
    """q of None leaves the queries out, as in the form that takes outputs: on host tensors it gets as far as that."""
    c = bm.KVCache.empty(3, 16, 2, 64, 32, device="cpu")
    k, slots = torch.zeros(4, 2, 64, **BF), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="on the GPU"):
        bm.qk_norm_rope_append(None, k, k, None, None, None, None, slots, c)
    with pytest.raises(ValueError, match="on the GPU"):
        bm.bitmm_qk_norm_rope_append(None, k, k, None, None, None, None, None, slots, c)


def test_shared_attention_without_a_workspace():
    """None, where a call needs none, as bitmm_kv_attention takes it: on host tensors it gets as far as that."""
    c = bm.KVCache.empty(3, 16, 2, 64, 32, device="cpu")
    q, two, cu = torch.zeros(2, 4, 64, **BF), torch.ones(2, **I32), torch.arange(3, **I32)
    table = torch.zeros(2, 1, **I32)
    assert bm.bitmm_kv_attention_shared_workspace_bytes(2, 2, 1, 2, 16, 1, 1, 4, 2, 64) == 0
    with pytest.raises(ValueError, match="on the GPU"):
        bm.bitmm_kv_attention_shared(q, c, table[:1], two[:1], torch.tensor([0, 2], **I32), table, two, cu, torch.zeros_like(q), None,
                                     max_group_q=2, max_prefix=16, max_q=1, max_kv=1)
