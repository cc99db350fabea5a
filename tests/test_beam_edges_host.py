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
