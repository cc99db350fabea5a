"""The attention block where it can go wrong, without a GPU."""

import pytest
import torch

import bit_matmul_amd as bm
from tests import attn_exact as X


def test_host_tensors_are_refused_on_any_stream():
    """A stream that is named does not make a host pointer one of the device's."""
    bf16, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    c = bm.KVCache.empty(3, 16, 2, 64, 32, device="cpu")
    k, slots = torch.zeros(4, 2, 64, **bf16), torch.zeros(4, dtype=torch.int64)
    q = torch.zeros(2, 4, 64, **bf16)
    table, lens, cu = torch.zeros(2, 3, **i32), torch.ones(2, **i32), torch.arange(3, **i32)
    x, w, s = torch.zeros(2, 64, **bf16), torch.zeros(8, 8, **i32), torch.zeros(8, 1, **bf16)
    e, eid = torch.zeros(1, 8, 8, **i32), torch.zeros(2, **i32)
    calls = [
        lambda **o: bm.bitmm_kv_append(k, k, slots, c, **o),
        lambda **o: bm.bitmm_kv_read(c, slots, k, k, **o),
        lambda **o: bm.kv_read(c, slots, **o),
        lambda **o: bm.bitmm_kv_attention(q, c, table, lens, cu, torch.zeros(2, 4, 64), None, max_q=1, max_kv=48, **o),
        lambda **o: bm.kv_attention(q, c, table, lens, cu, max_q=1, max_kv=48, **o),
        lambda **o: bm.bitmm_qk_norm_rope(q, None, None, None, None, None, q, None, **o),
        lambda **o: bm.qk_norm_rope(q, None, None, None, None, None, **o),
        lambda **o: bm.bitmm_qmm(x, w, s, s, torch.zeros(2, 8, **bf16), 4, **o),
        lambda **o: bm.qmv(x, w, s, s, 4, **o),
        lambda **o: bm.gather_qmm(x, e, s[None], s[None], eid, 4, **o),
        lambda **o: bm.gather_mm(x, torch.zeros(1, 8, 64, **bf16), None, eid, **o),
    ]
    for call in calls:
        for options in ({}, dict(stream=0), dict(stream=0x1000)):
            with pytest.raises(ValueError, match="GPU|cuda"):
                call(**options)


@pytest.mark.parametrize("window, sinks", X.WINDOWS)
@pytest.mark.parametrize("name", [n for n in X.CASES if not n[0].isdigit()])
def test_a_lost_step_shows(name, window, sinks):
    """The tolerances of tests/attn_exact.py are passed by any 32 tokens that are left out of the longest sequence, in
    the output and in the lse of every row that sees one of them."""
    seq = X.case(name)
    b = max(range(len(seq.lens)), key=lambda i: seq.lens[i][1])
    runs, total = seq.counts(b, window, sinks)
    want, lse = seq.expected(b, 0, runs, total)
    steps = -(-seq.lens[b][1] // X.STEP)
    for lost in sorted({0, 1, steps // 3, steps // 2, steps - 2, steps - 1}):
        less, left = seq.counts(b, window, sinks, lost)
        out, short = seq.expected(b, 0, less, left)
        sees = (runs - less).sum(-1) > 0
        assert ((short - lse)[sees].abs() > 4 * X.LSE).all()
        assert (((out - want).abs() > 4 * X.OUT * want).any(-1))[sees & (left > 0)].all()
