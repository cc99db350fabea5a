"""Refusals of the calls of include/bitmm_beam.h, without a GPU: each bad argument is turned down with
its status before the device is touched. Pointers are made up: validation follows none."""

import os
import re

import pytest
import torch

import bit_matmul_amd as bm
from bit_matmul_amd import attention as A
from tests.test_attention_host import CACHE_FAULTS, P, cache, status

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    return bm.lib()


def test_exports_every_declared_function(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "bitmm_beam.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(bitmm_\w+)\s*\(", text))
    assert names
    for n in names:
        assert hasattr(L, n) and n in bm.__all__


def rope_append(L, desc="", **kw):
    d = dict(q=P, qs=1024, k=P, ks=256, v=P, vs=256, qw=P, kw=P, pos=P, freq=P, qo=P, qos=1024, slots=P,
             cache=cache() if desc == "" else desc, T=4, hq=8, rot=128, il=0, eps=1e-6, off=0.0, scale=1.0, dtype=0,
             status=None, stream=None)
    d.update(kw)
    return L.bitmm_qk_norm_rope_append(*d.values())


@pytest.mark.parametrize("kw, want", [
    (dict(dtype=2), "UNSUPPORTED"), (dict(T=-1), "SHAPE"), (dict(hq=-1), "SHAPE"), (dict(rot=136), "SHAPE"),
    (dict(rot=-8), "SHAPE"), (dict(rot=12), "SHAPE"), (dict(T=2 ** 30), "SHAPE"), (dict(T=2 ** 24 + 1), "SHAPE"),
    (dict(hq=2 ** 29), "SHAPE"), (dict(qs=1016), "SHAPE"), (dict(ks=248), "SHAPE"), (dict(vs=248), "SHAPE"),
    (dict(qs=1028), "ALIGN"), (dict(vs=260), "ALIGN"), (dict(q=P + 2), "ALIGN"), (dict(v=P + 8), "ALIGN"),
    (dict(qo=P + 8), "ALIGN"), (dict(qw=P + 1), "ALIGN"), (dict(pos=P + 2), "ALIGN"), (dict(freq=P + 1), "ALIGN"),
    (dict(slots=P + 4), "ALIGN"), (dict(status=P + 2), "ALIGN"), (dict(q=None), "NULL"), (dict(qo=None), "NULL"),
    (dict(k=None), "NULL"), (dict(v=None), "NULL"), (dict(slots=None), "NULL"), (dict(pos=None), "NULL"),
    (dict(freq=None), "NULL"), (dict(desc=None), "NULL"),
])
def test_rope_append_refusals(L, kw, want):
    assert rope_append(L, **kw) == status(want)
    assert bm.bitmm_last_launches() == []


@pytest.mark.parametrize("kw, want", CACHE_FAULTS)
def test_rope_append_cache_faults(L, kw, want):
    assert rope_append(L, desc=cache(**kw)) == status(want)


def test_rope_append_empty_and_without_a_device(L):
    assert rope_append(L, T=0, q=None, k=None, v=None, slots=None) == bm.BITMM_OK
    if not torch.cuda.is_available():
        assert rope_append(L) == bm.BITMM_ERR_DEVICE
        assert rope_append(L, hq=0, q=None, qo=None, rot=0, pos=None, freq=None, qw=None, kw=None) == bm.BITMM_ERR_DEVICE


class _Host:
    """What the binding asks of a cache, without device memory."""
    kv_heads, head_dim, group_size, page_size, device_index = 2, 64, 32, 16, -1
    desc = None


def test_binding_refuses():
    bf, i64, i32 = torch.bfloat16, torch.int64, torch.int32
    q, k, v = (torch.zeros(3, n, 64, dtype=bf) for n in (4, 2, 2))
    slots, pos, freq = torch.zeros(3, dtype=i64), torch.zeros(3, dtype=i32), torch.zeros(32)

    def call(q=q, k=k, v=v, qw=None, kw=None, pos=pos, freq=freq, q_out=q, slots=slots):
        return bm.bitmm_qk_norm_rope_append(q, k, v, qw, kw, pos, freq, q_out, slots, _Host())

    for error, kw in [(TypeError, dict(k=k.float())), (TypeError, dict(v=v.half())), (TypeError, dict(q=q.half())),
                      (TypeError, dict(slots=slots.int())), (TypeError, dict(pos=pos.long())), (TypeError, dict(freq=freq.half())),
                      (ValueError, dict(k=k[:2])), (ValueError, dict(v=v[:, :1])), (ValueError, dict(q=q[:, :, :32])),
                      (ValueError, dict(q=None)), (ValueError, dict(q_out=None)), (ValueError, dict(pos=pos[:2])),
                      (ValueError, dict(qw=torch.zeros(32, dtype=bf))), (ValueError, dict(k=k.transpose(0, 1).contiguous().transpose(0, 1))),
                      (ValueError, {})]:   # the last: tensors that are not on the GPU
        with pytest.raises(error):
            call(**kw)


def select(L, **kw):
    d = dict(logits=P, stride=1000, scores=P, fin=P, so=P, par=P, tok=P, fo=P, G=3, K=4, V=1000, k=8, end=2, type=0, ws=P,
             ws_bytes=1 << 30, status=None, stream=None)
    d.update(kw)
    return L.bitmm_beam_select(*d.values())


@pytest.mark.parametrize("kw, want", [
    (dict(type=3), "UNSUPPORTED"), (dict(type=-1), "UNSUPPORTED"), (dict(G=-1), "SHAPE"), (dict(G=2 ** 20 + 1), "SHAPE"), (dict(G=2 ** 62), "SHAPE"),
    (dict(K=0), "SHAPE"), (dict(K=65), "SHAPE"), (dict(V=0), "SHAPE"), (dict(V=2 ** 30 + 1), "SHAPE"), (dict(k=0), "SHAPE"),
    (dict(k=65), "SHAPE"), (dict(stride=999), "SHAPE"), (dict(logits=None), "NULL"), (dict(scores=None), "NULL"),
    (dict(so=None), "NULL"), (dict(par=None), "NULL"), (dict(tok=None), "NULL"), (dict(logits=P + 1), "ALIGN"),
    (dict(logits=P + 2, type=1), "ALIGN"), (dict(scores=P + 2), "ALIGN"), (dict(so=P + 1), "ALIGN"), (dict(par=P + 2), "ALIGN"),
    (dict(tok=P + 2), "ALIGN"), (dict(status=P + 1), "ALIGN"), (dict(ws=P + 8), "ALIGN"), (dict(ws=None), "WORKSPACE"),
    (dict(ws_bytes=100), "WORKSPACE"),
])
def test_select_refusals(L, kw, want):
    assert select(L, **kw) == status(want)
    assert bm.bitmm_last_launches() == []


def test_select_empty_and_workspace(L):
    assert select(L, G=0, logits=None, ws=None) == bm.BITMM_OK
    need = bm.bitmm_beam_select_workspace_bytes
    assert need(0, 4, 1000, 8, torch.float32) == 0 and need(1, 65, 1000, 8, torch.float32) == 0
    for groups, beams, vocab, k in [(1, 1, 1, 1), (1, 4, 32000, 4), (300, 64, 131072, 64), (1 << 16, 64, 1 << 30, 64)]:
        for dtype in (torch.bfloat16, torch.float32):
            n = need(groups, beams, vocab, k, dtype)
            # a part of a row has a sum and k pairs, and a row at most 64 parts
            assert groups * beams * (16 + 8 * k) <= n <= 64 * groups * beams * (16 + 8 * k)
            if not torch.cuda.is_available():
                assert select(L, G=groups, K=beams, V=vocab, stride=vocab, k=k, type=1 if dtype is torch.float32 else 0,
                              ws_bytes=n) == bm.BITMM_ERR_DEVICE
                assert select(L, G=groups, K=beams, V=vocab, stride=vocab, k=k, type=1 if dtype is torch.float32 else 0,
                              ws_bytes=n - 1) == bm.BITMM_ERR_WORKSPACE


def test_select_binding_refuses():
    f32, i32 = torch.float32, torch.int32
    logits, scores = torch.zeros(6, 50), torch.zeros(6)
    so, par, tok = torch.zeros(2, 3), torch.zeros(2, 3, dtype=i32), torch.zeros(2, 3, dtype=i32)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)

    def call(logits=logits, scores=scores, so=so, par=par, tok=tok, ws=ws, **kw):
        return bm.bitmm_beam_select(logits, scores, so, par, tok, ws, **{"beams": 3, **kw})

    for error, kw in [(TypeError, dict(logits=logits.double())), (TypeError, dict(scores=scores.half())),
                      (TypeError, dict(tok=tok.long())), (TypeError, dict(finished=torch.zeros(6, dtype=torch.uint8))),
                      (ValueError, dict(beams=2)), (ValueError, dict(scores=scores[:5])), (ValueError, dict(so=so[:, :2])),
                      (ValueError, dict(logits=torch.zeros(50, 6).t())), (ValueError, dict(par=par[0])), (ValueError, dict(ws=ws[::2])),
                      (ValueError, dict(finished=torch.zeros(2, 3, dtype=torch.bool))), (ValueError, {})]:
        with pytest.raises(error):
            call(**kw)
    with pytest.raises(ValueError):
        bm.beam_select(logits, scores, 3, beams=4)


def reorder(L, n=3, caches=None, **kw):
    array = (A._CacheDesc * n)(*(caches or [cache(num_pages=1000)] * n))
    d = dict(caches=array, layers=n, table=P, table_out=P + 4096, pages=8, lens=P, lens_out=P, parents=P, slots=P, G=4, K=4,
             first=3, each=32, ws=P, ws_bytes=256, status=None, stream=None)
    d.update(kw)
    return L.bitmm_kv_beam_reorder(*d.values())


@pytest.mark.parametrize("kw, want", [
    (dict(caches=None), "NULL"), (dict(layers=0), "SHAPE"), (dict(layers=4097), "SHAPE"), (dict(G=-1), "SHAPE"),
    (dict(G=2 ** 20 + 1), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=65), "SHAPE"), (dict(pages=0), "SHAPE"),
    (dict(pages=2 ** 22 + 1), "SHAPE"), (dict(first=-1), "SHAPE"), (dict(first=1001), "SHAPE"), (dict(each=-1), "SHAPE"),
    (dict(each=250), "SHAPE"), (dict(first=873), "SHAPE"), (dict(each=2 ** 18 + 1), "SHAPE"), (dict(table=None), "NULL"),
    (dict(table_out=None), "NULL"), (dict(lens=None), "NULL"), (dict(lens_out=None), "NULL"), (dict(parents=None), "NULL"),
    (dict(slots=None), "NULL"), (dict(table=P + 2), "ALIGN"), (dict(lens_out=P + 1), "ALIGN"), (dict(slots=P + 4), "ALIGN"),
    (dict(status=P + 2), "ALIGN"), (dict(ws=P + 8), "ALIGN"), (dict(ws=None), "WORKSPACE"), (dict(ws_bytes=255), "WORKSPACE"),
])
def test_reorder_refusals(L, kw, want):
    if "caches" in kw:
        assert L.bitmm_kv_beam_reorder(None, 1, P, P, 8, P, P, P, P, 4, 4, 3, 32, P, 256, None, None) == status(want)
    else:
        assert reorder(L, **kw) == status(want)
    assert bm.bitmm_last_launches() == []


def test_reorder_caches(L):
    for kw, want in CACHE_FAULTS:
        faulty = [cache(num_pages=1000), cache(**{"num_pages": 1000, **kw})]
        assert reorder(L, n=2, caches=faulty) == status(want)
    for kw in (dict(num_pages=1001), dict(page_size=32), dict(kv_heads=3), dict(head_dim=64), dict(group_size=32)):
        assert reorder(L, n=2, caches=[cache(num_pages=1000), cache(**{"num_pages": 1000, **kw})]) == status("SHAPE")
    assert reorder(L, G=0, table=None) == bm.BITMM_OK
    assert bm.bitmm_kv_beam_reorder_workspace_bytes(4, 4) == 256 and bm.bitmm_kv_beam_reorder_workspace_bytes(4, 65) == 0
    if not torch.cuda.is_available():
        assert reorder(L) == bm.BITMM_ERR_DEVICE
        assert reorder(L, first=872) == bm.BITMM_ERR_DEVICE


def test_reorder_binding_refuses():
    i32, i64 = torch.int32, torch.int64
    with pytest.raises(ValueError):
        bm.KVLayers([])

    class Layers:
        caches, desc, device_index, page_size = [None], None, -1, 16

    table, lens, parents = torch.zeros(6, 4, dtype=i32), torch.zeros(6, dtype=i32), torch.zeros(2, 3, dtype=i32)
    slots, ws = torch.zeros(6, dtype=i64), torch.zeros(96, dtype=torch.uint8)

    def call(table=table, lens=lens, parents=parents, table_out=table, lens_out=lens, slots=slots, ws=ws):
        return bm.bitmm_kv_beam_reorder(Layers(), table, lens, parents, table_out, lens_out, slots, ws, first_page=0, pages_per_group=4)

    for error, kw in [(TypeError, dict(table=table.long())), (TypeError, dict(slots=slots.int())), (ValueError, dict(parents=parents[0])),
                      (ValueError, dict(parents=parents[:1])), (ValueError, dict(lens=lens[:5])), (ValueError, dict(table_out=table[:, :3])),
                      (TypeError, dict(parents=parents.long())), (ValueError, dict(ws=ws[::2])), (ValueError, {})]:
        with pytest.raises(error):
            call(**kw)


def shared(L, desc="", **kw):
    d = dict(q=P, qs=1024, cache=cache() if desc == "" else desc, pt=P, pp=4, pl=P, cg=P, table=P, pages=4, lens=P, cu=P, out=P,
             os=1024, lse=P, T=12, B=6, G=2, hq=8, mgq=6, mp=100, mq=2, mkv=50, scale=0.1, dtype=0, otype=0, ws=P, ws_bytes=1 << 40,
             status=None, stream=None)
    d.update(kw)
    return L.bitmm_kv_attention_shared(*d.values())


@pytest.mark.parametrize("kw, want", [
    (dict(desc=None), "NULL"), (dict(dtype=2), "UNSUPPORTED"), (dict(otype=3), "UNSUPPORTED"), (dict(T=-1), "SHAPE"), (dict(B=-1), "SHAPE"),
    (dict(G=-1), "SHAPE"), (dict(hq=0), "SHAPE"), (dict(hq=7), "SHAPE"), (dict(mgq=-1), "SHAPE"), (dict(mp=-1), "SHAPE"),
    (dict(mp=2 ** 31 - 1), "SHAPE"), (dict(mq=-1), "SHAPE"), (dict(mkv=2 ** 31), "SHAPE"), (dict(pp=-1), "SHAPE"), (dict(pages=2 ** 31), "SHAPE"),
    (dict(mgq=2 ** 30), "SHAPE"), (dict(hq=130, qs=130 * 128, os=130 * 128), "UNSUPPORTED"), (dict(B=65536), "UNSUPPORTED"),
    (dict(G=65536), "UNSUPPORTED"), (dict(qs=1016), "SHAPE"), (dict(os=1020), "SHAPE"), (dict(qs=1028), "ALIGN"), (dict(q=None), "NULL"),
    (dict(out=None), "NULL"), (dict(pt=None), "NULL"), (dict(pl=None), "NULL"), (dict(cg=None), "NULL"), (dict(table=None), "NULL"),
    (dict(lens=None), "NULL"), (dict(cu=None), "NULL"), (dict(q=P + 8), "ALIGN"), (dict(pt=P + 2), "ALIGN"), (dict(pl=P + 2), "ALIGN"),
    (dict(cg=P + 1), "ALIGN"), (dict(lse=P + 2), "ALIGN"), (dict(ws=P + 8), "ALIGN"), (dict(status=P + 2), "ALIGN"),
    (dict(ws=None, mp=5000), "WORKSPACE"), (dict(ws_bytes=100, mp=5000), "WORKSPACE"), (dict(B=60000, T=2 ** 24, mq=2 ** 16), "UNSUPPORTED"),
])
def test_shared_refusals(L, kw, want):
    assert shared(L, **kw) == status(want)
    assert bm.bitmm_last_launches() == []


def test_shared_empty_and_workspace(L):
    for kw in (dict(T=0), dict(B=0), dict(mq=0)):
        assert shared(L, **kw, q=None, out=None, ws=None) == bm.BITMM_OK
    for kw, want in CACHE_FAULTS:
        assert shared(L, desc=cache(**kw)) == status(want)
    need = bm.bitmm_kv_attention_shared_workspace_bytes
    assert need(12, 6, 2, 6, 100, 2, 50, 7, 2, 128) == 0 and need(12, 6, 2, 6, 100, 2, 50, 8, 2, 96) == 0 and need(0, 6, 2, 6, 100, 2, 50, 8, 2, 128) == 0
    for G, mgq, mp, mkv in ((0, 0, 0, 50), (2, 0, 0, 0), (2, 6, 0, 0), (2, 6, 100, 50), (1, 12, 10 ** 6, 0), (6, 2, 1, 10 ** 6)):
        n = need(12, 6, G, mgq, mp, 2, mkv, 8, 2, 128)
        # a partial result of each query row over the shared tokens at least, where these are a pass of their own
        assert n >= 4 * 130 * 2 * G * mgq * 4 or (n == 0 and max(mp, mkv) <= 1280)
        if not torch.cuda.is_available():
            kw = dict(G=G, mgq=mgq, mp=mp, mkv=mkv, ws_bytes=n)
            if G == 0:
                kw.update(pt=None, pl=None, cg=None)
            assert shared(L, **kw) == bm.BITMM_ERR_DEVICE
            if n:
                assert shared(L, **{**kw, "ws_bytes": n - 1}) == bm.BITMM_ERR_WORKSPACE


def test_shared_binding_refuses():
    i32, bf = torch.int32, torch.bfloat16
    q, out = torch.zeros(6, 4, 64, dtype=bf), torch.zeros(6, 4, 64, dtype=bf)
    pt, pl, cg = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32)
    table, lens, cu, ws = torch.zeros(6, 2, dtype=i32), torch.zeros(6, dtype=i32), torch.zeros(7, dtype=i32), torch.zeros(1 << 20, dtype=torch.uint8)

    def call(q=q, pt=pt, pl=pl, cg=cg, table=table, lens=lens, cu=cu, out=out, ws=ws, lse=None):
        return bm.bitmm_kv_attention_shared(q, _Host(), pt, pl, cg, table, lens, cu, out, ws, max_group_q=3, max_prefix=40, max_q=1,
                                            max_kv=30, lse=lse)

    for error, kw in [(TypeError, dict(q=q.float())), (TypeError, dict(out=out.double())), (ValueError, dict(q=q[:, :, :32])),
                      (ValueError, dict(out=out[:5])), (ValueError, dict(pt=pt[0])), (ValueError, dict(pt=pt[:1])), (TypeError, dict(pl=pl.long())),
                      (ValueError, dict(cg=cg[:2])), (ValueError, dict(table=table[0])), (ValueError, dict(table=table[:5])),
                      (ValueError, dict(cu=cu[:6])), (ValueError, dict(ws=ws[::2])), (ValueError, dict(lse=torch.zeros(6, 3))),
                      (ValueError, {})]:
        with pytest.raises(error):
            call(**kw)
