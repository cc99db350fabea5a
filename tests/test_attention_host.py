"""Refusals of the attention block, without a GPU: each bad argument is turned down with its
status before the device is touched. Pointers are made up: validation follows none."""

import ctypes
import os
import re

import pytest
import torch

import bit_matmul_amd as bm
from bit_matmul_amd import attention as A
from tests import attn_util as U

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    return bm.lib()


def test_exports_every_declared_function(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "bitmm_attn.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(bitmm_\w+)\s*\(", text))
    assert names == {"bitmm_qk_norm_rope", "bitmm_kv_append", "bitmm_kv_read", "bitmm_kv_attention_workspace_bytes",
                     "bitmm_kv_attention"}
    for n in names:
        assert hasattr(L, n) and n in bm.__all__


P = 0x10000  # 16-byte aligned


def cache(**kw):
    d = dict(k_codes=P, k_scales=P, v_codes=P, v_scales=P, num_pages=10, page_size=64, kv_heads=2, head_dim=128,
             group_size=64)
    d.update(kw)
    return A._CacheDesc(*d.values())


CACHE_FAULTS = [
    (dict(num_pages=0), "SHAPE"), (dict(num_pages=2 ** 31), "SHAPE"), (dict(kv_heads=0), "SHAPE"),
    (dict(kv_heads=70000), "SHAPE"), (dict(page_size=0), "UNSUPPORTED"), (dict(page_size=48), "UNSUPPORTED"),
    (dict(page_size=8), "UNSUPPORTED"), (dict(head_dim=96), "UNSUPPORTED"), (dict(group_size=16), "UNSUPPORTED"),
    (dict(head_dim=64, group_size=128), "UNSUPPORTED"), (dict(k_codes=None), "NULL"), (dict(v_scales=None), "NULL"),
    (dict(k_scales=P + 8), "ALIGN"), (dict(v_codes=P + 4), "ALIGN"),
]


def status(name):
    return getattr(bm, "BITMM_ERR_" + name)


def rope(L, **kw):
    d = dict(q=P, qs=1024, k=P, ks=256, qw=P, kw=P, pos=P, freq=P, qo=P, qos=1024, ko=P, kos=256, T=4, hq=8, hk=2,
             D=128, rot=128, il=0, eps=1e-6, off=0.0, scale=1.0, dtype=0, stream=None)
    d.update(kw)
    return L.bitmm_qk_norm_rope(*d.values())


@pytest.mark.parametrize("kw, want", [
    (dict(dtype=2), "UNSUPPORTED"), (dict(D=96), "UNSUPPORTED"), (dict(T=-1), "SHAPE"), (dict(hq=-1), "SHAPE"),
    (dict(rot=132), "SHAPE"), (dict(rot=136), "SHAPE"), (dict(rot=-8), "SHAPE"), (dict(rot=12), "SHAPE"),
    (dict(T=2 ** 30), "SHAPE"), (dict(qs=1016), "SHAPE"), (dict(kos=248), "SHAPE"), (dict(qs=1028), "ALIGN"),
    (dict(q=P + 2), "ALIGN"), (dict(ko=P + 8), "ALIGN"), (dict(qw=P + 1), "ALIGN"), (dict(pos=P + 2), "ALIGN"),
    (dict(q=None), "NULL"), (dict(ko=None), "NULL"), (dict(pos=None), "NULL"), (dict(freq=None), "NULL"),
])
def test_rope_refusals(L, kw, want):
    assert rope(L, **kw) == status(want)
    assert bm.bitmm_last_launches() == []


def test_rope_empty(L):
    assert rope(L, T=0, q=None, k=None) == bm.BITMM_OK
    assert rope(L, hq=0, hk=0, q=None, k=None) == bm.BITMM_OK


def append(L, desc="", **kw):
    d = dict(k=P, ks=256, v=P, vs=256, slots=P, T=3, cache=cache() if desc == "" else desc, dtype=0, status=None,
             stream=None)
    d.update(kw)
    return L.bitmm_kv_append(*d.values())


def read(L, desc="", **kw):
    d = dict(cache=cache() if desc == "" else desc, slots=P, T=3, k=P, ks=256, v=P, vs=256, dtype=0, status=None,
             stream=None)
    d.update(kw)
    return L.bitmm_kv_read(*d.values())


@pytest.mark.parametrize("call", [append, read])
def test_cache_refusals(L, call):
    assert call(L, None) == bm.BITMM_ERR_NULL
    for kw, want in CACHE_FAULTS:
        assert call(L, cache(**kw)) == status(want), kw
        assert bm.bitmm_last_launches() == []
    for kw, want in [(dict(dtype=3), "UNSUPPORTED"), (dict(T=-1), "SHAPE"), (dict(T=2 ** 29), "SHAPE"),
                     (dict(ks=248), "SHAPE"), (dict(vs=260), "ALIGN"), (dict(k=P + 8), "ALIGN"),
                     (dict(slots=None), "NULL"), (dict(slots=P + 4), "ALIGN"), (dict(status=P + 2), "ALIGN")]:
        assert call(L, **kw) == status(want), kw
    assert call(L, T=0, slots=None) == bm.BITMM_OK


def test_append_needs_both_sides_and_read_takes_either(L):
    assert append(L, k=None) == bm.BITMM_ERR_NULL
    assert append(L, v=None) == bm.BITMM_ERR_NULL
    assert read(L, k=None, v=None) == bm.BITMM_OK


def attend(L, desc="", **kw):
    d = dict(q=P, qs=1024, cache=cache() if desc == "" else desc, table=P, pages=8, lens=P, cu=P, out=P, os=1024,
             lse=None, T=4, B=4, hq=8, max_q=1, max_kv=512, scale=0.1, window=0, sinks=0, dtype=0, otype=0, ws=None,
             wsb=0, status=None, stream=None)
    d.update(kw)
    return L.bitmm_kv_attention(*d.values())


@pytest.mark.parametrize("kw, want", [
    (dict(dtype=2), "UNSUPPORTED"), (dict(otype=3), "UNSUPPORTED"), (dict(T=-1), "SHAPE"), (dict(B=-1), "SHAPE"),
    (dict(max_q=-1), "SHAPE"), (dict(max_kv=-1), "SHAPE"), (dict(max_kv=2 ** 31 - 1), "SHAPE"), (dict(hq=7), "SHAPE"),
    (dict(hq=0), "SHAPE"), (dict(window=-1), "SHAPE"), (dict(sinks=-1), "SHAPE"), (dict(pages=-1), "SHAPE"),
    (dict(hq=130, qs=130 * 128, os=130 * 128), "UNSUPPORTED"), (dict(B=70000), "UNSUPPORTED"),
    (dict(q=None), "NULL"), (dict(out=None), "NULL"), (dict(table=None), "NULL"), (dict(lens=None), "NULL"),
    (dict(cu=None), "NULL"), (dict(qs=1000), "SHAPE"), (dict(os=1020), "SHAPE"), (dict(qs=1028), "ALIGN"),
    (dict(q=P + 8), "ALIGN"), (dict(out=P + 4), "ALIGN"), (dict(table=P + 1), "ALIGN"), (dict(lse=P + 2), "ALIGN"),
    (dict(status=P + 1), "ALIGN"), (dict(ws=P + 8), "ALIGN"),
])
def test_attention_refusals(L, kw, want):
    assert attend(L, **kw) == status(want)
    assert bm.bitmm_last_launches() == []


def test_attention_cache_refusals_and_empty(L):
    assert attend(L, None) == bm.BITMM_ERR_NULL
    for kw, want in CACHE_FAULTS:
        assert attend(L, cache(**kw)) == status(want), kw
    assert attend(L, T=0, q=None) == bm.BITMM_OK
    assert attend(L, B=0) == bm.BITMM_OK
    assert attend(L, max_q=0) == bm.BITMM_OK


def test_workspace(L):
    f = bm.bitmm_kv_attention_workspace_bytes
    for bad in [(-1, 1, 1, 1, 8, 2, 128), (1, 1, 1, 1, 7, 2, 128), (1, 1, 1, 1, 8, 2, 96), (1, 1, 1, 1, 8, 0, 128)]:
        assert f(*bad) == 0
    assert f(0, 1, 1, 100000, 8, 2, 128) == 0
    need = f(1, 1, 1, 100000, 8, 2, 128)
    assert need > 0 and need % 256 == 0
    args = dict(T=1, B=1, max_kv=100000)
    assert attend(L, **args) == bm.BITMM_ERR_WORKSPACE
    assert attend(L, ws=P, wsb=need - 1, **args) == bm.BITMM_ERR_WORKSPACE


def test_valid_calls_without_a_device(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for st in (rope(L), append(L), read(L), attend(L), attend(L, scale=float("nan"))):
        assert st == bm.BITMM_ERR_DEVICE


def test_frequencies():
    f, s = bm.rope_frequencies(64, 10000.0)
    i = torch.arange(32, dtype=torch.float64)
    base = 10000.0 ** (-i / 32)
    assert f.dtype == torch.float32 and s == 1.0
    assert torch.equal(f, base.float())
    assert torch.equal(bm.rope_frequencies(64, factor=4.0, scaling="linear")[0], (base / 4).float())
    f, _ = bm.rope_frequencies(64, factor=4.0, scaling="base")
    assert f[0] == 1.0 and abs(f[-1].item() / (base[-1].item() / 4) - 1) < 1e-6
    f, s = bm.rope_frequencies(64, factor=4.0, scaling="by_parts", original_context=4096)
    turns = 4096 * base / (2 * torch.pi)
    assert torch.equal(f[turns > 32], base.float()[turns > 32])
    assert torch.equal(f[turns < 1], (base / 4).float()[turns < 1])
    mid = (turns < 32) & (turns > 1)
    assert mid.any() and ((f[mid] < base[mid]) & (f[mid] > base[mid] / 4)).all()
    assert abs(s - 1.13862943611) < 1e-9
    assert bm.rope_frequencies(0)[0].numel() == 0
    for kw in (dict(rot_dim=7), dict(rot_dim=64, scaling="other"), dict(rot_dim=64, factor=0.5),
               dict(rot_dim=64, scaling="by_parts", factor=2.0)):
        with pytest.raises(ValueError):
            bm.rope_frequencies(**kw)


def small_cache(**kw):
    d = dict(num_pages=3, page_size=16, kv_heads=2, head_dim=64, group_size=32, device="cpu")
    d.update(kw)
    return bm.KVCache.empty(**d)


def test_binding_checks():
    c = small_cache()
    assert (c.num_pages, c.page_size, c.kv_heads, c.head_dim, c.group_size) == (3, 16, 2, 64, 32)
    with pytest.raises(ValueError):
        bm.KVCache(c.k_codes, c.k_scales, c.v_codes[:, :1], c.v_scales)
    with pytest.raises(TypeError):
        bm.KVCache(c.k_codes.long(), c.k_scales, c.v_codes, c.v_scales)
    with pytest.raises(ValueError):
        bm.KVCache(c.k_codes[0], c.k_scales, c.v_codes, c.v_scales)
    with pytest.raises(ValueError):
        small_cache(group_size=48)
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        bm.bitmm_kv_append(k.float(), k, slots, c, stream=0)
    with pytest.raises(TypeError):
        bm.bitmm_kv_append(k, k.half(), slots, c, stream=0)
    with pytest.raises(TypeError):
        bm.bitmm_kv_append(k, k, slots.int(), c, stream=0)
    with pytest.raises(ValueError):
        bm.bitmm_kv_append(k[:3], k, slots, c, stream=0)
    with pytest.raises(ValueError, match="side by side"):
        bm.bitmm_kv_append(torch.zeros(4, 64, 2, dtype=torch.bfloat16).transpose(1, 2), k, slots, c, stream=0)
    with pytest.raises(ValueError):
        bm.bitmm_kv_read(c, slots, None, None, stream=0)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    table, lens, cu = torch.zeros(2, 3, **i32), torch.zeros(2, **i32), torch.zeros(3, **i32)
    good = dict(max_q=1, max_kv=48, stream=0)
    for bad in [dict(q=torch.zeros(2, 4, 128, dtype=torch.bfloat16)), dict(cu=cu[:2]), dict(table=table[:1]),
                dict(out=torch.zeros(2, 3, 64)), dict(ws=torch.zeros(9))]:
        a = {**dict(q=q, table=table, lens=lens, cu=cu, out=torch.zeros(2, 4, 64), ws=None), **bad}
        with pytest.raises(ValueError):
            bm.bitmm_kv_attention(a["q"], c, a["table"], a["lens"], a["cu"], a["out"], a["ws"], **good)
    with pytest.raises(TypeError):
        bm.bitmm_kv_attention(q, c, table, lens, cu, torch.zeros(2, 4, 64, dtype=torch.float64), None, **good)
    with pytest.raises(ValueError):
        bm.bitmm_qk_norm_rope(None, None, None, None, None, None, None, None)
    with pytest.raises(ValueError):
        bm.bitmm_qk_norm_rope(q, None, None, None, None, None, None, None)
    with pytest.raises(ValueError):
        bm.bitmm_qk_norm_rope(q, None, torch.ones(32, dtype=torch.bfloat16), None, None, None, q, None)


def test_reference_on_worked_values():
    """The oracle's own pieces: codes in the order the header gives, ties to even, and one
    query that averages two equal keys' values."""
    x = torch.tensor([0.0, 15.0, 0.5, 1.5, 2.5, 7.0, 14.5, 3.0] + [0.0] * 24).bfloat16()
    codes, s, b = U.quantise(x, 32)
    assert s.item() == 1.0 and b.item() == 0.0
    assert codes[:8].tolist() == [0, 15, 0, 2, 2, 7, 14, 3]
    assert U.pack(codes)[0].item() == 0x3E7220F0
    seq = U.Sequences([(1, 2)], q_heads=1, kv_heads=1, head_dim=64, group=64, page=16, dtype=torch.bfloat16)
    seq.q[:] = 0
    out, lse, tol, _ = seq.reference(torch.bfloat16, 1.0)
    v, _ = seq.tokens(1, 0, 2)
    assert torch.allclose(out[0, 0], v.mean(0)[0]) and abs(lse.item() - 0.6931471805599453) < 1e-12
    assert (tol > 0).all()
    y, _ = U.rope_reference(torch.tensor([[[3.0, 4.0, 5.0, 6.0]]]), None, torch.tensor([1]),
                            torch.tensor([torch.pi / 2]).double(), interleaved=True, eps=0.0)
    assert torch.allclose(y, torch.tensor([[[-4.0, 3.0, 5.0, 6.0]]]).double())
