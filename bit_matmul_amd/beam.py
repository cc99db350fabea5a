"""Decoding several continuations of one prompt (beams, samples, guesses) over the 4-bit paged cache.

A thin ctypes binding over the calls of ``include/bitmm_beam.h``, in the manner of ``attention.py``:
the ``bitmm_*`` functions carry the C names and check and marshal their arguments, the others allocate
the outputs.
"""

from __future__ import annotations

import ctypes

from ._alloc import new as _new
from .attention import KVCache, _CacheDesc, _dtype_code, _expect, _lib, _raise, _rows, _status_word, _stream, _torch

__all__ = ["bitmm_qk_norm_rope_append", "qk_norm_rope_append"]


def declare(L) -> None:
    """Argument types of the calls of include/bitmm_beam.h in the loaded library."""
    P, I64, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    C = ctypes.POINTER(_CacheDesc)
    L.bitmm_qk_norm_rope_append.argtypes = [P, I64, P, I64, P, I64, P, P, P, P, P, I64, P, C, I64, I64, I64, I, F, F, F, I, P, P]
    L.bitmm_qk_norm_rope_append.restype = I


def bitmm_qk_norm_rope_append(q, k, v, q_weight, k_weight, positions, inv_freq, q_out, slots, cache: KVCache, *,
                              interleaved: bool = False, eps: float = 1e-6, weight_offset: float = 0.0,
                              rope_scale: float = 1.0, status=None, stream=None):
    """bitmm_qk_norm_rope on q [T, q_heads, D] and k [T, kv_heads, D], and bitmm_kv_append of that k
    (not rounded on the way) and v into the cache's slots [T] (int64; -1 stores nothing), in one
    launch. q may be None, with q_out; q_out may be q. inv_freq None or empty: no rotation."""
    torch = _torch()
    T, index, D = slots.shape[0], cache.device_index, cache.head_dim
    code, dtype, shape = _dtype_code(k, "k"), k.dtype, (slots.shape[0], cache.kv_heads, cache.head_dim)
    ks, vs = _rows(k, "k", dtype, shape, index), _rows(v, "v", dtype, shape, index)
    at = _expect(slots, "slots", torch.int64, (T,), index)
    qa = qo = qw = kw = freq = pos = None
    qs = qos = heads = rot = 0
    if q is None or q_out is None:
        if q is not q_out:
            raise ValueError("q and q_out go together")
    else:
        heads = q.shape[1]
        qs, qos = (_rows(t, name, dtype, (T, heads, D), index) for t, name in ((q, "q"), (q_out, "q_out")))
        qa, qo = q.data_ptr(), q_out.data_ptr()
        if q_weight is not None:
            qw = _expect(q_weight, "q_weight", dtype, (D,), index)
    if k_weight is not None:
        kw = _expect(k_weight, "k_weight", dtype, (D,), index)
    if inv_freq is not None and inv_freq.shape != (0,):
        rot = 2 * inv_freq.shape[0]
        freq = _expect(inv_freq, "inv_freq", torch.float32, (rot // 2,), index)
        pos = _expect(positions, "positions", torch.int32, (T,), index)
    st = _lib().bitmm_qk_norm_rope_append(qa, qs, k.data_ptr(), ks, v.data_ptr(), vs, qw, kw, pos, freq, qo, qos, at,
                                          cache.desc, T, heads, rot, 1 if interleaved else 0, eps, weight_offset,
                                          rope_scale, code, _status_word(status, index), _stream(stream, index))
    if st:
        _raise(st, "bitmm_qk_norm_rope_append")
    return q_out


def qk_norm_rope_append(q, k, v, q_weight, k_weight, positions, inv_freq, slots, cache: KVCache, *, stream=None, **options):
    """Returns q_out, a new tensor."""
    return bitmm_qk_norm_rope_append(q, k, v, q_weight, k_weight, positions, inv_freq, _new(q, q.shape, q.dtype, stream),
                                     slots, cache, stream=stream, **options)
