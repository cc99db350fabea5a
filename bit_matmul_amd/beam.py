"""Decoding several continuations of one prompt (beams, samples, guesses) over the 4-bit paged cache.

A thin ctypes binding over the calls of ``include/bitmm_beam.h``, in the manner of ``attention.py``:
the ``bitmm_*`` functions carry the C names and check and marshal their arguments, the others allocate
the outputs.
"""

from __future__ import annotations

import ctypes
import functools
import math

from ._alloc import new as _new
from .attention import KVCache, _CacheDesc, _dtype_code, _expect, _lib, _raise, _rows, _status_word, _stream, _torch

__all__ = ["bitmm_qk_norm_rope_append", "qk_norm_rope_append", "bitmm_kv_attention_shared_workspace_bytes",
           "bitmm_kv_attention_shared", "kv_attention_shared", "bitmm_beam_select_workspace_bytes", "bitmm_beam_select",
           "beam_select", "KVLayers", "bitmm_kv_beam_reorder_workspace_bytes", "bitmm_kv_beam_reorder", "kv_beam_reorder"]


def declare(L) -> None:
    """Argument types of the calls of include/bitmm_beam.h in the loaded library."""
    P, I64, I, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    C = ctypes.POINTER(_CacheDesc)
    L.bitmm_qk_norm_rope_append.argtypes = [P, I64, P, I64, P, I64, P, P, P, P, P, I64, P, C, I64, I64, I64, I, F, F, F, I, P, P]
    L.bitmm_qk_norm_rope_append.restype = I
    L.bitmm_kv_attention_shared_workspace_bytes.argtypes = [I64] * 10
    L.bitmm_kv_attention_shared_workspace_bytes.restype = SZ
    L.bitmm_kv_attention_shared.argtypes = [P, I64, C, P, I64, P, P, P, I64, P, P, P, I64, P, I64, I64, I64, I64, I64, I64, I64,
                                            I64, F, I, I, P, SZ, P, P]
    L.bitmm_kv_attention_shared.restype = I
    L.bitmm_beam_select_workspace_bytes.argtypes = [I64, I64, I64, I64, I]
    L.bitmm_beam_select_workspace_bytes.restype = SZ
    L.bitmm_beam_select.argtypes = [P, I64, P, P, P, P, P, P, I64, I64, I64, I64, ctypes.c_int32, I, P, SZ, P, P]
    L.bitmm_beam_select.restype = I
    L.bitmm_kv_beam_reorder_workspace_bytes.argtypes = [I64, I64]
    L.bitmm_kv_beam_reorder_workspace_bytes.restype = SZ
    L.bitmm_kv_beam_reorder.argtypes = [C, I64, P, P, I64, P, P, P, P, I64, I64, I64, I64, P, SZ, P, P]
    L.bitmm_kv_beam_reorder.restype = I


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
    """Returns q_out, a new tensor, or None if q is None."""
    q_out = None if q is None else _new(q, q.shape, q.dtype, stream)
    return bitmm_qk_norm_rope_append(q, k, v, q_weight, k_weight, positions, inv_freq, q_out, slots, cache, stream=stream, **options)


def bitmm_kv_attention_shared_workspace_bytes(T, B, groups, max_group_q, max_prefix, max_q, max_kv, q_heads, kv_heads, head_dim) -> int:
    return int(_lib().bitmm_kv_attention_shared_workspace_bytes(T, B, groups, max_group_q, max_prefix, max_q, max_kv, q_heads,
                                                                kv_heads, head_dim))


def bitmm_kv_attention_shared(q, cache: KVCache, prefix_table, prefix_lens, cu_groups, page_table, kv_lens, cu_q, out, workspace, *,
                              max_group_q: int, max_prefix: int, max_q: int, max_kv: int, scale=None, lse=None, status=None,
                              stream=None):
    """Attention of q [T, q_heads, D] over tokens that the sequences of a group share and each one's own.
    prefix_table: int32 [groups, pages], prefix_lens: int32 [groups], cu_groups: int32 [groups + 1] (the
    sequences of each group); page_table: int32 [B, pages], kv_lens: int32 [B], cu_q: int32 [B + 1] as in
    bitmm_kv_attention, of the own tokens. max_group_q: a bound of a group's queries, max_prefix of the
    shared tokens, max_q and max_kv of a sequence's queries and own tokens. out, lse, scale: as there;
    workspace: uint8 of at least bitmm_kv_attention_shared_workspace_bytes(...), or None if that is 0."""
    torch = _torch()
    T, heads, D = shape = q.shape
    B, groups = kv_lens.shape[0], prefix_lens.shape[0]
    index, int32 = cache.device_index, torch.int32
    if D != cache.head_dim:
        raise ValueError(f"q has heads of {D} dims, the cache of {cache.head_dim}")
    code = _dtype_code(q, "q")
    out_code = 0 if out.dtype is torch.bfloat16 else 2 if out.dtype is torch.float16 else 1
    if out_code == 1 and out.dtype is not torch.float32:
        raise TypeError(f"out must be bfloat16, float16 or float32, got {out.dtype}")
    q_stride, out_stride = _rows(q, "q", q.dtype, shape, index), _rows(out, "out", out.dtype, shape, index)
    if page_table.dim() != 2 or prefix_table.dim() != 2:
        raise ValueError("page_table and prefix_table must have two dims (sequences or groups, pages)")
    pages, prefix_pages = page_table.shape[1], prefix_table.shape[1]
    at = [_expect(prefix_lens, "prefix_lens", int32, (groups,), index), _expect(cu_groups, "cu_groups", int32, (groups + 1,), index),
          _expect(page_table, "page_table", int32, (B, pages), index)]
    lens, cu = _expect(kv_lens, "kv_lens", int32, (B,), index), _expect(cu_q, "cu_q", int32, (B + 1,), index)
    prefix = _expect(prefix_table, "prefix_table", int32, (groups, prefix_pages), index)
    ws, ws_bytes = None, 0
    if workspace is not None:
        if workspace.dtype is not torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the same device")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel()
    st = _lib().bitmm_kv_attention_shared(
        q.data_ptr(), q_stride, cache.desc, prefix, prefix_pages, *at, pages, lens, cu, out.data_ptr(), out_stride,
        None if lse is None else _expect(lse, "lse", torch.float32, (T, heads), index), T, B, groups, heads, max_group_q, max_prefix,
        max_q, max_kv, 1.0 / math.sqrt(D) if scale is None else scale, code, out_code, ws, ws_bytes,
        _status_word(status, index), _stream(stream, index))
    if st:
        _raise(st, "bitmm_kv_attention_shared")
    return out


def kv_attention_shared(q, cache: KVCache, prefix_table, prefix_lens, cu_groups, page_table, kv_lens, cu_q, *, max_group_q: int,
                        max_prefix: int, max_q: int, max_kv: int, scale=None, out_dtype=None, workspace=None, lse=None,
                        status=None, stream=None):
    """Returns the output, a new tensor of q's type unless out_dtype is given. Rows of q that
    belong to no sequence are left uninitialised."""
    out = _new(q, q.shape, q.dtype if out_dtype is None else out_dtype, stream)
    if workspace is None:
        need = bitmm_kv_attention_shared_workspace_bytes(q.shape[0], kv_lens.shape[0], prefix_lens.shape[0], max_group_q, max_prefix,
                                                         max_q, max_kv, q.shape[1], cache.kv_heads, cache.head_dim)
        workspace = _new(q, max(need, 16), _torch().uint8, stream, returned=False)
    return bitmm_kv_attention_shared(q, cache, prefix_table, prefix_lens, cu_groups, page_table, kv_lens, cu_q, out, workspace,
                                     max_group_q=max_group_q, max_prefix=max_prefix, max_q=max_q, max_kv=max_kv, scale=scale,
                                     lse=lse, status=status, stream=stream)


def _logits_code(t):
    torch, dtype = _torch(), t.dtype
    if dtype is torch.bfloat16:
        return 0
    if dtype is torch.float32:
        return 1
    if dtype is torch.float16:
        return 2
    raise TypeError(f"logits must be bfloat16, float16 or float32, got {dtype}")


def bitmm_beam_select_workspace_bytes(groups, beams, vocab, k, logits_dtype) -> int:
    """Of a call on logits [groups * beams, vocab] of a torch type."""
    torch = _torch()
    return _select_bytes(groups, beams, vocab, k, {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}[logits_dtype])


@functools.lru_cache(maxsize=64)   # the sizes of a search are the same step after step
def _select_bytes(groups, beams, vocab, k, code):
    return int(_lib().bitmm_beam_select_workspace_bytes(groups, beams, vocab, k, code))


def bitmm_beam_select(logits, scores, scores_out, parents, tokens, workspace, *, beams: int, finished=None, finished_out=None,
                      end_token: int = -1, status=None, stream=None):
    """The k best continuations of each group of `beams` rows of logits [groups * beams, vocab] (rows any
    stride apart), whose beams have scores [groups * beams] (float32): scores_out (float32), parents and
    tokens (int32), all [groups, k], k being their second size. finished: bool [groups * beams] or None;
    finished_out: bool [groups, k] or None. See include/bitmm_beam.h for what counts as a candidate.
    workspace: uint8 of at least bitmm_beam_select_workspace_bytes(...)."""
    torch = _torch()
    if logits.dim() != 2 or parents.dim() != 2:
        raise ValueError("logits must have two dims (beams of all groups, vocabulary), and parents two (groups, places)")
    groups, k = shape = parents.shape
    index = logits.get_device()
    if logits.shape[0] != groups * beams:
        raise ValueError(f"{logits.shape[0]} rows of logits are not {groups} groups of {beams} beams")
    outs = (_expect(scores_out, "scores_out", torch.float32, shape, index), _expect(parents, "parents", torch.int32, shape, index),
            _expect(tokens, "tokens", torch.int32, shape, index),
            None if finished_out is None else _expect(finished_out, "finished_out", torch.bool, shape, index))
    if workspace.dtype is not torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the same device")
    _select(logits, scores, finished, outs, groups, beams, k, end_token, workspace, status, stream)
    return scores_out, parents, tokens, finished_out


def _select(logits, scores, finished, outs, groups, beams, k, end_token, workspace, status, stream):
    """The call, with its inputs checked. outs: the addresses of the outputs."""
    torch = _torch()
    (rows, vocab), (row_stride, step), index = logits.shape, logits.stride(), logits.get_device()
    if vocab > 1 and step != 1:
        raise ValueError("the logits of a row must lie side by side")
    st = _lib().bitmm_beam_select(
        logits.data_ptr(), row_stride if rows > 1 else vocab, _expect(scores, "scores", torch.float32, (rows,), index),
        None if finished is None else _expect(finished, "finished", torch.bool, (rows,), index), *outs, groups, beams, vocab, k,
        end_token, _logits_code(logits), workspace.data_ptr(), workspace.numel(), _status_word(status, index), _stream(stream, index))
    if st:
        _raise(st, "bitmm_beam_select")


def beam_select(logits, scores, k: int, *, beams: int, finished=None, end_token: int = -1, workspace=None, status=None,
                stream=None):
    """Returns (scores, parents, tokens, finished), new tensors [groups, k]."""
    torch = _torch()
    rows, vocab = logits.shape
    if beams < 1 or rows % beams:
        raise ValueError(f"{rows} rows of logits are not groups of {beams} beams")
    groups = rows // beams
    best, ended = _new(logits, (groups, k), torch.float32, stream), _new(logits, (groups, k), torch.bool, stream)
    parents, tokens = _new(logits, (2, groups, k), torch.int32, stream).unbind()
    if workspace is None:
        need = _select_bytes(groups, beams, vocab, k, _logits_code(logits))
        workspace = _new(logits, max(need, 16), torch.uint8, stream, returned=False)
    elif workspace.dtype is not torch.uint8 or workspace.device != logits.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the same device")
    outs = best.data_ptr(), parents.data_ptr(), tokens.data_ptr(), ended.data_ptr()
    _select(logits, scores, finished, outs, groups, beams, k, end_token, workspace, status, stream)
    return best, parents, tokens, ended


class KVLayers:
    """The caches of a model's layers, of the same sizes, whose pages share one table."""

    def __init__(self, caches):
        self.caches = list(caches)
        if not self.caches:
            raise ValueError("at least one cache is needed")
        sizes = [(c.num_pages, c.page_size, c.kv_heads, c.head_dim, c.group_size, c.device_index) for c in self.caches]
        if any(s != sizes[0] for s in sizes):
            raise ValueError("the layers' caches must have the same sizes and lie on one device")
        self.device_index, self.page_size = self.caches[0].device_index, self.caches[0].page_size
        self.desc = (_CacheDesc * len(self.caches))(*(c.desc for c in self.caches))


def bitmm_kv_beam_reorder_workspace_bytes(groups, beams) -> int:
    return int(_lib().bitmm_kv_beam_reorder_workspace_bytes(groups, beams))


def bitmm_kv_beam_reorder(layers: KVLayers, page_table, lens, parents, page_table_out, lens_out, slots, workspace, *,
                          first_page: int, pages_per_group: int, status=None, stream=None):
    """The cached states in the order of parents [groups, beams] (int32; the beam that each row goes on
    from, -1 for none), with room for one more token each. page_table: int32 [groups * beams, pages];
    lens: int32 [groups * beams]; slots: int64 [groups * beams], where the next tokens go; lens_out counts
    them. Outputs may be their inputs. New pages come from the group's pool of pages_per_group pages; see
    include/bitmm_beam.h. workspace: uint8 of at least bitmm_kv_beam_reorder_workspace_bytes(...)."""
    torch, index = _torch(), layers.device_index
    if page_table.dim() != 2:
        raise ValueError("page_table must have two dims (rows, pages)")
    outs = (_expect(page_table_out, "page_table_out", torch.int32, page_table.shape, index),
            _expect(lens_out, "lens_out", torch.int32, lens.shape, index), _expect(slots, "slots", torch.int64, lens.shape, index))
    if workspace.dtype is not torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the same device")
    _reorder(layers, page_table, lens, parents, outs, workspace, first_page, pages_per_group, status, stream)
    return page_table_out, lens_out, slots


def _reorder(layers, page_table, lens, parents, outs, workspace, first_page, pages_per_group, status, stream):
    """The call, with its inputs checked. outs: the addresses of the outputs, of the shapes of the inputs."""
    int32, index = _torch().int32, layers.device_index
    if parents.dim() != 2 or page_table.dim() != 2:
        raise ValueError("parents must have two dims (groups, beams), and page_table two (rows, pages)")
    (groups, beams), pages = parents.shape, page_table.shape[1]
    rows = groups * beams
    st = _lib().bitmm_kv_beam_reorder(
        layers.desc, len(layers.caches), _expect(page_table, "page_table", int32, (rows, pages), index), outs[0], pages,
        _expect(lens, "lens", int32, (rows,), index), outs[1], _expect(parents, "parents", int32, (groups, beams), index), outs[2],
        groups, beams, first_page, pages_per_group, workspace.data_ptr(), workspace.numel(), _status_word(status, index),
        _stream(stream, index))
    if st:
        _raise(st, "bitmm_kv_beam_reorder")


def kv_beam_reorder(layers: KVLayers, page_table, lens, parents, *, first_page: int, pages_per_group: int, workspace=None,
                    status=None, stream=None):
    """Returns (page_table, lens, slots), new tensors; the caches' copies are made in place."""
    torch = _torch()
    table, lens_out = _new(page_table, page_table.shape, torch.int32, stream), _new(lens, lens.shape, torch.int32, stream)
    slots = _new(lens, lens.shape, torch.int64, stream)
    if workspace is None:
        workspace = _new(lens, max(16 * lens.numel(), 16), torch.uint8, stream, returned=False)
    elif workspace.dtype is not torch.uint8 or workspace.device != lens.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the same device")
    outs = table.data_ptr(), lens_out.data_ptr(), slots.data_ptr()
    _reorder(layers, page_table, lens, parents, outs, workspace, first_page, pages_per_group, status, stream)
    return table, lens_out, slots
