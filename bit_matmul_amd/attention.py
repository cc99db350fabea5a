"""The attention block between the quantized projections: head norms with the position
rotation, a 4-bit paged cache of keys and values, and attention over it.

A thin ctypes binding over the calls of ``include/bitmm_attn.h``, in the manner of the rest of
the package: the ``bitmm_*`` functions carry the C names, check that tensors match what the C
call expects and pass raw device pointers and the current HIP stream; the others allocate the
outputs. Heads of one token lie side by side; consecutive tokens may be any stride apart (a
multiple of 8), so slices of a fused projection's output are passed as they are.

One decoding step of a layer:

    q, k = bm.qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq)
    bm.bitmm_kv_append(k, v, slots, cache)
    out = bm.kv_attention(q, cache, page_table, kv_lens, cu_q, max_q=1, max_kv=max_kv)
"""

from __future__ import annotations

import ctypes
import math
import sys

from ._alloc import new as _new

__all__ = [
    "KVCache", "rope_frequencies", "bitmm_qk_norm_rope", "qk_norm_rope", "bitmm_kv_append",
    "bitmm_kv_read", "kv_read", "bitmm_kv_attention_workspace_bytes", "bitmm_kv_attention",
    "kv_attention",
]


class _CacheDesc(ctypes.Structure):
    """bitmm_kv_cache of include/bitmm_attn.h."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("group_size", ctypes.c_int32)]


def declare(L) -> None:
    """Argument types of the calls of include/bitmm_attn.h in the loaded library."""
    P, I64, I, SZ, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    C = ctypes.POINTER(_CacheDesc)
    L.bitmm_qk_norm_rope.argtypes = [P, I64, P, I64, P, P, P, P, P, I64, P, I64, I64, I64, I64, I64, I64, I, F, F, F, I, P]
    L.bitmm_qk_norm_rope.restype = I
    L.bitmm_kv_append.argtypes = [P, I64, P, I64, P, I64, C, I, P, P]
    L.bitmm_kv_append.restype = I
    L.bitmm_kv_read.argtypes = [C, P, I64, P, I64, P, I64, I, P, P]
    L.bitmm_kv_read.restype = I
    L.bitmm_kv_attention_workspace_bytes.argtypes = [I64] * 9
    L.bitmm_kv_attention_workspace_bytes.restype = SZ
    L.bitmm_kv_attention.argtypes = [P, I64, C, P, I64, P, P, P, I64, P, I64, I64, I64, I64, I64, F, I64, I64, I, I, P, SZ, P, P]
    L.bitmm_kv_attention.restype = I


# A small call's time is mostly its marshalling, so the checks below are written for the case in
# which everything is right: one pass over what a call needs, and the reason looked for only when
# something is wrong.

_torch_module = None
_current_stream = None  # the current HIP stream of a device index, as an integer


def _torch():
    global _torch_module, _current_stream
    if _torch_module is None:
        import torch
        _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _torch_module = torch
    return _torch_module


def _lib():
    return sys.modules[__package__].lib()


def _raise(status: int, where: str):
    raise sys.modules[__package__].BitmmError(status, where)


def _stream(stream, index):
    if index < 0:
        raise ValueError("tensors must be on the GPU")
    if stream is None:
        return _current_stream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t, name):
    torch = _torch()
    if t.dtype is torch.bfloat16:
        return 0
    if t.dtype is torch.float16:
        return 1
    raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")


def _expect(t, name, dtype, shape, index):
    """The address of a contiguous tensor of exactly this type, shape and device."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, not where the call's other tensors are")


def _rows(t, name, dtype, shape, index):
    """Values between tokens of a [tokens, heads, head_dim] tensor whose heads lie side by side."""
    st = t.stride()
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and st[2] == 1 and st[1] == shape[2] and shape[0] > 1:
        return st[0]
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not where the call's other tensors are")
    if (shape[2] > 1 and st[2] != 1) or (shape[1] > 1 and st[1] != shape[2]):
        raise ValueError(f"{name}: the heads of a token must lie side by side (strides {st})")
    return st[0] if shape[0] > 1 else max(shape[1] * shape[2], 8)  # the stride of one token says nothing


def _status_word(status, index):
    return None if status is None else _expect(status, "status", _torch().int32, (1,), index)


class KVCache:
    """A 4-bit paged cache: four tensors (see include/bitmm_attn.h) and their sizes.

        k_codes, v_codes    int32    [num_pages, kv_heads, page_size, head_dim / 8]
        k_scales, v_scales  bfloat16 [num_pages, kv_heads, page_size, head_dim / group_size, 2]
    """

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        torch = _torch()
        if k_codes.dim() != 4 or k_scales.dim() != 5:
            raise ValueError("codes have 4 dims (pages, heads, slots, words) and scales 5 "
                             "(pages, heads, slots, groups, 2)")
        pages, heads, size, words = k_codes.shape
        groups = k_scales.shape[3]
        if groups < 1 or (8 * words) % groups:
            raise ValueError(f"{groups} groups do not divide a head of {8 * words} dims")
        index = k_codes.get_device()
        codes, scales = (pages, heads, size, words), (pages, heads, size, groups, 2)
        at = [_expect(k_codes, "k_codes", torch.int32, codes, index),
              _expect(k_scales, "k_scales", torch.bfloat16, scales, index),
              _expect(v_codes, "v_codes", torch.int32, codes, index),
              _expect(v_scales, "v_scales", torch.bfloat16, scales, index)]
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.num_pages, self.kv_heads, self.page_size = pages, heads, size
        self.head_dim, self.group_size = 8 * words, 8 * words // groups
        self.device, self.device_index = k_codes.device, index
        self.desc = _CacheDesc(*at, pages, size, heads, self.head_dim, self.group_size)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int, group_size: int = 64, device="cuda"):
        """A cache of num_pages pages, not initialised."""
        torch = _torch()
        if head_dim % 8 or group_size < 1 or head_dim % group_size:
            raise ValueError(f"group_size {group_size} does not divide head_dim {head_dim}, or that is no multiple of 8")
        codes = (num_pages, kv_heads, page_size, head_dim // 8)
        scales = (num_pages, kv_heads, page_size, head_dim // group_size, 2)
        sides = [t for _ in range(2) for t in (torch.empty(codes, dtype=torch.int32, device=device),
                                               torch.empty(scales, dtype=torch.bfloat16, device=device))]
        return cls(*sides)


def rope_frequencies(rot_dim: int, theta: float = 10000.0, *, factor: float = 1.0, scaling: str = "none",
                     original_context: int = 0, low: float = 1.0, high: float = 32.0, device="cpu"):
    """(inv_freq, rope_scale) for bitmm_qk_norm_rope: radians a position of each pair, f32
    [rot_dim / 2], from 64-bit arithmetic, scaled for contexts `factor` times the original.

    scaling "none":     theta^(-2 i / rot_dim)
            "linear":   that, divided by factor (positions squeezed into the original range)
            "base":     theta times factor^(rot_dim / (rot_dim - 2)): the slowest pair is
                        slowed by factor, the fastest not at all
            "by_parts": pairs that turn more than `high` times over original_context keep
                        their speed, those that turn less than `low` times are slowed by
                        factor, those between are blended linearly in their turns; rope_scale
                        is 0.1 ln(factor) + 1
    """
    torch = _torch()
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even, got {rot_dim}")
    if not factor >= 1.0:
        raise ValueError(f"factor must be at least 1, got {factor}")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "base" and rot_dim > 2:
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    freq = float(theta) ** (-i / max(rot_dim, 1))
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "by_parts":
        if original_context < 1 or not high > low:
            raise ValueError("by_parts needs original_context >= 1 and high > low")
        turns = original_context * freq / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        freq = freq * keep + freq / factor * (1 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.float().to(device), scale


def bitmm_qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, *, interleaved: bool = False,
                       eps: float = 1e-6, weight_offset: float = 0.0, rope_scale: float = 1.0, stream=None):
    """RMS norm of each head of q [T, q_heads, D] and k [T, kv_heads, D] (weights [D], or None
    for none), then the rotation of its first 2 * len(inv_freq) dims by positions [T] (int32).
    q or k may be None, with its output. An output may be its own input. inv_freq None or
    empty: no rotation."""
    torch = _torch()
    one = q if q is not None else k
    if one is None:
        raise ValueError("q and k are both None")
    T, _, D = one.shape
    dtype, index = one.dtype, one.get_device()
    code = _dtype_code(one, "q" if q is not None else "k")

    def side(name, x, weight, out):
        """(address, stride, weight's address, output's address, its stride, heads)"""
        if x is None or out is None:
            if x is not out:
                raise ValueError(f"{name} and {name}_out go together")
            return None, 0, None, None, 0, 0
        shape = (T, x.shape[1], D)
        stride, out_stride = _rows(x, name, dtype, shape, index), _rows(out, name + "_out", dtype, shape, index)
        w = None if weight is None else _expect(weight, name + "_weight", dtype, (D,), index)
        return x.data_ptr(), stride, w, out.data_ptr(), out_stride, shape[1]

    qa, qs, qw, qo, qos, hq = side("q", q, q_weight, q_out)
    ka, ks, kw, ko, kos, hk = side("k", k, k_weight, k_out)
    rot, freq, pos = 0, None, None
    if inv_freq is not None and inv_freq.shape != (0,):
        rot = 2 * inv_freq.shape[0]
        freq = _expect(inv_freq, "inv_freq", torch.float32, (rot // 2,), index)
        pos = _expect(positions, "positions", torch.int32, (T,), index)
    st = _lib().bitmm_qk_norm_rope(qa, qs, ka, ks, qw, kw, pos, freq, qo, qos, ko, kos, T, hq, hk, D, rot,
                                   1 if interleaved else 0, eps, weight_offset, rope_scale, code, _stream(stream, index))
    if st:
        _raise(st, "bitmm_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, *, stream=None, **options):
    """Returns (q_out, k_out), new tensors."""
    q_out, k_out = (None if x is None else _new(x, x.shape, x.dtype, stream) for x in (q, k))
    return bitmm_qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, stream=stream, **options)


def bitmm_kv_append(k, v, slots, cache: KVCache, status=None, stream=None):
    """Quantizes k and v [T, kv_heads, D] into the cache's slots [T] (int64; -1 skips a token).
    `status` (optional int32 tensor of one element) is set to 1 by a slot outside the cache."""
    index = cache.device_index
    shape = (slots.shape[0], cache.kv_heads, cache.head_dim)
    code = _dtype_code(k, "k")
    ks, vs = _rows(k, "k", k.dtype, shape, index), _rows(v, "v", k.dtype, shape, index)
    st = _lib().bitmm_kv_append(k.data_ptr(), ks, v.data_ptr(), vs, _expect(slots, "slots", _torch().int64, shape[:1], index),
                                shape[0], cache.desc, code, _status_word(status, index), _stream(stream, index))
    if st:
        _raise(st, "bitmm_kv_append")


def bitmm_kv_read(cache: KVCache, slots, k_out, v_out, status=None, stream=None):
    """The keys and values held at slots [T], into k_out and v_out [T, kv_heads, D] (either may
    be None); zeros for slots of -1 and for slots outside the cache, which set `status`."""
    index = cache.device_index
    shape = (slots.shape[0], cache.kv_heads, cache.head_dim)
    one = k_out if k_out is not None else v_out
    if one is None:
        raise ValueError("k_out and v_out are both None")
    code = _dtype_code(one, "k_out" if k_out is not None else "v_out")
    ka = va = None
    ks = vs = 0
    if k_out is not None:
        ka, ks = k_out.data_ptr(), _rows(k_out, "k_out", one.dtype, shape, index)
    if v_out is not None:
        va, vs = v_out.data_ptr(), _rows(v_out, "v_out", one.dtype, shape, index)
    st = _lib().bitmm_kv_read(cache.desc, _expect(slots, "slots", _torch().int64, shape[:1], index), shape[0], ka, ks, va,
                              vs, code, _status_word(status, index), _stream(stream, index))
    if st:
        _raise(st, "bitmm_kv_read")
    return k_out, v_out


def kv_read(cache: KVCache, slots, dtype=None, status=None, stream=None):
    """Returns (k, v), new tensors of `dtype` (bfloat16 by default)."""
    torch = _torch()
    shape = (slots.shape[0], cache.kv_heads, cache.head_dim)
    k, v = (_new(cache.k_scales, shape, dtype or torch.bfloat16, stream) for _ in range(2))
    return bitmm_kv_read(cache, slots, k, v, status=status, stream=stream)


def bitmm_kv_attention_workspace_bytes(T, B, max_q, max_kv, q_heads, kv_heads, head_dim, window=0, sinks=0) -> int:
    return int(_lib().bitmm_kv_attention_workspace_bytes(T, B, max_q, max_kv, q_heads, kv_heads, head_dim, window, sinks))


def bitmm_kv_attention(q, cache: KVCache, page_table, kv_lens, cu_q, out, workspace, *, max_q: int, max_kv: int,
                       scale=None, window: int = 0, sinks: int = 0, lse=None, status=None, stream=None):
    """Causal attention of q [T, q_heads, D] over the cache, with an optional sliding window and
    `sinks` first tokens that stay visible to it. page_table: int32 [B, pages]; kv_lens: int32
    [B]; cu_q: int32 [B + 1], the rows of each sequence's queries; max_q, max_kv: bounds of their
    lengths. out: [T, q_heads, D] in bfloat16, float16 or float32; lse: float32 [T, q_heads] or
    None; workspace: uint8 of at least bitmm_kv_attention_workspace_bytes(...), or None if that
    is 0. scale: 1 / sqrt(D) by default."""
    torch = _torch()
    T, heads, D = shape = q.shape
    B = kv_lens.shape[0]
    index, int32 = cache.device_index, torch.int32
    if D != cache.head_dim:
        raise ValueError(f"q has heads of {D} dims, the cache of {cache.head_dim}")
    code = _dtype_code(q, "q")
    out_code = 0 if out.dtype is torch.bfloat16 else 2 if out.dtype is torch.float16 else 1
    if out_code == 1 and out.dtype is not torch.float32:
        raise TypeError(f"out must be bfloat16, float16 or float32, got {out.dtype}")
    q_stride, out_stride = _rows(q, "q", q.dtype, shape, index), _rows(out, "out", out.dtype, shape, index)
    if page_table.dim() != 2:
        raise ValueError("page_table must have two dims (sequences, pages)")
    pages = page_table.shape[1]
    table = _expect(page_table, "page_table", int32, (B, pages), index)
    lens, cu = _expect(kv_lens, "kv_lens", int32, (B,), index), _expect(cu_q, "cu_q", int32, (B + 1,), index)
    ws, ws_bytes = None, 0
    if workspace is not None:
        if workspace.dtype is not torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the same device")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel()
    st = _lib().bitmm_kv_attention(
        q.data_ptr(), q_stride, cache.desc, table, pages, lens, cu, out.data_ptr(), out_stride,
        None if lse is None else _expect(lse, "lse", torch.float32, (T, heads), index), T, B, heads, max_q, max_kv,
        1.0 / math.sqrt(D) if scale is None else scale, window, sinks, code, out_code, ws, ws_bytes,
        _status_word(status, index), _stream(stream, index))
    if st:
        _raise(st, "bitmm_kv_attention")
    return out


def kv_attention(q, cache: KVCache, page_table, kv_lens, cu_q, *, max_q: int, max_kv: int, scale=None,
                 window: int = 0, sinks: int = 0, out_dtype=None, workspace=None, lse=None, status=None, stream=None):
    """Returns the output, a new tensor of q's type unless out_dtype is given. Rows of q that
    belong to no sequence are left uninitialised."""
    out = _new(q, q.shape, q.dtype if out_dtype is None else out_dtype, stream)
    if workspace is None:
        need = bitmm_kv_attention_workspace_bytes(q.shape[0], kv_lens.shape[0], max_q, max_kv, q.shape[1],
                                                  cache.kv_heads, cache.head_dim, window, sinks)
        if need:
            workspace = _new(q, need, _torch().uint8, stream, returned=False)
    return bitmm_kv_attention(q, cache, page_table, kv_lens, cu_q, out, workspace, max_q=max_q, max_kv=max_kv,
                              scale=scale, window=window, sinks=sinks, lse=lse, status=status, stream=stream)
