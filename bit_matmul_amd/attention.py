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


def _lib():
    import bit_matmul_amd as bm
    return bm.lib()


def _raise(status: int, where: str):
    import bit_matmul_amd as bm
    raise bm.BitmmError(status, where)


def _torch():
    import torch
    return torch


def _stream(stream, device):
    if stream is None:
        stream = _torch().cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t, name):
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return 0
    if t.dtype == torch.float16:
        return 1
    raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")


def _expect(t, name, dtype, shape, device):
    """A contiguous tensor of exactly this type, shape and device."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _rows(t, name, dtype, shape, device):
    """Values between tokens of a [tokens, heads, head_dim] tensor whose heads lie side by side."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    st = t.stride()
    if (shape[2] > 1 and st[2] != 1) or (shape[1] > 1 and st[1] != shape[2]):
        raise ValueError(f"{name}: the heads of a token must lie side by side (strides {st})")
    return st[0] if shape[0] > 1 else max(shape[1] * shape[2], 8)


def _address(t):
    return t.data_ptr() if t is not None and t.numel() > 0 else None


def _status_word(status, device):
    if status is None:
        return None
    _expect(status, "status", _torch().int32, (1,), device)
    return status.data_ptr()


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
        dev = k_codes.device
        for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
            _expect(t, name, torch.int32, (pages, heads, size, words), dev)
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            _expect(t, name, torch.bfloat16, (pages, heads, size, groups, 2), dev)
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.num_pages, self.kv_heads, self.page_size = pages, heads, size
        self.head_dim, self.group_size = 8 * words, 8 * words // groups
        self.device = dev
        self.desc = _CacheDesc(_address(k_codes), _address(k_scales), _address(v_codes), _address(v_scales), pages,
                               size, heads, self.head_dim, self.group_size)

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
    dev, code = one.device, _dtype_code(one, "q" if q is not None else "k")
    args = []
    for name, x, w, y in (("q", q, q_weight, q_out), ("k", k, k_weight, k_out)):
        if (x is None) != (y is None):
            raise ValueError(f"{name} and {name}_out go together")
        heads = 0 if x is None else x.shape[1]
        s = so = 0
        if x is not None:
            s = _rows(x, name, one.dtype, (T, heads, D), dev)
            so = _rows(y, name + "_out", one.dtype, (T, heads, D), dev)
            if w is not None:
                _expect(w, name + "_weight", one.dtype, (D,), dev)
        args.append((_address(x), s, _address(w) if x is not None else None, _address(y), so, heads))
    rot = 0
    if inv_freq is not None and inv_freq.numel():
        rot = 2 * inv_freq.numel()
        _expect(inv_freq, "inv_freq", torch.float32, (rot // 2,), dev)
        _expect(positions, "positions", torch.int32, (T,), dev)
    (qa, qs, qw, qo, qos, hq), (ka, ks, kw, ko, kos, hk) = args
    st = _lib().bitmm_qk_norm_rope(qa, qs, ka, ks, qw, kw, _address(positions) if rot else None,
                                   _address(inv_freq) if rot else None, qo, qos, ko, kos, T, hq, hk, D, rot,
                                   int(bool(interleaved)), eps, weight_offset, rope_scale, code, _stream(stream, dev))
    if st:
        _raise(st, "bitmm_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, **options):
    """Returns (q_out, k_out), new tensors."""
    torch = _torch()
    fresh = [None if x is None else torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in (q, k)]
    return bitmm_qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, *fresh, **options)


def bitmm_kv_append(k, v, slots, cache: KVCache, status=None, stream=None):
    """Quantizes k and v [T, kv_heads, D] into the cache's slots [T] (int64; -1 skips a token).
    `status` (optional int32 tensor of one element) is set to 1 by a slot outside the cache."""
    dev = cache.device
    shape = (slots.shape[0], cache.kv_heads, cache.head_dim)
    code = _dtype_code(k, "k")
    ks = _rows(k, "k", k.dtype, shape, dev)
    vs = _rows(v, "v", k.dtype, shape, dev)
    _expect(slots, "slots", _torch().int64, shape[:1], dev)
    st = _lib().bitmm_kv_append(_address(k), ks, _address(v), vs, _address(slots), shape[0], cache.desc, code,
                                _status_word(status, dev), _stream(stream, dev))
    if st:
        _raise(st, "bitmm_kv_append")


def bitmm_kv_read(cache: KVCache, slots, k_out, v_out, status=None, stream=None):
    """The keys and values held at slots [T], into k_out and v_out [T, kv_heads, D] (either may
    be None); zeros for slots of -1 and for slots outside the cache, which set `status`."""
    dev = cache.device
    shape = (slots.shape[0], cache.kv_heads, cache.head_dim)
    one = k_out if k_out is not None else v_out
    if one is None:
        raise ValueError("k_out and v_out are both None")
    code = _dtype_code(one, "k_out" if k_out is not None else "v_out")
    ks = _rows(k_out, "k_out", one.dtype, shape, dev) if k_out is not None else 0
    vs = _rows(v_out, "v_out", one.dtype, shape, dev) if v_out is not None else 0
    _expect(slots, "slots", _torch().int64, shape[:1], dev)
    st = _lib().bitmm_kv_read(cache.desc, _address(slots), shape[0], _address(k_out), ks, _address(v_out), vs, code,
                              _status_word(status, dev), _stream(stream, dev))
    if st:
        _raise(st, "bitmm_kv_read")
    return k_out, v_out


def kv_read(cache: KVCache, slots, dtype=None, status=None, stream=None):
    """Returns (k, v), new tensors of `dtype` (bfloat16 by default)."""
    torch = _torch()
    shape = (slots.shape[0], cache.kv_heads, cache.head_dim)
    fresh = [torch.empty(shape, dtype=dtype or torch.bfloat16, device=cache.device) for _ in range(2)]
    return bitmm_kv_read(cache, slots, *fresh, status=status, stream=stream)


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
    T, heads, D = q.shape
    B = kv_lens.shape[0]
    dev = cache.device
    if D != cache.head_dim:
        raise ValueError(f"q has heads of {D} dims, the cache of {cache.head_dim}")
    code = _dtype_code(q, "q")
    qs = _rows(q, "q", q.dtype, (T, heads, D), dev)
    kinds = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}
    if out.dtype not in kinds:
        raise TypeError(f"out must be bfloat16, float16 or float32, got {out.dtype}")
    os = _rows(out, "out", out.dtype, (T, heads, D), dev)
    if page_table.dim() != 2:
        raise ValueError("page_table must have two dims (sequences, pages)")
    _expect(page_table, "page_table", torch.int32, (B, page_table.shape[1]), dev)
    _expect(kv_lens, "kv_lens", torch.int32, (B,), dev)
    _expect(cu_q, "cu_q", torch.int32, (B + 1,), dev)
    if lse is not None:
        _expect(lse, "lse", torch.float32, (T, heads), dev)
    if workspace is not None and (workspace.dtype != torch.uint8 or workspace.device != dev or
                                  not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor on the same device")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    st = _lib().bitmm_kv_attention(_address(q), qs, cache.desc, _address(page_table), page_table.shape[1],
                                   _address(kv_lens), _address(cu_q), _address(out), os, _address(lse), T, B, heads,
                                   max_q, max_kv, scale, window, sinks, code, kinds[out.dtype], _address(workspace),
                                   workspace.numel() if workspace is not None else 0, _status_word(status, dev),
                                   _stream(stream, dev))
    if st:
        _raise(st, "bitmm_kv_attention")
    return out


def kv_attention(q, cache: KVCache, page_table, kv_lens, cu_q, *, max_q: int, max_kv: int, scale=None,
                 window: int = 0, sinks: int = 0, out_dtype=None, workspace=None, lse=None, status=None, stream=None):
    """Returns the output, a new tensor of q's type unless out_dtype is given. Rows of q that
    belong to no sequence are left uninitialised."""
    torch = _torch()
    out = torch.empty(q.shape, dtype=out_dtype or q.dtype, device=q.device)
    if workspace is None:
        need = bitmm_kv_attention_workspace_bytes(q.shape[0], kv_lens.shape[0], max_q, max_kv, q.shape[1],
                                                  cache.kv_heads, cache.head_dim, window, sinks)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    return bitmm_kv_attention(q, cache, page_table, kv_lens, cu_q, out, workspace, max_q=max_q, max_kv=max_kv,
                              scale=scale, window=window, sinks=sinks, lse=lse, status=status, stream=stream)
