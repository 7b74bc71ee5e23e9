"""Paged key/value cache: norm and rotation of heads, append, dense read, one-token attention.

The entry points wrap the calls of the same names in ``include/sage_fp4.h``. As in the rest of the package
they check arguments, allocate outputs and workspace with torch and launch on the current
stream of the tensors' device (natively, in ``csrc/binding.cpp``: a step's kernels take a few microseconds);
what the device tables hold (lengths, pages, positions) is checked on the device and reported by
``device_error()``.

    cache = sage.PagedKVCache.empty(num_pages, 64, num_kv_heads, head_dim, format="fp4")
    rope = sage.rope_table(max_positions, head_dim)
    # prompts: packed rows, seq_lens = their lengths
    out = sage.sageattn_prefill(q, k, v, cache, page_table, seq_lens, cu_seqlens, max_seqlen, rope=rope)
    # one token of each sequence: seq_lens += 1, then
    q = sage.cache_append(cache, k, v, page_table, seq_lens, q=q, rope=rope)
    out = sage.sageattn_decode(q, cache, page_table, seq_lens)
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

import microscaling_fp4_quantized_b200 as _sage

CACHE_FORMAT = {"16bit": 0, "fp4": 1}


class _Rope(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("weight_f32", ctypes.c_int),
                ("eps", ctypes.c_float), ("rope", ctypes.c_void_p), ("rope_len", ctypes.c_int),
                ("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int)]


class _Rows(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("heads", ctypes.c_int),
                ("x_stride", ctypes.c_int64 * 3), ("y_stride", ctypes.c_int64 * 3)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_sf", ctypes.c_void_p),
                ("v_sf", ctypes.c_void_p), ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("D", ctypes.c_int), ("dtype", ctypes.c_int), ("format", ctypes.c_int)]


class _Batch(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("table_width", ctypes.c_int), ("seq_lens", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p)]


_Stride3 = ctypes.c_int64 * 3


_native = None


def bind(L) -> None:
    """Argument types of the paged entry points."""
    i, vp, sz, f = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
    rows, rope, cache, batch = (ctypes.POINTER(t) for t in (_Rows, _Rope, _Cache, _Batch))
    st = ctypes.POINTER(ctypes.c_int64)
    L.sage_fp4_norm_rope.argtypes = [rows, rows, i, i, i, i, rope, vp, vp]
    L.sage_fp4_cache_append.argtypes = [cache, batch, vp, st, vp, st, i, rope, rows, vp]
    L.sage_fp4_cache_gather.argtypes = [cache, batch, vp, st, vp, st, i, vp]
    L.sage_fp4_decode_workspace_bytes.argtypes = [cache, batch, i]
    L.sage_fp4_decode_workspace_bytes.restype = sz
    L.sage_fp4_attn_decode.argtypes = [cache, batch, vp, st, vp, st, i, f, vp, sz, vp]


def _n():
    """The native binding, with the library's entry points (raises if it is missing)."""
    global _native
    if _native is None:
        L, vp = _sage.lib(), ctypes.c_void_p
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError("the native binding is missing; build it with "
                               "`python -m microscaling_fp4_quantized_b200.build`") from e
        calls = (L.sage_fp4_norm_rope, L.sage_fp4_cache_append, L.sage_fp4_cache_gather,
                 L.sage_fp4_decode_workspace_bytes, L.sage_fp4_attn_decode)
        _binding.bind(*(ctypes.cast(c, vp).value for c in calls), _sage._check)
        _native = _binding
    return _native


def _stride(t: torch.Tensor, d: int) -> int:
    """A dimension of size 1 has no stride that could matter."""
    return t.stride(d) if t.shape[d] != 1 else 0


def rope_table(max_positions: int, rotary_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """The rotation table the entry points take, [max_positions, rotary_dim] float32: the cosines of
    position * base^(-2i / rotary_dim), i < rotary_dim / 2, then their sines. The angles are formed
    in 64 bits (at far positions 32 would lose the turn). Built once per model."""
    if max_positions < 0 or rotary_dim <= 0 or rotary_dim % 32 != 0:
        raise ValueError("rotary_dim must be a positive multiple of 32 and max_positions not negative")
    inv = float(base) ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device) / rotary_dim)
    a = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), dim=1).float()


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor] = None, *, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, rope: Optional[torch.Tensor] = None,
                 positions: Optional[torch.Tensor] = None, interleaved: bool = False, tensor_layout: str = "HND",
                 q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """RMS norm of every query and key head and the position rotation, in one pass over q and k.

    q and k: [B, H, N, D] ("HND"), [B, N, H, D] ("NHD") or packed [tokens, H, D], bf16 or fp16, any strides
    with contiguous channels; k may have fewer heads and may be left out. Weights ([D], the tensors' dtype
    or float32) switch the norm on; rope (see rope_table) the rotation of the first rope.shape[1] channels,
    pairs (i, i + rotary_dim/2), or (2i, 2i+1) when interleaved. positions: int32, [B, N] or, for packed
    rows, [tokens]; without it token n of a 4-d tensor is at position n. A position outside the table
    is reported by device_error() and its rows are not written. q_out / k_out may be q / k (in place) and
    must not overlap them otherwise. Returns (q_out, k_out)."""
    return _n().norm_rope(q, k, q_weight, k_weight, eps, rope, positions, interleaved, tensor_layout, q_out, k_out)


class PagedKVCache:
    """The pages of one layer's keys and values, on the caller's buffers.

    k, v: [pages, heads, slots, D] ("HND") or [pages, slots, heads, D] ("NHD"), any strides with contiguous
    channels. 16-bit: bf16 or fp16. FP4: uint8 codes with D / 2 bytes per row, and k_sf, v_sf uint8 with D / 16
    bytes per row and an eighth of the codes' strides; `dtype` then names the dense side (queries, new
    keys and values, outputs)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_sf: Optional[torch.Tensor] = None,
                 v_sf: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
                 tensor_layout: str = "HND"):
        if tensor_layout not in ("HND", "NHD"):
            raise ValueError("tensor_layout must be 'HND' or 'NHD'")
        fp4 = k.dtype == torch.uint8
        if fp4 and (k_sf is None or v_sf is None or dtype is None):
            raise ValueError("an FP4 cache needs k_sf, v_sf and dtype")
        if not fp4 and (k_sf is not None or v_sf is not None or dtype not in (None, k.dtype)):
            raise ValueError("a 16-bit cache has no scales, and its own dtype")
        for name, t in (("k", k), ("v", v)) + ((("k_sf", k_sf), ("v_sf", v_sf)) if fp4 else ()):
            if not t.is_cuda or t.device != k.device or t.dtype != k.dtype:
                raise ValueError(f"{name} must be a {k.dtype} CUDA tensor on {k.device}")
            if t.dim() != 4 or (t.shape[-1] > 1 and t.stride(-1) != 1):
                raise ValueError(f"{name} must have 4 dimensions with contiguous channels")
        if k.shape != v.shape:
            raise ValueError("k and v must have the same shape")
        dims = (0, 1, 2) if tensor_layout == "HND" else (0, 2, 1)
        D = k.shape[3] * (2 if fp4 else 1)
        if fp4:
            for c, s in ((k, k_sf), (v, v_sf)):
                if tuple(s.shape) != tuple(k.shape[:3]) + (D // 16,):
                    raise ValueError("scales must have the codes' shape with D / 16 bytes per row")
                if any(c.shape[d] > 1 and c.stride(d) != 8 * s.stride(d) for d in range(3)):
                    raise ValueError("scales must have an eighth of the codes' strides")
        self._buffers = (k, v, k_sf, v_sf)
        self.format = "fp4" if fp4 else "16bit"
        self.dtype = dtype if fp4 else k.dtype
        self.tensor_layout = tensor_layout
        self.device = k.device
        self.num_pages, self.num_kv_heads, self.page_size = (k.shape[d] for d in dims)
        self.head_dim = D
        unit = 2 if fp4 else 1  # elements per code byte
        ks, vs = (_Stride3(*(unit * _stride(t, d) for d in dims)) for t in (k, v))
        self._c = _Cache(k.data_ptr(), v.data_ptr(), k_sf.data_ptr() if fp4 else None, v_sf.data_ptr() if fp4 else None,
                         ks, vs, self.num_pages, self.page_size, self.num_kv_heads, D, _sage._dtype_code(self.dtype),
                         CACHE_FORMAT[self.format])
        self._h = _n().make_cache(ctypes.addressof(self._c), k.device.index)

    # The buffers, fixed for the cache's life: the calls hold their addresses.
    k, v, k_sf, v_sf = (property(lambda self, i=i: self._buffers[i]) for i in range(4))

    @classmethod
    def empty(cls, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int,
              dtype: torch.dtype = torch.bfloat16, format: str = "16bit", tensor_layout: str = "HND",
              device="cuda") -> "PagedKVCache":
        """A cache on buffers of its own (not initialised: only appended tokens are ever read)."""
        if format not in CACHE_FORMAT:
            raise ValueError(f"format must be one of {tuple(CACHE_FORMAT)}")
        rows = (num_pages, num_kv_heads, page_size) if tensor_layout == "HND" else (num_pages, page_size, num_kv_heads)
        if format == "16bit":
            k, v = (torch.empty(rows + (head_dim,), dtype=dtype, device=device) for _ in range(2))
            return cls(k, v, tensor_layout=tensor_layout)
        k, v = (torch.empty(rows + (head_dim // 2,), dtype=torch.uint8, device=device) for _ in range(2))
        ks, vs = (torch.empty(rows + (head_dim // 16,), dtype=torch.uint8, device=device) for _ in range(2))
        return cls(k, v, ks, vs, dtype=dtype, tensor_layout=tensor_layout)


def cache_append(cache: PagedKVCache, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor,
                 seq_lens: torch.Tensor, *, cu_seqlens: Optional[torch.Tensor] = None,
                 q: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, rope: Optional[torch.Tensor] = None,
                 interleaved: bool = False, q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Append keys and values [tokens, Hkv, D] to their sequences' pages, the keys normed and rotated to their
    positions on the way (see qk_norm_rope); FP4 caches quantize them.

    page_table int32 [B, pages], seq_lens int32 [B]: lengths with the new tokens. Rows cu_seqlens[b] ..
    cu_seqlens[b+1] are the last tokens of sequence b (int32 [B+1]; without it one row per sequence); rows
    behind cu_seqlens[B] are left alone. With q [tokens, Hq, D] the same tokens' queries are normed and rotated
    too, into q_out (may be q), which is returned. Two tokens of a call must not share a slot. A page
    outside the cache, a negative position and one beyond the rotation table are reported by
    device_error(); such a token is left out."""
    return _n().append(cache._h, k, v, page_table, seq_lens, cu_seqlens, q, q_weight, k_weight, eps, rope, interleaved,
                       q_out)


def cache_gather(cache: PagedKVCache, page_table: torch.Tensor, seq_lens: torch.Tensor, *,
                 cu_seqlens: Optional[torch.Tensor] = None, total: Optional[int] = None,
                 k_out: Optional[torch.Tensor] = None,
                 v_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Keys and values of the last cu_seqlens[b+1] - cu_seqlens[b] tokens of each sequence as packed rows
    [total, Hkv, D] (without cu_seqlens: of the last one). total counts the rows; it is needed with
    cu_seqlens unless k_out and v_out are given, and may be larger than cu_seqlens[B]. Rows without a
    token are not written. FP4 values are decoded exactly. Returns (k_out, v_out)."""
    return _n().gather(cache._h, page_table, seq_lens, cu_seqlens, total, k_out, v_out)


def decode_workspace_bytes(cache: PagedKVCache, page_table: torch.Tensor, seq_lens: torch.Tensor,
                           num_q_heads: int) -> int:
    """Workspace of sageattn_decode for these shapes."""
    return _n().workspace(cache._h, page_table, seq_lens, num_q_heads)


def sageattn_decode(q: torch.Tensor, cache: PagedKVCache, page_table: torch.Tensor, seq_lens: torch.Tensor, *,
                    sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of one new token per sequence, q [B, Hq, D], over the seq_lens[b] cached tokens of its sequence
    (its own key and value among them, once appended). Hq is a multiple of the cache's heads. A sequence
    of length 0 gets zeros, and so does a head whose scores are all -inf; out may be q itself (not another
    view of its memory). A length outside the page table is clamped and a page outside the cache counts as
    zeros, both reported by device_error(). workspace: uint8, 256-byte aligned, of at least
    decode_workspace_bytes(); one that calls share must not serve two at once (allocated per call when
    left out)."""
    return _n().decode(cache._h, q, page_table, seq_lens, sm_scale, out, workspace)


def sageattn_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: PagedKVCache, page_table: torch.Tensor,
                     seq_lens: torch.Tensor, cu_seqlens: torch.Tensor, max_seqlen: int, *,
                     cu_seqlens_kv: Optional[torch.Tensor] = None, max_seqlen_kv: Optional[int] = None,
                     total_kv: Optional[int] = None, q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, rope: Optional[torch.Tensor] = None,
                     interleaved: bool = False, is_causal: bool = True, **attn) -> torch.Tensor:
    """Prompts into the cache and their attention: cache_append (with q), cache_gather, sageattn_varlen.

    q [tokens, Hq, D], k, v [tokens, Hkv, D] packed by cu_seqlens, with no rows behind the last prompt (as
    sageattn_varlen wants them); seq_lens as in cache_append. Prompts that
    continue a cached prefix attend to all of it: cu_seqlens_kv (offsets of the whole sequences, the sums of
    seq_lens), max_seqlen_kv and total_kv then describe the keys. Keys and values are read back from the
    cache, so the prompt sees what later tokens will see, an FP4 cache's rounding included. Further keyword
    arguments go to sageattn_varlen."""
    if (cu_seqlens_kv is None) != (max_seqlen_kv is None) or (cu_seqlens_kv is None) != (total_kv is None):
        raise ValueError("cu_seqlens_kv, max_seqlen_kv and total_kv go together")
    if cu_seqlens_kv is None:
        cu_seqlens_kv, max_seqlen_kv, total_kv = cu_seqlens, max_seqlen, k.shape[0]
    q = cache_append(cache, k, v, page_table, seq_lens, cu_seqlens=cu_seqlens, q=q, q_weight=q_weight, k_weight=k_weight,
                     eps=eps, rope=rope, interleaved=interleaved)
    k, v = cache_gather(cache, page_table, seq_lens, cu_seqlens=cu_seqlens_kv, total=total_kv)
    with torch.cuda.device(cache.device):
        return _sage.sageattn_varlen(q, k, v, cu_seqlens, cu_seqlens_kv, max_seqlen, max_seqlen_kv, is_causal=is_causal,
                                     **attn)
