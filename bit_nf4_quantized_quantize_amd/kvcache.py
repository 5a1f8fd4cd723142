"""Thin binding of the 8-bit and the shared key-value cache
(include/qlora_kvcache.h) in libqlora_nf4.so.

As in `decoder`: functions carry the names of the C entry points, the calls go
through a compiled module (csrc/kv_binding.cpp), a missing one raises, all
tensors of a call must be on one device, which need not be the current one, and
work runs on the current stream of that device, or on `stream`.  The calls are
below autograd; a tensor that a call writes into (outputs given, the cache)
counts as changed in place.
"""

import collections
import ctypes

import torch

from . import binding as B
from . import decoder as D

_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float

# Every function declared in include/qlora_kvcache.h.
EXPORTED = (
    "qlora_kv_write", "qlora_kv_read", "qlora_kv_attention_workspace", "qlora_kv_attention",
    "qlora_prefix_attention_workspace", "qlora_prefix_attention",
)


class KVCacheStruct(ctypes.Structure):
    """qlora_kv_cache."""

    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("num_pages", _i64), ("page_size", _i32),
                ("kv_heads", _i32), ("head_dim", _i32), ("type", _i32)]


_cp = ctypes.POINTER(KVCacheStruct)
_SIG = {
    "qlora_kv_write": [_vp, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _i32, _vp, _vp, _f32, _i32, _vp, _cp,
                       _vp],
    "qlora_kv_read": [_cp, _vp, _i64, _i32, _vp, _vp, _vp],
    "qlora_kv_attention_workspace": [_cp, _i64, _i32, _i64, ctypes.POINTER(_i64)],
    "qlora_kv_attention": [_vp, _i64, _i64, _i32, _cp, _vp, _i64, _vp, _f32, _vp, _vp, _vp, _i64, _vp],
    "qlora_prefix_attention_workspace": [_cp, _i64, _i32, _i64, _i64, ctypes.POINTER(_i64)],
    "qlora_prefix_attention": [_vp, _i64, _i64, _i32, _cp, _vp, _i64, _vp, _vp, _i64, _vp, _f32, _vp, _vp, _vp, _i64,
                               _vp],
}
CACHE_TYPES = {torch.bfloat16: 0, torch.int8: 1, torch.float8_e4m3fn: 2}   # qlora_cache_type

_lib = None


def lib():
    """The loaded library with this header's functions declared."""
    global _lib
    if _lib is None:
        L = B.lib()
        for name, args in _SIG.items():
            f = getattr(L, name)
            f.restype, f.argtypes = _i32, args
        _lib = L
    return _lib


_native = None


def native():
    """The compiled module over this header (raises QLoraLibraryError if it is
    not built)."""
    global _native
    if _native is None:
        lib()  # the library that the module calls: a missing one is reported as such
        try:
            from . import _kvcache
        except ImportError as e:
            raise B.QLoraLibraryError(f"cannot load the module of csrc/kv_binding.cpp ({e}): build it with "
                                      "`python -m bit_nf4_quantized_quantize_amd.build`") from e
        _native = _kvcache
    return _native


class KVCache(collections.namedtuple("KVCache", "k v k_scale v_scale")):
    """The rows of one layer's paged cache: k and v [num_pages, kv_heads,
    page_size, head_dim], bfloat16, or int8 or float8_e4m3fn codes with k_scale and
    v_scale float32 [num_pages, kv_heads, page_size] (None for bfloat16): an element
    is code * scale, the scale finite, or NaN for a row that could not be held."""

    __slots__ = ()

    @classmethod
    def zeros(cls, num_pages, kv_heads, page_size, head_dim, dtype=torch.bfloat16, device="cuda"):
        """A cache of zeros."""
        if dtype not in CACHE_TYPES:
            raise ValueError("a cache is bfloat16, int8 or float8_e4m3fn")
        rows = (num_pages, kv_heads, page_size)
        k, v = (torch.zeros(*rows, head_dim, dtype=dtype, device=device) for _ in "kv")
        if dtype == torch.bfloat16:
            return cls(k, v, None, None)
        return cls(k, v, *(torch.zeros(rows, dtype=torch.float32, device=device) for _ in "kv"))


def qlora_kv_write(q, k, v, table, positions, slots, cache, q_out=None, stream=None):
    """Tokens entering the cache: returns the rotated q (None for q None) and
    stores the rotated k and v [T, kv_heads, head_dim] bfloat16 in their slots
    (int32 [T]; a slot outside the cache is not stored) of the KVCache `cache`,
    coded if that holds codes.  `table` a decoder.RopeTable, or None: no rotation.
    q_out may be q itself."""
    turns, rot, mscale, inter = (None, 0, 1.0, False) if table is None else (table.turns, table.rot_dim, table.mscale,
                                                                             table.interleaved)
    f = (_native or native()).write
    args = (q, k, v, positions, turns, rot, mscale, inter, slots, *cache, q_out)
    r = f(*args) if stream is None else None
    if r.__class__ is not tuple:
        used = (k, v, q, turns, None if table is None else positions, slots, *cache, q_out)
        r = D._call("qlora_kv_write", f, args, stream, used, r)
    return r[0]


def qlora_kv_read(cache, slots, dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
    """The keys and values in `slots` (int32 [T], any order; zeros for a slot
    outside the cache) as numbers: (k, v) [T, kv_heads, head_dim], bfloat16 or
    float32."""
    code = D._DTYPES.get(dtype)
    if code is None:
        raise ValueError("dtype must be torch.float32 or torch.bfloat16")
    f = (_native or native()).read
    args = (*cache, slots, code, k_out, v_out)
    r = f(*args) if stream is None else None
    if r.__class__ is not tuple:
        r = D._call("qlora_kv_read", f, args, stream, (*cache, slots, k_out, v_out), r)
    return r


def qlora_kv_attention(q, cache, block_table, lengths, scale=None, out=None, lse=None, stream=None):
    """decoder.qlora_paged_attention over a KVCache of any type: attention of
    one new token per sequence, q bfloat16 [S, heads, head_dim], block_table
    int32 [S, columns], lengths int32 [S]."""
    f = (_native or native()).attention
    args = (q, *cache, None, None, block_table, lengths, scale, out, lse)
    r = f(*args) if stream is None else None
    if r.__class__ is not tuple:
        r = D._call("qlora_kv_attention", f, args, stream, (q, *cache, block_table, lengths, out, lse), r)
    return r[0]


def qlora_prefix_attention(q, cache, prefix_table, prefix_len, block_table, lengths, scale=None, out=None, lse=None,
                           stream=None):
    """Attention of one new token per sequence for a batch that shares a prefix:
    q bfloat16 [S, heads, head_dim] over the first prefix_len (int32 [1], on the
    device) tokens of the pages prefix_table (int32 [columns]) and the first
    lengths[s] of row s of block_table, which hold the sequence's own tokens.
    Returns bfloat16 [S, heads, head_dim] (zeros where there is no token at all);
    `lse` (float32 [S, heads]) receives the log of the sum of exponentials."""
    if prefix_table is None or prefix_len is None:
        raise TypeError("prefix_table and prefix_len must be tensors")
    f = (_native or native()).attention
    args = (q, *cache, prefix_table, prefix_len, block_table, lengths, scale, out, lse)
    r = f(*args) if stream is None else None
    if r.__class__ is not tuple:
        used = (q, *cache, prefix_table, prefix_len, block_table, lengths, out, lse)
        r = D._call("qlora_prefix_attention", f, args, stream, used, r)
    return r[0]
