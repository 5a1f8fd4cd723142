"""Thin binding of the decoder-block operators (include/qlora_decoder.h) in
libqlora_nf4.so: the residual update with its norms, rotary positions, and
decoding from a paged key-value cache.

As in `binding`: argument marshalling only, functions carry the names of the C
entry points, and a missing library raises.  The calls that a token makes go
through a compiled module (csrc/decoder_binding.cpp), which checks the tensors
and allocates what a call returns: decoding has little work per call, and the
same through ctypes costs more than the kernels.  All tensors of a call must be
on one device, which need not be the current one.  Work runs on the current
stream of that device, or on `stream`; outputs and workspaces a call allocates
belong to the stream it runs on, and tensors it is given are marked as used
there, so their memory is not handed out again before the call has run.

These calls are below autograd: results do not require gradients, whatever the
arguments do (block.norm_residual and block.rope are the differentiable forms).
A tensor that a call writes into (outputs given, the block table, the caches)
counts as changed in place, so a backward that saved it raises.
"""

import collections
import contextlib
import ctypes

import torch

from . import binding as B

_vp, _i64, _i32, _f32, _f64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_double

NORM_MAX_WIDTH = 16384
PLAN_MAX_SEQS = 4096
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

# Every function declared in include/qlora_decoder.h.
EXPORTED = (
    "qlora_norm_residual_fwd", "qlora_norm_residual_bwd_workspace", "qlora_norm_residual_bwd",
    "qlora_rope_frequencies", "qlora_rope", "qlora_rope_cache_write", "qlora_paged_plan",
    "qlora_paged_attention_workspace", "qlora_paged_attention",
)

_SIG = {
    "qlora_norm_residual_fwd": [_vp, _i32, _vp, _i32, _i64, _i64, _vp, _vp, _f32, _vp, _f32, _vp, _vp, _vp],
    "qlora_norm_residual_bwd_workspace": [_i64, _i64, _i32, _i32, _i32, ctypes.POINTER(_i64)],
    "qlora_norm_residual_bwd": [_vp, _vp, _i32, _vp, _vp, _i32, _i64, _i64, _vp, _vp, _f32, _vp, _f32, _vp, _vp, _vp,
                                _vp, _vp, _vp, _i64, _vp],
    "qlora_rope_frequencies": [_i32, _f64, _i32, _f64, _f64, _f64, _f64, ctypes.POINTER(_f64), ctypes.POINTER(_f32)],
    "qlora_rope": [_vp, _i64, _i32, _vp, _i64, _vp, _i64, _i32, _vp, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _f32,
                   _i32, _i32, _vp],
    "qlora_rope_cache_write": [_vp, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _i64, _i32, _i32, _vp, _vp,
                               _f32, _i32, _vp, _vp, _vp, _i64, _i32, _vp],
    "qlora_paged_plan": [_vp, _vp, _i64, _i32, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp],
    "qlora_paged_attention_workspace": [_i64, _i32, _i32, _i32, _i64, _i32, ctypes.POINTER(_i64)],
    "qlora_paged_attention": [_vp, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _i64, _i32, _vp, _i64, _vp, _f32, _vp, _vp,
                              _vp, _i64, _vp],
}

_lib = None
_DTYPES = {torch.float32: B.QLORA_DTYPE_F32, torch.bfloat16: B.QLORA_DTYPE_BF16}


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
            from . import _decoder
        except ImportError as e:
            raise B.QLoraLibraryError(f"cannot load the module of csrc/decoder_binding.cpp ({e}): build it with "
                                      "`python -m bit_nf4_quantized_quantize_amd.build`") from e
        _native = _decoder
    return _native


@contextlib.contextmanager
def _there(stream, tensors):
    """Makes the tensors' device, and `stream` if given, current for a call."""
    given = [t for t in tensors if t is not None]
    dev = given[0].device
    for t in given:
        if t.device.type != "cuda":
            raise ValueError("qlora_nf4 tensors must live on a HIP device")
        if t.device != dev:
            raise ValueError("all tensors of a call must be on one device")
    if stream is None:
        with torch.cuda.device(dev):
            yield
        return
    if stream.device != dev:
        raise ValueError("stream must belong to the tensors' device")
    if stream != torch.cuda.current_stream(dev):
        for t in given:
            t.record_stream(stream)
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        yield


def _call(name, f, args, stream, tensors, r):
    """The results of f(*args), a function of the module.  r: what the call as
    things stood gave, when there is no `stream`: None (the tensors are on
    another device) or a status."""
    if r is None:
        with _there(stream, tensors):
            r = f(*args)
    if r.__class__ is not tuple:
        B._check(r, name)
    return r


# --------------------------------------------------- norm, gate and residual

def qlora_norm_residual_fwd(x, h=None, w_pre=None, w_post=None, gate=None, alpha=1.0, eps=1e-6, n_dtype=None, xo=None,
                            n=None, stream=None):
    """The step between two branches: xo = x + alpha * gate * norm(h) w_post,
    n = norm(xo) w_pre (rms norms over the last dimension).  x [..., D] float32
    or bfloat16; h (or None) of x's shape, bfloat16 or x's type; gains and gate
    float32 [D] or None.  Returns (xo, n): xo is x when h is None, n is None
    without w_pre and has h's type (n_dtype, or x's, without h).  xo may be
    given as x itself: the stream is then updated in place."""
    nd = -1 if n_dtype is None else _DTYPES.get(n_dtype)
    if nd is None:
        raise ValueError("n_dtype must be torch.float32 or torch.bfloat16")
    f = (_native or native()).norm_fwd
    args = (x, h, w_pre, w_post, gate, alpha, eps, nd, xo, n)
    r = f(*args) if stream is None else None
    if r.__class__ is tuple:
        return r
    return _call("qlora_norm_residual_fwd", f, args, stream, (x, h, w_pre, w_post, gate, xo, n), r)


NormGrads = collections.namedtuple("NormGrads", "dx dh dw_pre dw_post dgate")


def qlora_norm_residual_bwd(dxo, dn, xo, h=None, w_pre=None, w_post=None, gate=None, alpha=1.0, eps=1e-6,
                            need_dh=True, need_gains=False, dx=None, dh=None, stream=None):
    """Gradients of qlora_norm_residual_fwd: dxo, dn (either may be None) the
    gradients of its outputs, xo the stream it returned, h its branch (needed
    for w_post and the gradient of the gate).  Returns NormGrads: dx, dh (None
    without need_dh) and, with need_gains, the float32 gradients of the gains
    and the gate that the forward had; need_gains may also name the wanted ones
    of "w_pre", "w_post" and "gate"."""
    wanted = 7 if need_gains is True else 0
    if need_gains and not wanted:
        wanted = ("w_pre" in need_gains) + 2 * ("w_post" in need_gains) + 4 * ("gate" in need_gains)
    f = (_native or native()).norm_bwd
    args = (dxo, dn, xo, h, w_pre, w_post, gate, alpha, eps, need_dh, wanted, dx, dh)
    r = f(*args) if stream is None else None
    if r.__class__ is not tuple:
        r = _call("qlora_norm_residual_bwd", f, args, stream, (xo, dxo, dn, h, w_pre, w_post, gate, dx, dh), r)
    return NormGrads._make(r)


# ---------------------------------------------------------- rotary positions

def qlora_rope_frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0,
                           beta_slow=1.0):
    """(turns per position of each pair as a list of rot_dim / 2 floats, factor
    of the rotated values); see qlora_rope_scaling for `scaling`."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {', '.join(ROPE_SCALING)}")
    if rot_dim > 1024:
        raise ValueError("rot_dim must be at most 1024")
    turns, m = (_f64 * max(rot_dim // 2, 1))(), _f32(0.0)
    status = (_lib or lib()).qlora_rope_frequencies(
        rot_dim, base, ROPE_SCALING[scaling], factor, original_len, beta_fast, beta_slow, turns, ctypes.byref(m))
    if status:
        B._check(status, "qlora_rope_frequencies")
    return list(turns), m.value


class RopeTable:
    """The frequencies of rotary positions on a device, built once per model:
    `turns` (float64 [rot_dim / 2]), `mscale`, and the pair layout."""

    def __init__(self, rot_dim, base=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0,
                 beta_slow=1.0, interleaved=False, device=None):
        turns, self.mscale = qlora_rope_frequencies(rot_dim, base, scaling, factor, original_len, beta_fast,
                                                    beta_slow)
        self.rot_dim, self.interleaved = int(rot_dim), bool(interleaved)
        self.turns = torch.tensor(turns, dtype=torch.float64, device=device if device is not None else "cuda")


def qlora_rope(q, k, table, positions, inverse=False, q_out=None, k_out=None, stream=None):
    """Rotates q [T, heads, head_dim] and k (either may be None) to `positions`
    (int32 [T]); tokens may be strided, float32 or bfloat16.  With `inverse`
    the gradient of that.  Returns (q_out, k_out); q_out and k_out may be q and
    k themselves."""
    f = (_native or native()).rope
    args = (q, k, positions, table.turns, table.rot_dim, table.mscale, table.interleaved, inverse, q_out, k_out)
    r = f(*args) if stream is None else None
    if r.__class__ is tuple:
        return r
    return _call("qlora_rope", f, args, stream, (q, k, table.turns, positions, q_out, k_out), r)


# ------------------------------------------------------ paged key-value cache

def qlora_rope_cache_write(q, k, v, table, positions, slots, k_cache, v_cache, q_out=None, stream=None):
    """Tokens entering the cache: returns the rotated q (None for q None) and
    stores the rotated k and v [T, kv_heads, head_dim] in their slots (int32
    [T]; a slot outside the cache is not stored) of the bfloat16 caches
    [num_pages, kv_heads, page_size, head_dim].  `table` None: no rotation."""
    turns, rot, mscale, inter = (None, 0, 1.0, False) if table is None else (table.turns, table.rot_dim, table.mscale,
                                                                             table.interleaved)
    f = (_native or native()).cache_write
    args = (q, k, v, positions, turns, rot, mscale, inter, slots, k_cache, v_cache, q_out)
    r = f(*args) if stream is None else None
    if r.__class__ is not tuple:
        used = (k, v, q, turns, None if table is None else positions, slots, k_cache, v_cache, q_out)
        r = _call("qlora_rope_cache_write", f, args, stream, used, r)
    return r[0]


PagedPlan = collections.namedtuple("PagedPlan", "total_lens starts slots positions pages_needed")


def qlora_paged_plan(cached_lens, new_lens, free_pages, block_table, page_size, tokens, out=None, stream=None):
    """Pages, slots and positions of a batch (all int32): sequence s has
    cached_lens[s] tokens in the cache and gets new_lens[s] more.  Takes pages
    from the front of free_pages, writes them into block_table [S, columns],
    and returns PagedPlan: total_lens [S], starts [S + 1], slots and positions
    [tokens] (rows behind the last new token: -1 and 0) and pages_needed [1],
    parts of one allocation.  `out`: a PagedPlan of these shapes to write to."""
    f = (_native or native()).plan
    args = (cached_lens, new_lens, free_pages, block_table, page_size, tokens, out)
    r = f(*args) if stream is None else None
    if r.__class__ is not tuple:
        r = _call("qlora_paged_plan", f, args, stream, (*args[:4], *(out or ())), r)
    return PagedPlan._make(r) if out is None else out


def qlora_paged_attention(q, k_cache, v_cache, block_table, lengths, scale=None, out=None, lse=None, stream=None):
    """Attention of one new token per sequence over the cache: q bfloat16 [S,
    heads, head_dim], block_table int32 [S, columns], lengths int32 [S] (tokens
    in the cache, the new one among them), scale 1 / sqrt(head_dim) unless
    given.  Returns bfloat16 [S, heads, head_dim] (zeros for a length of 0);
    `lse` (float32 [S, heads]) receives the log of the sum of exponentials."""
    f = (_native or native()).attention
    args = (q, k_cache, v_cache, block_table, lengths, scale, out, lse)
    r = f(*args) if stream is None else None
    if r.__class__ is not tuple:
        r = _call("qlora_paged_attention", f, args, stream, (q, k_cache, v_cache, block_table, lengths, out, lse), r)
    return r[0]
