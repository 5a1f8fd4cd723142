"""Thin ctypes binding of the decoder-block operators (include/qlora_decoder.h)
in libqlora_nf4.so: the residual update with its norms, rotary positions, and
decoding from a paged key-value cache.

As in `binding`: argument marshalling only, functions carry the names of the C
entry points, and a missing library raises.  All tensors of a call must be on
one device, which need not be the current one.  Work runs on the current
stream of that device, or on `stream`; outputs and workspaces a call allocates
belong to the stream it runs on, and tensors it is given are marked as used
there, so their memory is not handed out again before the call has run.
"""

import collections
import contextlib
import ctypes
import functools
import math

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


def _ptr(t):
    return None if t is None else t.data_ptr()


_raw_stream = torch._C._cuda_getCurrentRawStream  # what torch.cuda.current_stream wraps, without the object
_device = torch._C._cuda_getDevice


def _here(stream, *tensors):
    """The handle of the stream to launch on if the call can run as things
    stand (the tensors' device is the current one and `stream`, if given, its
    current stream), else None."""
    dev = None
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if i != dev:
                if i < 0:
                    raise ValueError("qlora_nf4 tensors must live on a HIP device")
                if dev is not None:
                    raise ValueError("all tensors of a call must be on one device")
                dev = i
    if dev != _device():
        return None
    raw = _raw_stream(dev)
    return raw if stream is None or (stream.cuda_stream == raw and stream.device_index == dev) else None


@contextlib.contextmanager
def _there(stream, *tensors):
    """Makes the tensors' device, and `stream` if given, current, for a call that
    cannot run as things stand."""
    given = [t for t in tensors if t is not None]
    dev = given[0].device
    if stream is None:
        with torch.cuda.device(dev):
            yield
        return
    if stream.device != dev:
        raise ValueError("stream must belong to the tensors' device")
    for t in given:
        t.record_stream(stream)
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        yield


def _dense(t, name, shape, dtypes):
    if t.dtype not in dtypes or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)} and type "
                         f"{' or '.join(str(d) for d in dtypes)}")


def _new_like(t):
    """A contiguous tensor of t's shape, type and device."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


_F32, _BF16 = (torch.float32,), (torch.bfloat16,)


# --------------------------------------------------- norm, gate and residual

def qlora_norm_residual_fwd(x, h=None, w_pre=None, w_post=None, gate=None, alpha=1.0, eps=1e-6, n_dtype=None, xo=None,
                            n=None, stream=None):
    """The step between two branches: xo = x + alpha * gate * norm(h) w_post,
    n = norm(xo) w_pre (rms norms over the last dimension).  x [..., D] float32
    or bfloat16; h (or None) of x's shape, bfloat16 or x's type; gains and gate
    float32 [D] or None.  Returns (xo, n): xo is x when h is None, n is None
    without w_pre and has h's type (n_dtype, or x's, without h).  xo may be
    given as x itself: the stream is then updated in place."""
    shape, xt = x.shape, x.dtype
    D = shape[-1]
    if xt not in _DTYPES or not x.is_contiguous():
        _dense(x, "x", shape, _DTYPES)
    if h is not None:
        _dense(h, "h", shape, _DTYPES)
        nd = h.dtype
        if n_dtype is not None and n_dtype != nd:
            raise ValueError("n has the type of h")
    else:
        nd = n_dtype if n_dtype is not None else xt
        if nd not in _DTYPES:
            raise ValueError("n_dtype must be torch.float32 or torch.bfloat16")
    for t, name in ((w_pre, "w_pre"), (w_post, "w_post"), (gate, "gate")):
        if t is not None:
            _dense(t, name, (D,), _F32)
    on = _here(stream, x, h, w_pre, w_post, gate, xo, n)
    if on is None:
        with _there(stream, x, h, w_pre, w_post, gate, xo, n):
            return qlora_norm_residual_fwd(x, h, w_pre, w_post, gate, alpha, eps, n_dtype, xo, n)
    if xo is not None:
        _dense(xo, "xo", shape, (xt,))
    elif h is not None:
        xo = torch.empty_like(x)
    if n is not None:
        _dense(n, "n", shape, (nd,))
    elif w_pre is not None:
        n = torch.empty_like(x) if nd == xt else torch.empty_like(x, dtype=nd)
    status = (_lib or lib()).qlora_norm_residual_fwd(
        x.data_ptr(), _DTYPES[xt], _ptr(h), _DTYPES[nd], x.numel() // D if D else 0, D, _ptr(w_post), _ptr(gate),
        float(alpha), _ptr(w_pre), float(eps), _ptr(xo), _ptr(n), on)
    if status:
        B._check(status, "qlora_norm_residual_fwd")
    return (x if xo is None else xo), n


NormGrads = collections.namedtuple("NormGrads", "dx dh dw_pre dw_post dgate")


@functools.lru_cache(maxsize=256)
def _norm_bwd_workspace(T, D, xt, ht):
    nws = _i64(0)
    status = (_lib or lib()).qlora_norm_residual_bwd_workspace(
        T, D, xt, ht, 3, ctypes.byref(nws))
    if status:
        B._check(status, "qlora_norm_residual_bwd_workspace")
    return nws.value


def qlora_norm_residual_bwd(dxo, dn, xo, h=None, w_pre=None, w_post=None, gate=None, alpha=1.0, eps=1e-6,
                            need_dh=True, need_gains=False, dx=None, dh=None, stream=None):
    """Gradients of qlora_norm_residual_fwd: dxo, dn (either may be None) the
    gradients of its outputs, xo the stream it returned, h its branch (needed
    for w_post and the gradient of the gate).  Returns NormGrads: dx, dh (None
    without need_dh) and, with need_gains, the float32 gradients of the gains
    and the gate that the forward had; need_gains may also name the wanted ones
    of "w_pre", "w_post" and "gate"."""
    shape, xt = xo.shape, xo.dtype
    D = shape[-1]
    T = xo.numel() // D if D else 0
    _dense(xo, "xo", shape, _DTYPES)
    hd = next((t.dtype for t in (h, dn, dh) if t is not None), xt)
    if hd not in _DTYPES:
        raise ValueError("h, dn and dh must be float32 or bfloat16")
    for t, name, dt in ((dxo, "dxo", xt), (dx, "dx", xt), (dn, "dn", hd), (h, "h", hd), (dh, "dh", hd)):
        if t is not None:
            _dense(t, name, shape, (dt,))
    for t, name in ((w_pre, "w_pre"), (w_post, "w_post"), (gate, "gate")):
        if t is not None:
            _dense(t, name, (D,), _F32)
    on = _here(stream, xo, dxo, dn, h, w_pre, w_post, gate, dx, dh)
    if on is None:
        with _there(stream, xo, dxo, dn, h, w_pre, w_post, gate, dx, dh):
            return qlora_norm_residual_bwd(dxo, dn, xo, h, w_pre, w_post, gate, alpha, eps, need_dh, need_gains, dx,
                                           dh)
    dx = torch.empty_like(xo) if dx is None else dx
    if dh is None and need_dh:
        dh = torch.empty_like(xo, dtype=hd)
    dw_pre = dw_post = dgate = ws = None
    nws = 0
    if need_gains:
        wanted = ("w_pre", "w_post", "gate") if need_gains is True else need_gains
        new = lambda: torch.empty(D, dtype=torch.float32, device=xo.device)  # noqa: E731
        dw_pre = new() if dn is not None and "w_pre" in wanted else None
        dw_post = new() if w_post is not None and "w_post" in wanted else None
        dgate = new() if gate is not None and "gate" in wanted else None
        nws = _norm_bwd_workspace(T, D, _DTYPES[xt], _DTYPES[hd])
        ws = torch.empty(nws, dtype=torch.uint8, device=xo.device)
    status = (_lib or lib()).qlora_norm_residual_bwd(
        _ptr(dxo), xo.data_ptr(), _DTYPES[xt], _ptr(dn), _ptr(h), _DTYPES[hd], T, D, _ptr(w_post), _ptr(gate),
        float(alpha), _ptr(w_pre), float(eps), dx.data_ptr(), _ptr(dh), _ptr(dw_post), _ptr(dgate), _ptr(dw_pre),
        _ptr(ws), nws, on)
    if status:
        B._check(status, "qlora_norm_residual_bwd")
    return NormGrads(dx, dh, dw_pre, dw_post, dgate)


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


def _heads(t, name, T, d, dtype):
    """[T, heads, head_dim] with dense heads; returns (heads, token stride)."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != T or shape[2] != d or t.dtype != dtype:
        raise ValueError(f"{name} must be a {dtype} tensor [{T}, heads, {d}]")
    h = shape[1]
    if t.is_contiguous():
        return h, h * d
    st = t.stride()
    if (d > 1 and st[2] != 1) or (h > 1 and st[1] != d):
        raise ValueError(f"the heads of a token of {name} must be dense")
    return h, (st[0] if T > 1 else h * d)


def _index(t, name, shape):
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape}")


def qlora_rope(q, k, table, positions, inverse=False, q_out=None, k_out=None, stream=None):
    """Rotates q [T, heads, head_dim] and k (either may be None) to `positions`
    (int32 [T]); tokens may be strided, float32 or bfloat16.  With `inverse`
    the gradient of that.  Returns (q_out, k_out); q_out and k_out may be q and
    k themselves."""
    t = q if q is not None else k
    if t is None or t.dim() != 3:
        raise ValueError("q or k must be given, as [T, heads, head_dim]")
    dt = t.dtype
    if dt not in _DTYPES:
        raise ValueError("q and k must be float32 or bfloat16")
    T, _, d = t.shape
    _index(positions, "positions", (T,))
    on = _here(stream, q, k, table.turns, positions, q_out, k_out)
    if on is None:
        with _there(stream, q, k, table.turns, positions, q_out, k_out):
            return qlora_rope(q, k, table, positions, inverse, q_out, k_out)
    qh = qs = qos = kh = ks = kos = 0
    if q is not None:
        qh, qs = _heads(q, "q", T, d, dt)
        if q_out is None:
            q_out, qos = _new_like(q), qh * d
        else:
            h, qos = _heads(q_out, "q_out", T, d, dt)
            if h != qh:
                raise ValueError("q_out must have the heads of q")
    else:
        q_out = None
    if k is not None:
        kh, ks = _heads(k, "k", T, d, dt)
        if k_out is None:
            k_out, kos = _new_like(k), kh * d
        else:
            h, kos = _heads(k_out, "k_out", T, d, dt)
            if h != kh:
                raise ValueError("k_out must have the heads of k")
    else:
        k_out = None
    status = (_lib or lib()).qlora_rope(
        _ptr(q), qs, qh, _ptr(q_out), qos, _ptr(k), ks, kh, _ptr(k_out), kos, T, d, table.rot_dim, _DTYPES[dt],
        positions.data_ptr(), table.turns.data_ptr(), table.mscale, table.interleaved, bool(inverse), on)
    if status:
        B._check(status, "qlora_rope")
    return q_out, k_out


# ------------------------------------------------------ paged key-value cache

def _cache(k_cache, v_cache):
    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError("the caches must be [num_pages, kv_heads, page_size, head_dim]")
    _dense(k_cache, "k_cache", shape, _BF16)
    _dense(v_cache, "v_cache", shape, _BF16)
    return shape


def qlora_rope_cache_write(q, k, v, table, positions, slots, k_cache, v_cache, q_out=None, stream=None):
    """Tokens entering the cache: returns the rotated q (None for q None) and
    stores the rotated k and v [T, kv_heads, head_dim] in their slots (int32
    [T]; a slot outside the cache is not stored) of the bfloat16 caches
    [num_pages, kv_heads, page_size, head_dim].  `table` None: no rotation."""
    pages, kvh, page, d = _cache(k_cache, v_cache)
    T = k.shape[0]
    bf = torch.bfloat16
    _index(slots, "slots", (T,))
    turns, rot, mscale, inter = None, 0, 1.0, False
    if table is not None:
        turns, rot, mscale, inter = table.turns, table.rot_dim, table.mscale, table.interleaved
        _index(positions, "positions", (T,))
    else:
        positions = None
    on = _here(stream, k, v, q, turns, positions, slots, k_cache, v_cache, q_out)
    if on is None:
        with _there(stream, k, v, q, turns, positions, slots, k_cache, v_cache, q_out):
            return qlora_rope_cache_write(q, k, v, table, positions, slots, k_cache, v_cache, q_out)
    kh, ks = _heads(k, "k", T, d, bf)
    vh, vs = _heads(v, "v", T, d, bf)
    if kh != kvh or vh != kvh:
        raise ValueError("k and v must have the cache's heads")
    qh = qs = qos = 0
    if q is not None:
        qh, qs = _heads(q, "q", T, d, bf)
        if q_out is None:
            q_out, qos = _new_like(q), qh * d
        else:
            h, qos = _heads(q_out, "q_out", T, d, bf)
            if h != qh:
                raise ValueError("q_out must have the heads of q")
    else:
        q_out = None
    status = (_lib or lib()).qlora_rope_cache_write(
        _ptr(q), qs, qh, _ptr(q_out), qos, k.data_ptr(), ks, v.data_ptr(), vs, kvh, T, d, rot, _ptr(positions),
        _ptr(turns), mscale, inter, slots.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), pages, page, on)
    if status:
        B._check(status, "qlora_rope_cache_write")
    return q_out


PagedPlan = collections.namedtuple("PagedPlan", "total_lens starts slots positions pages_needed")


def qlora_paged_plan(cached_lens, new_lens, free_pages, block_table, page_size, tokens, out=None, stream=None):
    """Pages, slots and positions of a batch (all int32): sequence s has
    cached_lens[s] tokens in the cache and gets new_lens[s] more.  Takes pages
    from the front of free_pages, writes them into block_table [S, columns],
    and returns PagedPlan: total_lens [S], starts [S + 1], slots and positions
    [tokens] (rows behind the last new token: -1 and 0) and pages_needed [1],
    parts of one allocation.  `out`: a PagedPlan of these shapes to write to."""
    if not 0 < page_size < 2 ** 31 or not 0 <= tokens < 2 ** 31:
        raise ValueError("page_size must be positive and tokens not negative")
    S = cached_lens.shape[0]
    _index(cached_lens, "cached_lens", (S,))
    _index(new_lens, "new_lens", (S,))
    nfree = free_pages.numel()
    _index(free_pages, "free_pages", (nfree,))
    cols = block_table.shape[-1]
    _index(block_table, "block_table", (S, cols))
    on = _here(stream, cached_lens, new_lens, free_pages, block_table, *(out or ()))
    if on is None:
        with _there(stream, cached_lens, new_lens, free_pages, block_table, *(out or ())):
            return qlora_paged_plan(cached_lens, new_lens, free_pages, block_table, page_size, tokens, out)
    if out is None:
        sizes = (S, S + 1, tokens, tokens, 1)
        out = PagedPlan._make(cached_lens.new_empty(2 * (S + tokens + 1)).split_with_sizes(sizes))
    else:
        for name, n in zip(PagedPlan._fields, (S, S + 1, tokens, tokens, 1)):
            _index(getattr(out, name), name, (n,))
    total, starts, slots, positions, needed = out
    status = (_lib or lib()).qlora_paged_plan(
        cached_lens.data_ptr(), new_lens.data_ptr(), S, page_size, free_pages.data_ptr(), nfree, block_table.data_ptr(),
        cols, tokens, total.data_ptr(), starts.data_ptr(), slots.data_ptr(), positions.data_ptr(), needed.data_ptr(), on)
    if status:
        B._check(status, "qlora_paged_plan")
    return out


@functools.lru_cache(maxsize=256)
def _attention_workspace(S, H, kvh, d, cols, page):
    nws = _i64(0)
    status = (_lib or lib()).qlora_paged_attention_workspace(
        S, H, kvh, d, cols, page, ctypes.byref(nws))
    if status:
        B._check(status, "qlora_paged_attention_workspace")
    return nws.value


def qlora_paged_attention(q, k_cache, v_cache, block_table, lengths, scale=None, out=None, lse=None, stream=None):
    """Attention of one new token per sequence over the cache: q bfloat16 [S,
    heads, head_dim], block_table int32 [S, columns], lengths int32 [S] (tokens
    in the cache, the new one among them), scale 1 / sqrt(head_dim) unless
    given.  Returns bfloat16 [S, heads, head_dim] (zeros for a length of 0);
    `lse` (float32 [S, heads]) receives the log of the sum of exponentials."""
    pages, kvh, page, d = _cache(k_cache, v_cache)
    S = q.shape[0]
    H, qs = _heads(q, "q", S, d, torch.bfloat16)
    _index(lengths, "lengths", (S,))
    cols = block_table.shape[-1]
    _index(block_table, "block_table", (S, cols))
    on = _here(stream, q, k_cache, v_cache, block_table, lengths, out, lse)
    if on is None:
        with _there(stream, q, k_cache, v_cache, block_table, lengths, out, lse):
            return qlora_paged_attention(q, k_cache, v_cache, block_table, lengths, scale, out, lse)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _new_like(q)
    else:
        _dense(out, "out", (S, H, d), _BF16)
    if lse is not None:
        _dense(lse, "lse", (S, H), _F32)
    nws = _attention_workspace(S, H, kvh, d, cols, page)
    ws = q.new_empty(nws // 2) if nws else None  # in q's elements of two bytes
    status = (_lib or lib()).qlora_paged_attention(
        q.data_ptr(), qs, S, H, kvh, d, k_cache.data_ptr(), v_cache.data_ptr(), pages, page, block_table.data_ptr(),
        cols, lengths.data_ptr(), float(scale), out.data_ptr(), _ptr(lse), _ptr(ws), nws, on)
    if status:
        B._check(status, "qlora_paged_attention")
    return out
