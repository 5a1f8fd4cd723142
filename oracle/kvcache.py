"""The 8-bit and the shared key-value cache by their definitions, in fp64.

A row (the keys or the values of one token and kv head) of largest size a is
held as codes and a scale: scale = a / M in fp32, M = 127 for whole numbers and
448 for E4M3, code = the one nearest to z / scale, ties to the even code.  Rows
with a NaN or an infinity have scale NaN and codes 0.
"""

import math

import numpy as np

MOST = {"int8": 127.0, "e4m3": 448.0}

# The 127 sizes of E4M3 in order: seven subnormal steps of 2^-9, then eight to
# each power of two from 2^-6 up to 448.
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16)
                                                     for m in range(8)][:119])


def nearest(y, kind):
    """The codes (as numbers) nearest to y, ties to the even one."""
    if kind == "int8":
        return np.clip(np.rint(y), -127, 127)
    a = np.minimum(np.abs(y), 448.0)
    low = np.clip(np.searchsorted(E4M3, a, side="right") - 1, 0, 125)
    under, over = a - E4M3[low], E4M3[low + 1] - a
    return np.copysign(E4M3[low + ((over < under) | ((over == under) & (low % 2 == 1)))], y)


def encode(z, kind):
    """(codes as numbers, fp32 scales) of rows z [..., d]."""
    z = np.asarray(z, np.float64)
    top = np.abs(z).max(-1)
    ok = np.isfinite(top)
    scale = np.where(ok, np.where(ok, top, 0.0) / MOST[kind], np.nan).astype(np.float32)
    s = scale.astype(np.float64)[..., None]
    held = ok[..., None] & (s > 0)
    y = np.divide(np.where(held, z, 0.0), np.where(held, s, 1.0))
    return nearest(y, kind), scale


def half_step(code, kind):
    """Half of the distance between the codes next to a code, the larger one."""
    if kind == "int8":
        return np.full_like(code, 0.5)
    e = np.floor(np.log2(np.maximum(np.abs(code), 2.0 ** -6)))
    return 2.0 ** (e - 4)


def values(codes, scale):
    """The numbers that rows stand for."""
    z = np.asarray(codes, np.float64)
    return z if scale is None else z * np.asarray(scale, np.float64)[..., None]


def read(k, slots):
    """Rows of values [pages, KV, page, d] in slots: [T, KV, d], zeros outside."""
    pages, KV, page, d = k.shape
    out = np.zeros((len(slots), KV, d))
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            out[t] = k[s // page, :, s % page]
    return out


def _tokens(table, n, page, pages):
    n = min(max(int(n), 0), len(table) * page)
    at = [(int(table[i // page]), i % page) for i in range(n)]
    return [(p, o) for p, o in at if 0 <= p < pages]


def attention(q, k, v, table, lengths, scale, prefix_table=(), prefix_len=0):
    """(out, lse, weight) in fp64 for values k, v [pages, KV, page, d]: sequence s
    attends to the prefix and its own tokens; weight = sum_i p_i |v_i|."""
    q = np.asarray(q, np.float64)
    S, H, d = q.shape
    pages, KV, page, _ = k.shape
    out, wt, lse = np.zeros((S, H, d)), np.zeros((S, H, d)), np.full((S, H), -np.inf)
    common = _tokens(prefix_table, prefix_len, page, pages)
    for s in range(S):
        at = common + _tokens(table[s], lengths[s], page, pages)
        if not at:
            continue
        p_, o_ = np.array([a[0] for a in at]), np.array([a[1] for a in at])
        for h in range(H):
            j = h // (H // KV)
            kk, vv = k[p_, j, o_], v[p_, j, o_]
            sc = scale * (kk @ q[s, h])
            top = sc.max()
            e = np.exp(sc - top)
            den = e.sum()
            out[s, h], wt[s, h], lse[s, h] = e @ vv / den, e @ np.abs(vv) / den, top + math.log(den)
    return out, lse, wt
