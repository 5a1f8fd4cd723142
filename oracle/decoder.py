"""The decoder-block operators around the linears, from their definitions in
fp64 (oracle side).  Test infrastructure only; see the package docstring.

  norm_residual / norm_residual_grads   the step between two branches of a
      block: residual update with norms, gate and scale, and its gradients
  rope_frequencies / rope               rotary positions (Su et al., RoFormer,
      arXiv 2104.09864), with the stretched frequencies of Peng et al., YaRN,
      arXiv 2309.00071
  paged_attention                       attention of one token over a paged
      cache
  paged_plan                            pages, slots and positions of a batch
  block                                 the decoder block of oracle/block.py with
      rotary positions, norms behind the branches, gates and a residual scale

numpy (torch's fp64 autograd for the block); nothing is shared with the HIP path.
"""

import math

import numpy as np
import torch

from . import block as oblock


def _f(a):
    return np.asarray(a, np.float64)


# ------------------------------------------------------- norm and residual

def rms(z, eps):
    return np.sqrt(np.mean(z * z, axis=-1, keepdims=True) + eps)


def norm_residual(x, h, w_pre, w_post=None, gate=None, alpha=1.0, eps=1e-6):
    """(xo, n); h None: xo = x."""
    xo = _f(x)
    if h is not None:
        u = _f(h)
        if w_post is not None:
            u = u / rms(u, eps) * _f(w_post)
        if gate is not None:
            u = u * _f(gate)
        xo = xo + alpha * u
    n = None if w_pre is None else xo / rms(xo, eps) * _f(w_pre)
    return xo, n


def rms_grad(z, dy, eps):
    """Gradient for z of sum(dy * z / rms(z))."""
    r = rms(z, eps)
    return dy / r - z * np.mean(dy * z, axis=-1, keepdims=True) / r ** 3


def norm_residual_grads(dxo, dn, xo, h, w_pre, w_post=None, gate=None, alpha=1.0, eps=1e-6):
    """dict dx, dh, dw_pre, dw_post, dgate of sum(dxo * xo) + sum(dn * n); xo is
    the forward's output (its rounding included)."""
    xo = _f(xo)
    dx = np.zeros_like(xo) if dxo is None else _f(dxo)
    out = {}
    if dn is not None:
        dn = _f(dn)
        dx = dx + rms_grad(xo, dn * _f(w_pre), eps)
        out["dw_pre"] = (dn * xo / rms(xo, eps)).reshape(-1, xo.shape[-1]).sum(0)
    out["dx"] = dx
    one = np.ones(xo.shape[-1])
    g = one if gate is None else _f(gate)
    w = one if w_post is None else _f(w_post)
    b = alpha * dx * g
    if h is not None:
        h = _f(h)
        y = h / rms(h, eps) if w_post is not None else h
        out["dgate"] = (alpha * dx * w * y).reshape(-1, xo.shape[-1]).sum(0)
        out["dw_post"] = (b * y).reshape(-1, xo.shape[-1]).sum(0)
    out["dh"] = rms_grad(h, b * w, eps) if w_post is not None else b
    return out


# ------------------------------------------------------------------- rotary

def rope_frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0,
                     beta_slow=1.0):
    """(angle per position of each pair in radians, factor of the values)."""
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** (-np.arange(0, rot_dim, 2, dtype=np.float64) / rot_dim)
    m = 1.0
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        g = np.clip((original_len * f / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
        f = (1 - g) * f / factor + g * f
        m = 0.1 * math.log(factor) + 1.0
    return f, m


def rope(z, positions, freq, mscale=1.0, interleaved=False, inverse=False):
    """z [T, heads, head_dim]; the first 2 len(freq) elements of a head turn."""
    z = _f(z).copy()
    r = 2 * len(freq)
    if r == 0:
        return z
    t = _f(positions)[:, None, None] * freq * (-1.0 if inverse else 1.0)
    c, s = mscale * np.cos(t), mscale * np.sin(t)
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    x, y = z[..., a].copy(), z[..., b].copy()
    z[..., a], z[..., b] = x * c - y * s, x * s + y * c
    return z


# -------------------------------------------------------------- paged cache

def paged_attention(q, k_cache, v_cache, table, lengths, scale):
    """(out, lse, weight) in fp64; weight [S, H, d] = sum_i p_i |v_i|, the scale
    of the rounding of the weights.  Caches [pages, kv_heads, page, d]."""
    q = _f(q)
    S, H, d = q.shape
    pages, KV, page, _ = k_cache.shape
    out, wt, lse = np.zeros((S, H, d)), np.zeros((S, H, d)), np.full((S, H), -np.inf)
    for s in range(S):
        n = min(max(int(lengths[s]), 0), table.shape[1] * page)
        at = [(int(table[s, i // page]), i % page) for i in range(n)]
        at = [(p, o) for p, o in at if 0 <= p < pages]
        if not at:
            continue
        p_, o_ = np.array([a[0] for a in at]), np.array([a[1] for a in at])
        for h in range(H):
            j = h // (H // KV)
            k, v = _f(k_cache[p_, j, o_]), _f(v_cache[p_, j, o_])
            sc = scale * (k @ q[s, h])
            top = sc.max()
            e = np.exp(sc - top)
            den = e.sum()
            out[s, h], wt[s, h], lse[s, h] = e @ v / den, e @ np.abs(v) / den, top + math.log(den)
    return out, lse, wt


def paged_plan(cached, new, free, table, page, tokens):
    """(table, total_lens, starts, slots, positions, pages_needed) by walking
    the tokens one at a time."""
    table = np.array(table, np.int64).copy()
    free = [int(p) for p in free]
    cols = table.shape[1]
    total, starts, slots, positions, used = [], [0], [], [], 0
    for s, (c, n) in enumerate(zip(cached, new)):
        c, n = max(int(c), 0), max(int(n), 0)
        have = -(-c // page)
        mine = {j: int(table[s, j]) for j in range(min(have, cols))}
        for j in range(have, min(-(-(c + n) // page), cols)):
            mine[j] = table[s, j] = free[used] if used < len(free) else -1
            used += 1
        for p in range(c, c + n):
            pg = mine.get(p // page, -1)
            slots.append(pg * page + p % page if pg >= 0 else -1)
            positions.append(p)
        total.append(c + n)
        starts.append(starts[-1] + n)
    slots, positions = slots[:tokens], positions[:tokens]
    pad = tokens - len(slots)
    return table, np.array(total, np.int64), np.array(starts), np.array(slots + [-1] * pad), \
        np.array(positions + [0] * pad), used


# --------------------------------------------------------------------- block

def _rope_torch(z, freq, mscale, interleaved):
    """z [batch, seq, heads, d] at positions 0 .. seq - 1."""
    r = 2 * len(freq)
    t = torch.arange(z.shape[1], dtype=torch.float64)[:, None, None] * torch.tensor(freq)
    c, s = mscale * torch.cos(t), mscale * torch.sin(t)
    p = z[..., :r]
    x, y = (p[..., 0::2], p[..., 1::2]) if interleaved else (p[..., :r // 2], p[..., r // 2:])
    x, y = x * c - y * s, x * s + y * c
    p = torch.stack((x, y), -1).flatten(-2) if interleaved else torch.cat((x, y), -1)
    return torch.cat((p, z[..., r:]), -1)


def block(x, W, A, B, s, heads, gains, rope=None, scale=1.0, dy=None):
    """The block of oracle/block.py with h = x + scale * gate1 * post1(L_o(..))
    and likewise after L_down.  gains: dict with g1, g2 and any of post1, post2,
    gate1, gate2; rope: (frequencies, factor, interleaved) or None.  Returns y,
    or with dy (y, dx, dA, dB, dgains) as numpy arrays."""
    t = lambda a, g=False: torch.tensor(_f(a), requires_grad=g)  # noqa: E731
    xt, gt = t(x, True), {n: t(v, True) for n, v in gains.items()}
    At, Bt, Wt = {n: t(v, True) for n, v in A.items()}, {n: t(v, True) for n, v in B.items()}, {n: t(W[n]) for n in W}

    def L(n, X):
        return oblock.qlora_linear(X, Wt[n], At[n], Bt[n], s)

    def step(x, u, i):
        if f"post{i}" in gt:
            u = oblock.rms_norm(u, gt[f"post{i}"])
        if f"gate{i}" in gt:
            u = u * gt[f"gate{i}"]
        return x + scale * u

    b, n, hid = xt.shape
    n1 = oblock.rms_norm(xt, gt["g1"])
    q, k = L("q", n1), L("k", n1)
    if rope is not None:
        q, k = (_rope_torch(z.view(b, n, heads, -1), *rope).reshape(b, n, hid) for z in (q, k))
    h = step(xt, L("o", oblock.causal_attention(q, k, L("v", n1), heads)), 1)
    n2 = oblock.rms_norm(h, gt["g2"])
    y = step(h, L("down", torch.nn.functional.silu(L("gate", n2)) * L("up", n2)), 2)
    if dy is None:
        return y.detach().numpy()
    (y * t(dy)).sum().backward()
    num = lambda d: {k: v.grad.numpy() for k, v in d.items()}  # noqa: E731
    return y.detach().numpy(), xt.grad.numpy(), num(At), num(Bt), num(gt)
