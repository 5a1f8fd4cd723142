"""Pins of the decoder-block oracle (CPU): gradients against finite
differences, rotary properties and special cases, paged attention against
torch's attention in fp64, the plan's invariants."""

import math

import numpy as np
import pytest
import torch

from oracle import decoder as od


def _rand(rng, *shape):
    return rng.standard_normal(shape)


@pytest.mark.parametrize("post,gate", [(False, False), (True, False), (False, True), (True, True)])
def test_norm_gradients_match_differences(post, gate):
    rng = np.random.default_rng(1)
    T, D, alpha = 3, 7, 0.7
    x, h = _rand(rng, T, D), _rand(rng, T, D)
    w_pre, w_post = 1 + 0.3 * _rand(rng, D), (1 + 0.3 * _rand(rng, D)) if post else None
    g = _rand(rng, D) if gate else None
    dxo, dn = _rand(rng, T, D), _rand(rng, T, D)

    def loss(x, h, w_pre, w_post, g):
        xo, n = od.norm_residual(x, h, w_pre, w_post, g, alpha)
        return float((dxo * xo).sum() + (dn * n).sum())

    xo, _ = od.norm_residual(x, h, w_pre, w_post, g, alpha)
    got = od.norm_residual_grads(dxo, dn, xo, h, w_pre, w_post, g, alpha)
    args = [x, h, w_pre, w_post, g]
    for i, name in enumerate(("dx", "dh", "dw_pre", "dw_post", "dgate")):
        if args[i] is None:
            continue
        num = np.zeros_like(args[i])
        for at in np.ndindex(args[i].shape):
            lo, hi = [a if a is None else a.copy() for a in args], [a if a is None else a.copy() for a in args]
            lo[i][at] -= 1e-5
            hi[i][at] += 1e-5
            num[at] = (loss(*hi) - loss(*lo)) / 2e-5
        assert np.allclose(got[name], num, rtol=1e-6, atol=1e-7), name


def test_norm_special_cases():
    rng = np.random.default_rng(2)
    x, h, w = _rand(rng, 4, 16), _rand(rng, 4, 16), np.ones(16)
    assert np.array_equal(od.norm_residual(x, None, w)[0], x)
    assert np.allclose(od.norm_residual(x, h, w)[0], x + h)
    n = od.norm_residual(x, None, w, eps=0.0)[1]
    assert np.allclose((n * n).mean(-1), 1.0)
    # a norm behind the branch makes the step blind to the branch's size
    a, b = (od.norm_residual(x, c * h, w, w_post=w, eps=0.0)[0] for c in (1.0, 1000.0))
    assert np.allclose(a, b)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_properties(interleaved):
    rng = np.random.default_rng(3)
    T, d, r = 6, 16, 12
    f, m = od.rope_frequencies(r)
    assert m == 1.0 and f[0] == 1.0
    q, k = _rand(rng, T, 2, d), _rand(rng, T, 2, d)
    pos = np.array([0, 1, 5, 17, -3, 100000])
    rq = od.rope(q, pos, f, interleaved=interleaved)
    assert np.array_equal(rq[0], q[0]) and np.array_equal(rq[..., r:], q[..., r:])
    assert np.allclose(np.linalg.norm(rq, axis=-1), np.linalg.norm(q, axis=-1))
    assert np.allclose(od.rope(rq, pos, f, interleaved=interleaved, inverse=True), q)
    # products depend on the distance alone
    for shift in (7, 1000):
        a = (od.rope(q, pos, f, interleaved=interleaved) * od.rope(k, pos + 4, f, interleaved=interleaved)).sum(-1)
        b = (od.rope(q, pos + shift, f, interleaved=interleaved)
             * od.rope(k, pos + 4 + shift, f, interleaved=interleaved)).sum(-1)
        assert np.allclose(a, b, atol=1e-8)
    # the first pair turns by one radian per position
    e = np.zeros((1, 1, d))
    e[0, 0, 0] = 1.0
    out = od.rope(e, np.array([2]), f, interleaved=interleaved)[0, 0]
    assert np.isclose(out[0], math.cos(2)) and np.isclose(out[1 if interleaved else r // 2], math.sin(2))


def test_rope_scalings():
    f, _ = od.rope_frequencies(64)
    lin, _ = od.rope_frequencies(64, scaling="linear", factor=4.0)
    ntk, _ = od.rope_frequencies(64, scaling="ntk", factor=4.0)
    yarn, m = od.rope_frequencies(64, scaling="yarn", factor=4.0, original_len=4096)
    assert np.allclose(lin, f / 4)
    assert ntk[0] == f[0] and np.isclose(ntk[-1], f[-1] / 4)   # fastest kept, slowest interpolated
    assert np.isclose(yarn[0], f[0]) and np.isclose(yarn[-1], f[-1] / 4) and np.isclose(m, 0.1 * math.log(4) + 1)
    assert np.all(np.diff(yarn) < 0)


def test_paged_attention_matches_torch():
    rng = np.random.default_rng(4)
    S, H, KV, d, page, cols = 3, 4, 2, 8, 4, 3
    pages = S * cols
    kc, vc = _rand(rng, pages, KV, page, d), _rand(rng, pages, KV, page, d)
    q = _rand(rng, S, H, d)
    table = rng.permutation(pages).reshape(S, cols)
    lengths = [0, 5, 12]
    out, lse, wt = od.paged_attention(q, kc, vc, table, lengths, 0.3)
    assert np.all(out[0] == 0) and np.all(lse[0] == -np.inf)
    for s in (1, 2):
        n = lengths[s]
        k = torch.tensor(kc[table[s]].transpose(1, 0, 2, 3).reshape(KV, -1, d)[:, :n]).repeat_interleave(2, 0)
        v = torch.tensor(vc[table[s]].transpose(1, 0, 2, 3).reshape(KV, -1, d)[:, :n]).repeat_interleave(2, 0)
        ref = torch.nn.functional.scaled_dot_product_attention(torch.tensor(q[s])[:, None], k, v, scale=0.3)[:, 0]
        assert np.allclose(out[s], ref.numpy())
        sc = 0.3 * (k @ torch.tensor(q[s])[:, :, None])[..., 0]
        assert np.allclose(lse[s], torch.logsumexp(sc, -1).numpy())
    table[2, 1] = -1   # the tokens of a missing page take no part
    out2, _, _ = od.paged_attention(q, kc, vc, table, lengths, 0.3)
    assert not np.allclose(out2[2], out[2]) and np.allclose(out2[1], out[1])


def test_paged_plan_invariants():
    rng = np.random.default_rng(5)
    S, page, cols = 9, 4, 6
    cached, new = rng.integers(0, 12, S), rng.integers(0, 9, S)
    pages = S * cols
    ids = rng.permutation(pages)
    table = np.full((S, cols), -1)
    used = 0
    for s in range(S):
        n = -(-cached[s] // page)
        table[s, :n] = ids[used:used + n]
        used += n
    t2, total, starts, slots, pos, need = od.paged_plan(cached, new, ids[used:], table, page, int(new.sum()) + 5)
    assert need == sum(-(-(c + n) // page) + c // -page for c, n in zip(cached, new))
    real = slots[:starts[-1]]
    assert len(set(real.tolist())) == len(real) and (real >= 0).all()
    assert (slots[starts[-1]:] == -1).all()
    held = {int(table[s, i // page]) * page + i % page for s in range(S) for i in range(cached[s])}
    assert not held & set(real.tolist())
    for s in range(S):
        for r in range(starts[s], starts[s + 1]):
            assert pos[r] == cached[s] + r - starts[s]
            assert slots[r] == t2[s, pos[r] // page] * page + pos[r] % page
    _, _, _, slots, _, need = od.paged_plan([0], [10], [7], [[-1] * 3], 4, 10)   # the free list runs out
    assert need == 3 and slots.tolist() == [28, 29, 30, 31] + [-1] * 6
    _, _, _, slots, _, need = od.paged_plan([0], [10], [7, 1, 2], [[-1]], 4, 10)  # the table does
    assert need == 1 and slots.tolist() == [28, 29, 30, 31] + [-1] * 6


def test_block_reduces_to_the_plain_block():
    """Without the additions it is oracle/block.py's; gates of one, a scale of
    one and a turn of nothing change nothing; with them, finite differences."""
    from oracle import block as oblock
    rng = np.random.default_rng(6)
    hid, mlp, heads, r, b, n = 16, 24, 2, 3, 2, 5
    sh = oblock.shapes(hid, mlp)
    W = {k: 0.3 * _rand(rng, *v) for k, v in sh.items()}
    A = {k: 0.3 * _rand(rng, v[1], r) for k, v in sh.items()}
    B = {k: 0.3 * _rand(rng, r, v[0]) for k, v in sh.items()}
    g = {"g1": 1 + 0.1 * _rand(rng, hid), "g2": 1 + 0.1 * _rand(rng, hid)}
    x, dy = _rand(rng, b, n, hid), _rand(rng, b, n, hid)
    y0, dx0, dA0, dB0 = oblock.forward_backward(x, W, A, B, g["g1"], g["g2"], 0.5, heads, dy)
    y, dx, dA, dB, _ = od.block(x, W, A, B, 0.5, heads, g, dy=dy)
    assert np.allclose(y, y0) and np.allclose(dx, dx0) and all(np.allclose(dA[k], dA0[k]) for k in dA)
    one = np.ones(hid)
    assert np.allclose(od.block(x, W, A, B, 0.5, heads, dict(g, gate1=one, gate2=one),
                                rope=(np.zeros(4), 1.0, False)), y0)
    full = dict(g, post1=1 + 0.1 * _rand(rng, hid), post2=1 + 0.1 * _rand(rng, hid), gate1=_rand(rng, hid),
                gate2=_rand(rng, hid))
    f = od.rope_frequencies(8)[0]
    for inter in (False, True):
        args = dict(rope=(f, 1.1, inter), scale=0.7)
        y, dx, _, dB, dg = od.block(x, W, A, B, 0.5, heads, full, dy=dy, **args)
        v = _rand(rng, b, n, hid)
        hi, lo = (od.block(x + e * v, W, A, B, 0.5, heads, full, **args) for e in (1e-5, -1e-5))
        assert np.isclose(((hi - lo) * dy).sum() / 2e-5, (dx * v).sum(), rtol=1e-5)
        for name in full:
            v = _rand(rng, hid)
            hi, lo = (od.block(x, W, A, B, 0.5, heads, dict(full, **{name: full[name] + e * v}), **args)
                      for e in (1e-5, -1e-5))
            assert np.isclose(((hi - lo) * dy).sum() / 2e-5, (dg[name] * v).sum(), rtol=1e-5), name
        # the rotation used here is the other one's
        z = _rand(rng, 1, n, 2, 12)
        assert np.allclose(od._rope_torch(torch.tensor(z), f, 1.1, inter).numpy()[0],
                           od.rope(z[0], np.arange(n), f, 1.1, inter))
