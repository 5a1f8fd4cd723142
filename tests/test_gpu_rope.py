"""GPU parity: rotary positions, and their form that writes the paged cache,
against the fp64 oracle.

Tolerance: the cosine and sine are within 4 u (u = 2^-24: the reduced angle is
exact to about u / 8 of a turn's radian, the functions to 2 ulp, one rounding of
the factor), the rotation is three fp32 operations, and the result is rounded
once: |err| <= 8 u m (|a| + |b|) + half a step of the value (2^-8 bfloat16,
2^-24 float32)."""

import sys

import numpy as np
import pytest
import torch

from oracle import decoder as od

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F = torch.bfloat16, torch.float32


def _log(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def D():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_quantize_amd import decoder
    decoder.lib()
    return decoder


def _n(t):
    return t.detach().double().cpu().numpy()


def _pair_size(z, rot, inter):
    """|a| + |b| of the pair each element belongs to (0 outside the pairs)."""
    z, out = np.abs(z), np.zeros_like(z)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    out[..., a] = out[..., b] = z[..., a] + z[..., b]
    return out


def _check(got, z, pos, f, m, inter, inverse, name):
    zn = _n(z)
    ref = od.rope(zn, pos.cpu().numpy(), f, m, inter, inverse)
    E = 8 * U * m * _pair_size(zn, 2 * len(f), inter)
    bad = ~(np.abs(_n(got) - ref) <= E + HALF[got.dtype] * (np.abs(ref) + E))
    assert not bad.any(), (name, int(bad.sum()), float(np.abs(_n(got) - ref)[bad].max()))
    r = 2 * len(f)
    assert torch.equal(got[..., r:], z[..., r:])


def _randn(g, *s, dtype=F):
    return torch.randn(*s, generator=g, device="cuda").to(dtype)


CASES = [  # T, q heads, kv heads, head_dim, rot_dim
    (1, 1, 1, 2, 2), (1, 32, 32, 128, 128), (3, 4, 2, 64, 64), (5, 7, 1, 80, 40), (17, 8, 8, 96, 96),
    (9, 3, 0, 128, 64), (9, 0, 3, 128, 32), (4, 2, 2, 256, 256), (33, 5, 5, 50, 22), (1031, 4, 1, 128, 128),
    (1025, 2, 2, 20, 12), (6, 64, 8, 128, 128), (2, 1, 1, 1024, 1024), (5, 3, 3, 33, 10)]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,KV,d,rot", CASES)
def test_rope(D, T, H, KV, d, rot, inter, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + d)
    pos = torch.randint(-50, 300000, (T,), generator=g, device="cuda").to(torch.int32)
    pos[0] = 2 ** 31 - 1 if T > 1 else 0
    for scaling, factor in (("none", 1.0), ("linear", 3.0), ("ntk", 8.0), ("yarn", 16.0)):
        if scaling == "ntk" and rot < 4:
            continue
        _log(f"rope T={T} H={H} KV={KV} d={d} rot={rot} inter={inter} {dtype} {scaling}")
        kw = dict(base=10000.0, scaling=scaling, factor=factor, original_len=4096)
        tab = D.RopeTable(rot, interleaved=inter, device="cuda", **kw)
        f, m = od.rope_frequencies(rot, **kw)
        # the angle of the farthest position, from the table the call was given
        f = tab.turns.cpu().numpy() * 2 * np.pi if T > 1 else f
        q = _randn(g, T, H, d, dtype=dtype) if H else None
        k = _randn(g, T, KV, d, dtype=dtype) if KV else None
        for inverse in (False, True):
            qo, ko = D.qlora_rope(q, k, tab, pos, inverse=inverse)
            for z, o, name in ((q, qo, "q"), (k, ko, "k")):
                if z is not None:
                    p = pos if T == 1 else pos.clone()
                    if T > 1:   # 2^31 - 1 radians times 2 pi rounding in the oracle's own product: checked apart
                        _check(o[1:], z[1:], p[1:], f, m, inter, inverse, name)
                    else:
                        _check(o, z, p, f, m, inter, inverse, name)


def test_frequencies_match_oracle(D):
    for rot in (2, 22, 64, 128):
        for scaling, factor in (("none", 1.0), ("linear", 3.0), ("ntk", 8.0), ("yarn", 16.0), ("yarn", 1.0)):
            if scaling == "ntk" and rot < 4:
                continue
            kw = dict(base=500000.0, scaling=scaling, factor=factor, original_len=8192)
            t, m = D.qlora_rope_frequencies(rot, **kw)
            f, mr = od.rope_frequencies(rot, **kw)
            assert np.allclose(np.array(t) * 2 * np.pi, f, rtol=1e-14, atol=0)
            assert abs(m - mr) <= 2.0 ** -24 * mr


def test_far_positions_exact_angle(D):
    """Positions up to 2^31 - 1: turns of exact binary fractions, whose angle is
    known without rounding."""
    _log("rope far positions")
    tab = D.RopeTable(4, device="cuda")
    tab.turns.copy_(torch.tensor([0.125, 2.0 ** -33], dtype=torch.float64))
    pos = torch.tensor([2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31, 5], dtype=torch.int32, device="cuda")
    q = torch.ones(4, 1, 4, device="cuda")
    q[..., 2:] = 0
    out, _ = D.qlora_rope(q, None, tab, pos)
    for i, p in enumerate(pos.tolist()):
        for j, t in enumerate(((p % 8) / 8, p * 2.0 ** -33)):
            got = out[i, 0, [j, 2 + j]].double().cpu().numpy()
            assert np.allclose(got, [np.cos(2 * np.pi * t), np.sin(2 * np.pi * t)], rtol=0, atol=8 * U), (p, j)


def test_strided_and_in_place(D):
    """q, k and v as slices of one projection; outputs strided; in place."""
    _log("rope strided")
    g = torch.Generator(device="cuda").manual_seed(1)
    for T, H, KV, d, dtype in ((13, 4, 2, 64, BF), (13, 4, 2, 64, F), (7, 3, 1, 18, BF), (1500, 2, 1, 128, BF)):
        tab = D.RopeTable(d // 2 // 2 * 2, device="cuda")
        pos = torch.arange(T, device="cuda", dtype=torch.int32)
        for pad in (0, 8, 3):
            full = _randn(g, T, (H + 2 * KV) * d + pad, dtype=dtype)
            q = full[:, :H * d].view(T, H, d)
            k = full[:, H * d:(H + KV) * d].view(T, KV, d)
            if k.data_ptr() % 16 or q.data_ptr() % 16:
                k = k.clone()
            ref = D.qlora_rope(q.clone(), k.clone(), tab, pos)
            buf = torch.zeros(T, (H + KV) * d + pad, dtype=dtype, device="cuda")
            qo = buf[:, :H * d].view(T, H, d)
            got = D.qlora_rope(q, k, tab, pos, q_out=qo)
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
            assert not buf[:, H * d:].any()
            rest = full[:, (H + KV) * d:].clone()
            D.qlora_rope(q, k, tab, pos, q_out=q, k_out=k)
            assert torch.equal(q, ref[0]) and torch.equal(k, ref[1])
            assert torch.equal(full[:, (H + KV) * d:], rest)


def test_gradient_against_differences(D):
    """<dy, R x> has the gradient R^T dy: the inverse call, times mscale."""
    _log("rope gradient")
    g = torch.Generator(device="cuda").manual_seed(2)
    tab = D.RopeTable(16, scaling="yarn", factor=4.0, original_len=64, device="cuda")
    pos = torch.randint(0, 1000, (3,), generator=g, device="cuda").to(torch.int32)
    x, dy = _randn(g, 3, 2, 24), _randn(g, 3, 2, 24)
    grad, _ = D.qlora_rope(dy, None, tab, pos, inverse=True)
    for at in [(0, 0, 0), (1, 1, 9), (2, 0, 15), (2, 1, 20)]:
        step = torch.zeros_like(x)
        step[at] = 1.0   # the map is linear: a step of one has no truncation error
        hi, _ = D.qlora_rope(x + step, None, tab, pos)
        lo, _ = D.qlora_rope(x - step, None, tab, pos)
        num = float(((hi.double() - lo.double()) * dy.double()).sum()) / 2
        # every one of the 144 products carries a few u of (|x| + 1) m |dy| < 2^6
        assert abs(num - float(grad[at])) < 144 * 16 * U * 64


WRITES = [  # T, q heads, kv heads, head_dim, rot_dim, page, pages
    (1, 32, 32, 128, 128, 16, 4), (16, 64, 8, 128, 128, 16, 40), (5, 0, 2, 64, 64, 1, 9), (7, 6, 3, 80, 40, 32, 3),
    (1100, 4, 2, 128, 0, 64, 30), (9, 2, 1, 34, 16, 8, 5), (40, 8, 4, 96, 96, 128, 2)]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,KV,d,rot,page,pages", WRITES)
def test_cache_write(D, T, H, KV, d, rot, page, pages, inter):
    _log(f"cache write T={T} H={H} KV={KV} d={d} rot={rot} page={page} inter={inter}")
    g = torch.Generator(device="cuda").manual_seed(T * d)
    tab = D.RopeTable(rot, interleaved=inter, device="cuda") if rot else None
    f = od.rope_frequencies(rot)[0] if rot else np.zeros(0)
    q = _randn(g, T, H, d, dtype=BF) if H else None
    k, v = _randn(g, T, KV, d, dtype=BF), _randn(g, T, KV, d, dtype=BF)
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda").to(torch.int32)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    T0 = slots.numel()
    slots = torch.cat([slots, torch.full((T - T0,), -1, dtype=torch.int32, device="cuda")])
    if T > 4:   # rows without a slot: padding, and slots that the cache does not have
        slots[1], slots[3], slots[4] = -1, pages * page, -2 ** 31
    kc, vc = _randn(g, pages, KV, page, d, dtype=BF), _randn(g, pages, KV, page, d, dtype=BF)
    k0, v0 = kc.clone(), vc.clone()
    qo = D.qlora_rope_cache_write(q, k, v, tab, pos if rot else None, slots, kc, vc)
    if H:
        _check(qo, q, pos, f, 1.0, inter, False, "q")
    sl = slots.cpu().tolist()
    flat_k, flat_v = kc.transpose(1, 2).reshape(-1, KV, d), vc.transpose(1, 2).reshape(-1, KV, d)
    real = [t for t in range(T) if 0 <= sl[t] < pages * page]
    at = torch.tensor([sl[t] for t in real], device="cuda")
    tt = torch.tensor(real, device="cuda")
    _check(flat_k[at], k[tt], pos[tt], f, 1.0, inter, False, "k")
    assert torch.equal(flat_v[at], v[tt])
    keep = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    keep[at] = False
    assert torch.equal(flat_k[keep], k0.transpose(1, 2).reshape(-1, KV, d)[keep])
    assert torch.equal(flat_v[keep], v0.transpose(1, 2).reshape(-1, KV, d)[keep])


def test_no_tokens(D):
    tab = D.RopeTable(8, device="cuda")
    e = torch.empty(0, 2, 8, dtype=BF, device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    q, k = D.qlora_rope(e, e, tab, i)
    assert q.shape == k.shape == (0, 2, 8)
    kc = torch.ones(2, 2, 16, 8, dtype=BF, device="cuda")
    assert D.qlora_rope_cache_write(e, e, e, tab, i, i, kc, kc.clone()).shape == (0, 2, 8)


def test_other_stream_and_graph(D):
    _log("rope stream and graph")
    g = torch.Generator(device="cuda").manual_seed(4)
    T, H, KV, d, page, pages = 50, 8, 2, 64, 16, 8
    tab = D.RopeTable(d, device="cuda")
    q, k, v = _randn(g, T, H, d, dtype=BF), _randn(g, T, KV, d, dtype=BF), _randn(g, T, KV, d, dtype=BF)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    kc, vc = torch.zeros(pages, KV, page, d, dtype=BF, device="cuda"), torch.zeros(pages, KV, page, d, dtype=BF, device="cuda")

    def both(stream=None):
        a = D.qlora_rope(q, k, tab, pos, stream=stream)
        return a + (D.qlora_rope_cache_write(q, k, v, tab, pos, slots, kc, vc, stream=stream),)

    ref = both() + (kc.clone(), vc.clone())
    kc.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got + (kc, vc)))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = both()
    for n in range(4):
        pos.add_(n * 17)
        q.mul_(-1)
        kc.zero_()
        ref = both() + (kc.clone(), vc.clone())
        kc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, out + (kc, vc))), n


def test_offsets_beyond_32_bits(D):
    """More than 2^32 elements of q: the last tokens equal a call on them alone."""
    _log("rope 64-bit offsets")
    T, H, d = 2 ** 19 + 3, 64, 128
    q = torch.zeros(T, H, d, dtype=BF, device="cuda")
    q[-3:] = torch.randn(3, H, d, device="cuda").to(BF)
    tab = D.RopeTable(d, device="cuda")
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    ref, _ = D.qlora_rope(q[-3:].clone(), None, tab, pos[-3:].clone())
    out, _ = D.qlora_rope(q, None, tab, pos, q_out=q)
    assert torch.equal(out[-3:], ref) and not out[:-3].any()


def test_cache_write_from_slices_and_in_place(D):
    """q, k and v as slices of one projection, q rotated where it lies."""
    _log("cache write from slices")
    g = torch.Generator(device="cuda").manual_seed(8)
    T, H, KV, d, page, pages = 21, 6, 2, 64, 16, 4
    tab = D.RopeTable(48, device="cuda")
    pos = torch.arange(T, device="cuda", dtype=torch.int32) + 5
    slots = torch.randperm(page * pages, generator=g, device="cuda")[:T].to(torch.int32)
    full = _randn(g, T, (H + 2 * KV) * d, dtype=BF)
    q, k, v = (full[:, a * d:b * d].view(T, b - a, d) for a, b in ((0, H), (H, H + KV), (H + KV, H + 2 * KV)))
    c = [torch.zeros(pages, KV, page, d, dtype=BF, device="cuda") for _ in range(4)]
    ref = D.qlora_rope_cache_write(q.clone(), k.clone(), v.clone(), tab, pos, slots, c[0], c[1])
    got = D.qlora_rope_cache_write(q, k, v, tab, pos, slots, c[2], c[3], q_out=q)
    assert got is q and torch.equal(q, ref) and torch.equal(c[0], c[2]) and torch.equal(c[1], c[3])
