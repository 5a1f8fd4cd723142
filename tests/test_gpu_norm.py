"""GPU parity: the residual update with its norms, forward and backward,
against the fp64 oracle.

Tolerances.  The kernels compute in fp32 and round each output once, so an
output may be off by half a step of its type (2^-8 of the value for bfloat16,
2^-24 for float32) plus the fp32 error: u = 2^-24 per operation.  A row mean
is a tree of at most 8 NV + 16 + 10 additions per element chain (NV <= 2), so
C = 64 covers a mean, the square root, the reciprocal and the few products
behind it; E below carries C u times the sum of the magnitudes that enter.  A
sum over T tokens has chains of at most T + 64 additions."""

import sys

import numpy as np
import pytest
import torch

from oracle import decoder as od

pytestmark = pytest.mark.gpu

U, C = 2.0 ** -24, 64.0
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
EPS = 1e-6


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
    return None if t is None else t.detach().double().cpu().numpy()


def _close(got, ref, E, dtype, name):
    got = _n(got)
    tol = HALF[dtype] * (np.abs(ref) + E) + E
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (name, int(bad.sum()), float(np.abs(got - ref)[bad].max()))


def _inputs(T, W, xt, ht, post, gate, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, h = n(T, W).to(xt), (0.5 * n(T, W)).to(ht)
    return (x, h, 1 + 0.2 * n(W), (1 + 0.2 * n(W)) if post else None, n(W) if gate else None,
            n(T, W).to(xt), n(T, W).to(ht))


def _check_fwd(D, x, h, w_pre, w_post, gate, alpha, got):
    xo, n = got
    rx, rn = od.norm_residual(_n(x), _n(h), _n(w_pre), _n(w_post), _n(gate), alpha, EPS)
    ht = x.dtype if n is None else n.dtype
    E = C * U * (np.abs(_n(x)) + np.abs(rx - _n(x)))
    _close(xo, rx, E if h is not None else 0.0, x.dtype, "xo")
    if n is not None:
        En = (E + C * U * np.abs(rx)) / od.rms(rx, EPS) * np.abs(_n(w_pre))
        _close(n, rn, En, ht, "n")


def _check_bwd(got, dxo, dn, xo, h, w_pre, w_post, gate, alpha, gains=True):
    T, W = xo.shape
    ref = od.norm_residual_grads(_n(dxo), _n(dn), _n(xo), _n(h), _n(w_pre), _n(w_post), _n(gate), alpha, EPS)
    x = _n(xo)
    E = C * U * (np.abs(_n(dxo)) if dxo is not None else np.zeros_like(x))
    if dn is not None:
        r = 1 / od.rms(x, EPS)
        a = np.abs(_n(dn) * _n(w_pre))
        E = E + C * U * r * (a + np.abs(x) * r * r * (a * np.abs(x)).mean(-1, keepdims=True))
        if gains:
            S = (np.abs(_n(dn) * x) * r).sum(0)
            _close(got.dw_pre, ref["dw_pre"], (T + 64 + C) * U * S, torch.float32, "dw_pre")
    _close(got.dx, ref["dx"], E, xo.dtype, "dx")
    gt = np.ones(W) if gate is None else np.abs(_n(gate))
    wp = np.ones(W) if w_post is None else np.abs(_n(w_post))
    Eb = alpha * gt * (E + C * U * np.abs(ref["dx"]))
    b = alpha * gt * np.abs(ref["dx"])
    if got.dh is not None:
        Eh = Eb
        if w_post is not None:
            hh = _n(h)
            rh = 1 / od.rms(hh, EPS)
            y = np.abs(hh) * rh
            both = wp * (Eb + C * U * b)
            Eh = rh * (both + y * (both * y).mean(-1, keepdims=True) + C * U * y * (wp * b * y).mean(-1, keepdims=True))
        _close(got.dh, ref["dh"], Eh, got.dh.dtype, "dh")
    if gains and h is not None and (w_post is not None or gate is not None):
        y = np.abs(_n(h)) / (od.rms(_n(h), EPS) if w_post is not None else 1.0)
        raw = alpha * np.abs(ref["dx"])
        if w_post is not None:
            E1 = ((T + 64 + C) * U * b * y + Eb * y).sum(0)
            _close(got.dw_post, ref["dw_post"], E1, torch.float32, "dw_post")
        if gate is not None:
            E1 = ((T + 64 + C) * U * raw * y * wp + alpha * E * y * wp).sum(0)
            _close(got.dgate, ref["dgate"], E1, torch.float32, "dgate")


BF, F = torch.bfloat16, torch.float32
TYPES = [(BF, BF), (F, BF), (F, F)]
SIZES = [(1, 1), (3, 7), (5, 64), (9, 100), (70, 512), (33, 520), (4, 1000), (6, 1025), (5, 2048), (7, 2056), (3, 4096),
         (2, 4097), (3, 8192), (2, 8200), (2, 9001), (2, 16384)]


@pytest.mark.parametrize("xt,ht", TYPES)
@pytest.mark.parametrize("T,W", SIZES)
def test_forward_and_backward(D, T, W, xt, ht):
    for post, gate in ((False, False), (True, True), (True, False), (False, True)):
        _log(f"norm T={T} W={W} {xt} {ht} post={post} gate={gate}")
        x, h, w_pre, w_post, gt, dxo, dn = _inputs(T, W, xt, ht, post, gate, seed=T * 131 + W)
        xo, n = D.qlora_norm_residual_fwd(x, h, w_pre=w_pre, w_post=w_post, gate=gt, alpha=0.7, eps=EPS)
        assert xo.dtype == xt and n.dtype == ht
        _check_fwd(D, x, h, w_pre, w_post, gt, 0.7, (xo, n))
        got = D.qlora_norm_residual_bwd(dxo, dn, xo, h, w_pre=w_pre, w_post=w_post, gate=gt, alpha=0.7, eps=EPS,
                                        need_gains=True)
        assert (got.dw_post is None) == (not post) and (got.dgate is None) == (not gate)
        _check_bwd(got, dxo, dn, xo, h, w_pre, w_post, gt, 0.7)
        plain = D.qlora_norm_residual_bwd(dxo, dn, xo, h, w_pre=w_pre, w_post=w_post, gate=gt, alpha=0.7, eps=EPS)
        assert torch.equal(plain.dx, got.dx) and torch.equal(plain.dh, got.dh) and plain.dw_pre is None


def test_parts_left_out(D):
    _log("norm: parts left out")
    x, h, w_pre, w_post, gt, dxo, dn = _inputs(11, 768, F, BF, True, True, seed=5)
    xo, n = D.qlora_norm_residual_fwd(x, None, w_pre=w_pre, n_dtype=BF)
    assert xo is x and n.dtype == BF
    _check_fwd(D, x, None, w_pre, None, None, 1.0, (xo, n))
    xo, n = D.qlora_norm_residual_fwd(x, h, w_post=w_post)
    assert n is None
    _check_fwd(D, x, h, None, w_post, None, 1.0, (xo, None))
    got = D.qlora_norm_residual_bwd(None, dn, x, None, w_pre=w_pre, need_dh=False, need_gains=True)
    _check_bwd(got, None, dn, x, None, w_pre, None, None, 1.0)
    got = D.qlora_norm_residual_bwd(dxo, None, xo, h, w_post=w_post, gate=gt, alpha=0.3, need_gains=True)
    assert got.dw_pre is None
    _check_bwd(got, dxo, None, xo, h, None, w_post, gt, 0.3)
    got = D.qlora_norm_residual_bwd(dxo, dn, xo, None, w_pre=w_pre, alpha=0.3)
    _check_bwd(got, dxo, dn, xo, None, w_pre, None, None, 0.3, gains=False)


def test_in_place(D):
    _log("norm in place")
    for W in (200, 4096, 4099, 12290):
        x, h, w_pre, w_post, gt, dxo, dn = _inputs(9, W, BF, BF, True, True, seed=W)
        xo, n = D.qlora_norm_residual_fwd(x, h, w_pre=w_pre, w_post=w_post, gate=gt)
        x2 = x.clone()
        xo2, n2 = D.qlora_norm_residual_fwd(x2, h, w_pre=w_pre, w_post=w_post, gate=gt, xo=x2)
        assert xo2 is x2 and torch.equal(xo, x2) and torch.equal(n, n2)
        a = D.qlora_norm_residual_bwd(dxo, dn, xo, h, w_pre=w_pre, w_post=w_post, gate=gt)
        d2, n3 = dxo.clone(), dn.clone()
        b = D.qlora_norm_residual_bwd(d2, n3, xo, h, w_pre=w_pre, w_post=w_post, gate=gt, dx=d2, dh=n3)
        assert torch.equal(a.dx, d2) and torch.equal(a.dh, n3) and b.dx is d2


@pytest.mark.parametrize("T,W", [(3000, 256), (1111, 1024), (700, 4096), (600, 8192), (600, 16384), (270, 9001), (301, 1536)])
def test_many_tokens_sums(D, T, W):
    """More rows than workgroups keep sums for, and results that repeat."""
    _log(f"norm sums T={T} W={W}")
    x, h, w_pre, w_post, gt, dxo, dn = _inputs(T, W, F, BF, True, True, seed=T)
    xo, _ = D.qlora_norm_residual_fwd(x, h, w_pre=w_pre, w_post=w_post, gate=gt)
    kw = dict(w_pre=w_pre, w_post=w_post, gate=gt, need_gains=True)
    a = D.qlora_norm_residual_bwd(dxo, dn, xo, h, **kw)
    _check_bwd(a, dxo, dn, xo, h, w_pre, w_post, gt, 1.0)
    b = D.qlora_norm_residual_bwd(dxo, dn, xo, h, **kw)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_no_tokens(D):
    _log("norm no tokens")
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    w = torch.ones(64, device="cuda")
    xo, n = D.qlora_norm_residual_fwd(x, x, w_pre=w, w_post=w)
    assert xo.shape == n.shape == (0, 64)
    g = D.qlora_norm_residual_bwd(x, x, x, x, w_pre=w, w_post=w, gate=w, need_gains=True)
    assert all(torch.equal(t, torch.zeros(64, device="cuda")) for t in (g.dw_pre, g.dw_post, g.dgate))


def test_zero_rows_and_large_values(D):
    """A zero row has rms sqrt(eps) and stays zero; squares beyond fp32's small
    end vanish against eps; a row with an infinity or a NaN spoils no other."""
    _log("norm zero rows")
    x, h, w_pre, w_post, gt, dxo, dn = _inputs(6, 1024, F, F, True, True, seed=3)
    x[1] = 0
    h[1] = 0
    x[2] = 1e-30
    h[2] = 1e-30
    x[3, 7] = float("nan")
    h[4, 9] = float("inf")
    xo, n = D.qlora_norm_residual_fwd(x, h, w_pre=w_pre, w_post=w_post, gate=gt)
    assert not xo[1].any() and not n[1].any()
    assert torch.isnan(n[3]).all() and torch.isnan(n[4]).all()
    ok = [0, 1, 2, 5]
    _check_fwd(D, x[ok], h[ok], w_pre, w_post, gt, 1.0, (xo[ok], n[ok]))
    g = D.qlora_norm_residual_bwd(dxo, dn, xo, h, w_pre=w_pre, w_post=w_post, gate=gt)
    sub = type(g)(g.dx[ok], g.dh[ok], None, None, None)
    _check_bwd(sub, dxo[ok], dn[ok], xo[ok], h[ok], w_pre, w_post, gt, 1.0, gains=False)


def test_other_stream_and_graph(D):
    """On a stream of its own, and captured: every replay, with eager work
    between, equals the eager result."""
    _log("norm stream and graph")
    x, h, w_pre, w_post, gt, dxo, dn = _inputs(300, 2048, F, BF, True, True, seed=9)
    kw = dict(w_pre=w_pre, w_post=w_post, gate=gt)

    def both(stream=None):
        xo, n = D.qlora_norm_residual_fwd(x, h, stream=stream, **kw)
        return (xo, n) + tuple(D.qlora_norm_residual_bwd(dxo, dn, xo, h, need_gains=True, stream=stream, **kw))

    ref = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = both()
    for k in range(4):
        x.mul_(1.0 + 0.25 * k)
        dn.mul_(-1.0)
        ref = both()
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, out)), k


def test_offsets_beyond_32_bits(D):
    """More than 2^32 elements: the last rows equal a call on them alone."""
    _log("norm 64-bit offsets")
    T, W = 2 ** 19 + 5, 8192
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(T, W, dtype=BF, device="cuda")
    h, dxo = torch.zeros_like(x), torch.zeros_like(x)
    for t in (x, h, dxo):
        t[-5:] = torch.randn(5, W, generator=g, device="cuda").to(BF)
    w = 1 + 0.1 * torch.randn(W, generator=g, device="cuda")
    kw = dict(w_pre=w, w_post=w, alpha=0.5)
    xo, n = D.qlora_norm_residual_fwd(x, h, **kw)
    ref = D.qlora_norm_residual_fwd(x[-5:].clone(), h[-5:].clone(), **kw)
    assert torch.equal(xo[-5:], ref[0]) and torch.equal(n[-5:], ref[1]) and not xo[:-5].any()
    last = [t[-5:].clone() for t in (dxo, h, xo)]
    got = D.qlora_norm_residual_bwd(dxo, h, xo, h, dx=dxo, **kw)   # in place
    ref = D.qlora_norm_residual_bwd(last[0], last[1], last[2], last[1], **kw)
    assert torch.equal(got.dx[-5:], ref.dx) and torch.equal(got.dh[-5:], ref.dh)
    assert not got.dx[:-5].any() and not got.dh[:-5].any()


def test_views_that_start_off_a_16_byte_boundary_are_refused(D):
    from bit_nf4_quantized_quantize_amd import binding
    x = torch.zeros(9 * 64, dtype=BF, device="cuda")[1:1 + 8 * 64].view(8, 64)
    w = torch.ones(64, device="cuda")
    with pytest.raises(binding.QLoraError) as e:
        D.qlora_norm_residual_fwd(x, None, w_pre=w)
    assert e.value.status == binding.QLORA_ERR_MISALIGNED


def test_leading_dimensions_and_extremes_of_the_scalars(D):
    _log("norm shapes and scalars")
    x, h, w_pre, w_post, gt, dxo, dn = _inputs(12, 96, F, BF, True, True, seed=21)
    kw = dict(w_pre=w_pre, w_post=w_post, gate=gt)
    ref = D.qlora_norm_residual_fwd(x, h, **kw)
    got = D.qlora_norm_residual_fwd(x.view(2, 3, 2, 96), h.view(2, 3, 2, 96), **kw)
    assert got[0].shape == (2, 3, 2, 96) and torch.equal(got[0].view(12, 96), ref[0])
    one = D.qlora_norm_residual_fwd(x[3], h[3], **kw)
    assert one[0].shape == (96,) and torch.equal(one[1], ref[1][3])
    assert torch.equal(D.qlora_norm_residual_fwd(x, h, alpha=0.0, **kw)[0], x)
    xo, n = D.qlora_norm_residual_fwd(x, h, eps=0.0, alpha=-2.0, **kw)
    rx, rn = od.norm_residual(_n(x), _n(h), _n(w_pre), _n(w_post), _n(gt), -2.0, 0.0)
    E = C * U * (np.abs(_n(x)) + np.abs(rx - _n(x)))
    _close(xo, rx, E, F, "xo")
    _close(n, rn, (E + C * U * np.abs(rx)) / od.rms(rx, 0.0) * np.abs(_n(w_pre)), BF, "n")
