"""GPU parity: the decoder block on the fused glue (norms, residual, rotary
positions) against the fp64 oracle block, its gradients, checkpointing, and
decoding token by token from the paged cache against the whole sequence at
once.

Tolerances are those of the plain block's test (2e-2 rel-L2 for the output and
dx, 3e-2 for parameter gradients): a path crosses at most four linears and here
the attention's and the branches' values are rounded to bfloat16 as well,
2^-8 each at most, seven roundings on the longest path."""

import sys

import numpy as np
import pytest
import torch

from oracle import blockwise
from oracle import decoder as od

pytestmark = pytest.mark.gpu


def _log(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def BL():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_quantize_amd import binding, block
    binding.lib()
    return block


def _rel(a, b):
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    return float(np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-30))


def _setup(BL, hidden, mlp, heads, r, batch, seq, seed, rot=None, inter=False, extras=True):
    from bit_nf4_quantized_quantize_amd import RopeTable
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    shapes = BL.linear_shapes(hidden, mlp)
    W = {n: rn(*sh) * 0.02 for n, sh in shapes.items()}
    A = {n: (rn(shapes[n][1], r) * 0.05).to(torch.bfloat16) for n in BL.LINEARS}
    Bm = {n: (rn(r, shapes[n][0]) * 0.05).to(torch.bfloat16) for n in BL.LINEARS}
    gains = {"g1": 1 + 0.1 * rn(hidden), "g2": 1 + 0.1 * rn(hidden)}
    if extras:
        gains.update(post1=1 + 0.1 * rn(hidden), post2=1 + 0.1 * rn(hidden), gate1=1 + 0.3 * rn(hidden),
                     gate2=1 + 0.3 * rn(hidden))
    x, dy = rn(batch, seq, hidden), rn(batch, seq, hidden)
    s = 16.0 / r
    scale = 0.5 if extras else 1.0
    dev = {n: v.cuda().requires_grad_(True) for n, v in gains.items()}
    tab = RopeTable(rot, interleaved=inter, scaling="yarn", factor=2.0, original_len=16, device="cuda") if rot else None
    c = lambda d: {n: v.cuda() for n, v in d.items()}  # noqa: E731
    blk = BL.QLoraBlock(c(W), c(A), c(Bm), dev["g1"], dev["g2"], s, heads, rope=tab, residual_scale=scale, fused=True,
                        **{n: v for n, v in dev.items() if n not in ("g1", "g2")})
    Wo = {n: blockwise.bf16_round(blockwise.quantize(W[n].numpy(), True).dequantize()).astype(np.float64) for n in W}
    f = od.rope_frequencies(rot, scaling="yarn", factor=2.0, original_len=16) if rot else None
    f64 = lambda d: {n: v.double().numpy() for n, v in d.items()}  # noqa: E731

    def ref(x, dy=None):
        return od.block(x, Wo, f64(A), f64(Bm), s, heads, f64(gains), (*f, inter) if f else None, scale, dy)

    return blk, dev, x, dy, ref


def _run(blk, dev, x, dy, checkpoint=False):
    for p in list(blk.parameters()) + list(dev.values()):
        p.grad = None
    xg = x.cuda().requires_grad_(True)
    y = blk(xg, checkpoint=checkpoint)
    y.backward(dy.cuda())
    torch.cuda.synchronize()
    n = lambda t: t.detach().float().cpu().numpy()  # noqa: E731
    return (n(y), n(xg.grad), {k: n(v.A.grad) for k, v in blk.lin.items()},
            {k: n(v.B.grad) for k, v in blk.lin.items()}, {k: n(v.grad) for k, v in dev.items()})


@pytest.mark.parametrize("hidden,mlp,heads,r,batch,seq,rot,inter,extras", [
    (256, 512, 4, 16, 2, 32, 64, False, True), (128, 320, 2, 64, 1, 48, 32, True, True),
    (256, 512, 4, 16, 2, 32, None, False, False), (128, 256, 8, 8, 3, 17, 16, False, False)])
def test_fused_block_matches_oracle(BL, hidden, mlp, heads, r, batch, seq, rot, inter, extras):
    _log(f"fused block hidden={hidden} seq={seq} rot={rot} extras={extras}")
    blk, dev, x, dy, ref = _setup(BL, hidden, mlp, heads, r, batch, seq, hidden + seq, rot, inter, extras)
    got, want = _run(blk, dev, x, dy), ref(x.numpy(), dy.numpy())
    assert _rel(got[0], want[0]) < 2e-2 and _rel(got[1], want[1]) < 2e-2
    for i in (2, 3, 4):
        for n in want[i]:
            assert _rel(got[i][n], want[i][n]) < 3e-2, (i, n)
    again = _run(blk, dev, x, dy, checkpoint=True)
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1])
    for i in (2, 3, 4):
        assert all(np.array_equal(got[i][n], again[i][n]) for n in got[i])


def test_frozen_gains_get_no_gradient(BL):
    _log("fused block frozen gains")
    blk, dev, x, dy, _ = _setup(BL, 128, 256, 2, 8, 1, 9, 5, 32)
    ref = _run(blk, dev, x, dy)
    for v in dev.values():
        v.requires_grad_(False)
        v.grad = None
    xg = x.cuda().requires_grad_(True)
    blk(xg).backward(dy.cuda())
    assert np.array_equal(xg.grad.cpu().numpy(), ref[1]) and all(v.grad is None for v in dev.values())


def test_plain_block_is_as_it_was(BL):
    """Without the additions a block is the torch-glue one, and refuses the
    cache's calls."""
    blk, _, x, _, _ = _setup(BL, 128, 256, 2, 8, 1, 9, 6, None, extras=False)
    plain = BL.QLoraBlock.__new__(BL.QLoraBlock)
    plain.__dict__.update(blk.__dict__)
    plain.fused = False
    assert _rel(plain(x.cuda()).detach().cpu(), blk(x.cuda()).detach().cpu()) < 2e-2
    with pytest.raises(ValueError):
        plain.prefill(x.cuda(), blk.cache(4, 16, 1, 32))
    with pytest.raises(ValueError):
        plain.decode(x[0, :1].cuda(), blk.cache(4, 16, 1, 32))


@pytest.mark.parametrize("rot,inter", [(64, False), (32, True), (None, False)])
def test_decoding_equals_the_whole_sequence(BL, rot, inter):
    """Three sequences: a prompt of 21 tokens, then 20 tokens one at a time; the
    outputs at every position are the whole sequence's."""
    _log(f"fused block decode rot={rot}")
    batch, prompt, total = 3, 21, 41
    blk, _, x, _, ref = _setup(BL, 256, 512, 4, 16, batch, total, 77, rot, inter)
    want = ref(x.numpy())
    cache = blk.cache(num_pages=12, page_size=16, max_seqs=batch, max_len=48)
    xc = x.cuda()
    out = [blk.prefill(xc[:, :prompt].contiguous(), cache)]
    for i in range(prompt, total):
        out.append(blk.decode(xc[:, i].contiguous(), cache)[:, None])
    got = torch.cat(out, 1).cpu().numpy()
    assert cache.host_lens == [total] * batch and cache.lens.tolist() == [total] * batch
    assert _rel(got, want) < 2e-2
    for i in range(total):
        assert _rel(got[:, i], want[:, i]) < 3e-2, i
    for _ in range(48 - total):
        blk.decode(xc[:, 0].contiguous(), cache)
    with pytest.raises(ValueError, match="max_len"):
        blk.decode(xc[:, 0].contiguous(), cache)
    small = blk.cache(num_pages=2, page_size=16, max_seqs=batch, max_len=48)
    with pytest.raises(ValueError, match="pages needed"):
        small.add([1, 1, 1])
    assert small.host_lens == [0, 0, 0] and small.used == 0


@pytest.mark.parametrize("which", ["w_pre", "w_post", "gate"])
def test_norm_residual_gradients_one_at_a_time(BL, which):
    """Every gain alone trainable, the others frozen or absent: the gradient is
    the one of all together."""
    _log(f"norm_residual autograd {which}")
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, h = n(2, 5, 96), n(2, 5, 96).to(torch.bfloat16)
    dxo, dn = n(2, 5, 96), n(2, 5, 96).to(torch.bfloat16)
    gains = {"w_pre": n(96), "w_post": n(96), "gate": n(96)}

    def grads(gains, train):
        leaf = {k: v.clone().requires_grad_(k in train) for k, v in gains.items()}
        hl = h.clone().requires_grad_(True)
        xo, nn = BL.norm_residual(x, hl, **leaf, alpha=0.5)
        ((xo * dxo).sum() + (0.0 if nn is None else (nn.float() * dn.float()).sum())).backward()
        return {k: v.grad for k, v in leaf.items()}, hl.grad

    full, dh = grads(gains, list(gains))
    one, dh1 = grads(gains, [which])
    assert torch.equal(dh, dh1) and torch.equal(one[which], full[which])
    assert all(v is None for k, v in one.items() if k != which)
    for drop in gains:
        if drop == which:
            continue
        rest = {k: v for k, v in gains.items() if k != drop}
        a, da = grads(rest, list(rest))
        b, db = grads(rest, [which])
        assert torch.equal(da, db) and torch.equal(a[which], b[which])
    if which == "gate":   # neither norm: the step itself
        leaf = gains["gate"].clone().requires_grad_(True)
        BL.norm_residual(x, h, gate=leaf, alpha=0.5)[0].backward(dxo)
        ref = (0.5 * dxo.double() * h.double()).sum((0, 1))
        size = (0.5 * dxo.double() * h.double()).abs().sum((0, 1))
        assert ((leaf.grad.double() - ref).abs() <= 32 * 2.0 ** -24 * size).all()


def test_second_derivatives_are_refused(BL):
    x = torch.randn(3, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda")
    _, n = BL.norm_residual(x, None, w, n_dtype=torch.float32)
    (gx,) = torch.autograd.grad(n.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()


def test_rope_autograd(BL):
    """Gradients of q alone, of k alone and of both; positions changed between
    forward and backward are noticed."""
    _log("rope autograd")
    from bit_nf4_quantized_quantize_amd import RopeTable
    tab = RopeTable(32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k = (torch.randn(7, h, 64, generator=g, device="cuda") for h in (4, 2))
    w = torch.randn(7, 4, 64, generator=g, device="cuda")
    pos = torch.arange(7, device="cuda", dtype=torch.int32) * 100

    def grads(use_q, use_k, loss_q, loss_k):
        ql, kl = (z.clone().requires_grad_(True) if u else None for z, u in ((q, use_q), (k, use_k)))
        qo, ko = BL.rope(ql, kl, tab, pos)
        loss = 0
        if loss_q:
            loss = loss + (qo * w).sum()
        if loss_k:
            loss = loss + (ko * w[:, :2]).sum()
        loss.backward()
        return ql.grad if use_q else None, kl.grad if use_k else None

    both = grads(True, True, True, True)
    assert torch.equal(grads(True, False, True, False)[0], both[0])
    assert torch.equal(grads(False, True, False, True)[1], both[1])
    only = grads(True, True, True, False)
    assert torch.equal(only[0], both[0]) and (only[1] is None or not only[1].any())
    # the map is linear and orthogonal: <R q, w> = <q, R^T w>
    lhs = (BL.rope(q, None, tab, pos)[0].double() * w.double()).sum()
    size = (q.double().abs().sum(-1) * w.double().abs().sum(-1)).sum()
    assert abs(float(lhs - (q.double() * both[0].double()).sum())) <= 16 * 2.0 ** -24 * float(size)
    ql = q.clone().requires_grad_(True)
    p2 = pos.clone()
    out = BL.rope(ql, None, tab, p2)[0]
    p2.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


def test_gradients_that_start_off_a_16_byte_boundary(BL):
    """A contiguous slice of a larger gradient (as cat's backward hands out)."""
    _log("norm_residual: gradient slices")
    from bit_nf4_quantized_quantize_amd import RopeTable
    x, h = torch.randn(3, 33, device="cuda"), torch.randn(3, 33, device="cuda").to(torch.bfloat16)
    w, dy = torch.randn(33, device="cuda"), torch.randn(4, 33, device="cuda")

    def run(cat):
        xl, hl = x.clone().requires_grad_(True), h.clone().requires_grad_(True)
        xo, n = BL.norm_residual(xl, hl, w)
        if cat:
            (torch.cat([torch.zeros(1, 33, device="cuda"), xo]) * dy).sum().backward(retain_graph=True)
            torch.cat([n[:1] * 0, n]).backward(dy.to(torch.bfloat16))
        else:
            (xo * dy[1:]).sum().backward(retain_graph=True)
            n.backward(dy[1:].to(torch.bfloat16).clone())
        return xl.grad, hl.grad

    assert all(torch.equal(a, b) for a, b in zip(run(True), run(False)))
    tab = RopeTable(2, device="cuda")
    q, pos = torch.randn(3, 1, 3, device="cuda"), torch.arange(3, device="cuda", dtype=torch.int32)
    dq = torch.randn(4, 1, 3, device="cuda")

    def turn(cat):
        ql = q.clone().requires_grad_(True)
        o = BL.rope(ql, None, tab, pos)[0]
        torch.cat([torch.zeros(1, 1, 3, device="cuda"), o]).backward(dq) if cat else o.backward(dq[1:].clone())
        return ql.grad

    assert torch.equal(turn(True), turn(False))


def test_cached_calls_check_before_they_touch_the_cache(BL):
    blk, _, x, _, _ = _setup(BL, 128, 256, 2, 8, 2, 9, 6, 32)
    for bad in (dict(page_size=8), dict(page_size=48), dict(head_dim=20), dict(head_dim=264)):
        with pytest.raises(ValueError):
            BL.PagedCache(**{**dict(num_pages=2, page_size=16, heads=2, head_dim=64, max_seqs=1, max_len=32), **bad})
    c = blk.cache(8, 16, 2, 32)
    xc = x.cuda()
    other = BL.PagedCache(8, 16, 4, 32, 2, 32)
    for f in (lambda: blk.prefill(xc.double(), c), lambda: blk.prefill(xc[..., :64].contiguous(), c),
              lambda: blk.prefill(x, c), lambda: blk.decode(xc[:, 0].half(), c), lambda: blk.decode(xc[0], c),
              lambda: blk.prefill(xc, other), lambda: blk.decode(xc[:, 0], other)):
        with pytest.raises(ValueError):
            f()
    assert c.host_lens == [0, 0] and c.used == 0 and other.used == 0 and c.lens.tolist() == [0, 0]
