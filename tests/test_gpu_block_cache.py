"""The fused block's cached calls where something is wrong or missing: a call that
fails leaves the cache as it was."""

import pytest
import torch

pytestmark = pytest.mark.gpu

HIDDEN, MLP, HEADS, R = 128, 256, 2, 8


@pytest.fixture(scope="module")
def BL():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_quantize_amd import binding, block
    binding.lib()
    return block


def _block(BL, rope=None, **extras):
    g = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    shapes = BL.linear_shapes(HIDDEN, MLP)
    W = {n: rn(*sh) * 0.02 for n, sh in shapes.items()}
    A = {n: rn(shapes[n][1], R) * 0.05 for n in BL.LINEARS}
    Bm = {n: rn(R, shapes[n][0]) * 0.05 for n in BL.LINEARS}
    return BL.QLoraBlock(W, A, Bm, torch.ones(HIDDEN, device="cuda"), torch.ones(HIDDEN, device="cuda"), 2.0, HEADS,
                         rope=rope, fused=True, **extras)


def _state(c):
    return c.lens.tolist(), list(c.host_lens), c.used


def _bad_blocks(BL):
    from bit_nf4_quantized_quantize_amd import RopeTable
    return {
        "more rotated elements than a head has": _block(BL, rope=RopeTable(128, device="cuda")),
        "a rotary table on the host": _block(BL, rope=RopeTable(64, device="cpu")),
        "a gain of another type": _block(BL, post1=torch.ones(HIDDEN, dtype=torch.bfloat16, device="cuda")),
        "a gate of another width": _block(BL, gate2=torch.ones(HIDDEN - 1, device="cuda")),
    }


@pytest.mark.parametrize("what", ["more rotated elements than a head has", "a rotary table on the host",
                                  "a gain of another type", "a gate of another width"])
def test_a_failing_call_leaves_the_cache(BL, what):
    bad, good = _bad_blocks(BL)[what], _block(BL)
    x = torch.randn(2, 6, HIDDEN, device="cuda")
    cache, ref = good.cache(8, 16, 2, 32), good.cache(8, 16, 2, 32)
    for c in (cache, ref):
        if c is cache:
            with pytest.raises(Exception):
                bad.prefill(x[:, :5].contiguous(), c)
            assert _state(c) == ([0, 0], [0, 0], 0)
        first = good.prefill(x[:, :5].contiguous(), c)
        before = _state(c)
        if c is cache:
            with pytest.raises(Exception):
                bad.decode(x[:, 5].contiguous(), c)
            assert _state(c) == before == ([5, 5], [5, 5], 2)
        last = good.decode(x[:, 5].contiguous(), c)
        if c is cache:
            got = first.clone(), last.clone()
    assert torch.equal(got[0], first) and torch.equal(got[1], last) and _state(cache) == _state(ref)


def test_a_wrong_rotary_table_is_named(BL):
    blocks = _bad_blocks(BL)
    x = torch.randn(1, 3, HIDDEN, device="cuda")
    for what in ("more rotated elements than a head has", "a rotary table on the host"):
        with pytest.raises(ValueError, match="rotary table"):
            blocks[what].prefill(x, blocks[what].cache(4, 16, 1, 32))


@pytest.mark.parametrize("shape", [(0, 4, HIDDEN), (2, 0, HIDDEN)])
def test_no_tokens(BL, shape):
    """As the plain form: an empty result, an empty gradient and zeros for the
    adapters."""
    from bit_nf4_quantized_quantize_amd import RopeTable
    plain = _block(BL)
    plain.fused = False
    for blk in (plain, _block(BL), _block(BL, rope=RopeTable(64, device="cuda"),
                                          post1=torch.ones(HIDDEN, device="cuda", requires_grad=True))):
        x = torch.randn(*shape, device="cuda", requires_grad=True)
        y = blk(x)
        assert y.shape == shape
        y.sum().backward()
        assert x.grad.shape == shape
        assert all(p.grad is not None and not p.grad.any() for p in blk.parameters())
        if blk.post1 is not None:
            assert torch.equal(blk.post1.grad, torch.zeros(HIDDEN, device="cuda"))
        if blk.fused:
            c = blk.cache(4, 16, 2, 32)
            assert blk.prefill(x.detach(), c).shape == shape and _state(c) == ([0, 0], [0, 0], 0)


def test_cached_calls_are_refused_in_a_capture(BL):
    """The counts come from the host: a replay could not make them again."""
    blk = _block(BL)
    cache = blk.cache(8, 16, 2, 32)
    x = torch.randn(2, 3, HIDDEN, device="cuda")
    first = blk.prefill(x, cache)
    torch.cuda.synchronize()
    before = _state(cache)
    graph = torch.cuda.CUDAGraph()
    row = x[:, 0].contiguous()
    with torch.cuda.graph(graph):
        y = row * 2
        with pytest.raises(RuntimeError, match="captured"):
            blk.decode(row, cache)
    graph.replay()
    torch.cuda.synchronize()
    assert _state(cache) == before and torch.equal(y, row * 2) and first.isfinite().all()
    assert blk.decode(row, cache).isfinite().all()
