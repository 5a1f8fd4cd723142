"""Fused blocks on several streams and in captured graphs: nothing of a call is shared
with another, so each gives, bit for bit, what it gives alone."""

import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

HIDDEN, MLP, HEADS, R = 256, 704, 4, 16


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


def _block(BL, seed):
    from bit_nf4_quantized_quantize_amd import RopeTable
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    shapes = BL.linear_shapes(HIDDEN, MLP)
    W = {n: rn(*sh) * 0.02 for n, sh in shapes.items()}
    A = {n: rn(shapes[n][1], R) * 0.05 for n in BL.LINEARS}
    Bm = {n: rn(R, shapes[n][0]) * 0.05 for n in BL.LINEARS}
    one = torch.ones(HIDDEN, device="cuda")
    return BL.QLoraBlock(W, A, Bm, one, one, 1.0, HEADS, rope=RopeTable(64, device="cuda"))


def _step(blk, x, dy):
    """Output, input gradient and adapter gradients of one training step."""
    for p in blk.parameters():
        p.grad = None
    xl = x.clone().requires_grad_(True)
    y = blk(xl)
    y.backward(dy)
    return [y.detach(), xl.grad] + [p.grad for p in blk.parameters()]


def test_a_block_takes_no_shared_workspace(BL, monkeypatch):
    _log("block workspaces")
    from bit_nf4_quantized_quantize_amd import binding
    blk = _block(BL, 1)
    shared = {}
    monkeypatch.setattr(binding, "_default_ws", shared)
    x = torch.randn(2, 9, HIDDEN, device="cuda")
    _step(blk, x, x)
    cache = blk.cache(8, 16, 2, 32)
    blk.prefill(x, cache)
    blk.decode(x[:, 0].contiguous(), cache)
    torch.cuda.synchronize()
    assert not shared


def test_two_streams(BL):
    """Two threads, each training a block and decoding with it on a stream of its
    own."""
    _log("blocks on two streams")
    jobs = []
    for seed, seq in ((2, 33), (3, 64)):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x, dy = (torch.randn(2, seq, HIDDEN, generator=g, device="cuda") for _ in range(2))
        blk = _block(BL, seed)

        def work(blk=blk, x=x, dy=dy, seq=seq):
            out = _step(blk, x, dy)
            cache = blk.cache(16, 16, 2, 96)
            return out + [blk.prefill(x, cache)] + [blk.decode(x[:, i].contiguous(), cache) for i in range(3)]
        jobs.append((work, [t.clone() for t in work()]))
    torch.cuda.synchronize()
    wrong = []

    def run(work, want):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(15):
                    got = work()
                    stream.synchronize()
                    wrong.extend(i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b))
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))

    threads = [threading.Thread(target=run, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_a_captured_forward_and_larger_eager_calls(BL):
    """A graph replayed between eager calls of more tokens and other tensors' life:
    every replay is the eager result, and the other tensors keep their values."""
    _log("captured block")
    blk = _block(BL, 4)
    x = torch.randn(1, 20, HIDDEN, device="cuda")
    with torch.no_grad():
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            blk(x)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = blk(x)
        for k in range(4):
            x.copy_(torch.randn(1, 20, HIDDEN, device="cuda"))
            big = blk(torch.randn(4, 100 * (k + 1), HIDDEN, device="cuda"))
            held = [torch.full((16 << 20,), float(i), device="cuda") for i in range(4)]
            want = blk(x)
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), k
            assert all(bool((t == float(i)).all()) for i, t in enumerate(held)) and big.isfinite().all()
            del held, big
