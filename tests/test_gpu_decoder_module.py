"""The compiled module behind decoder.py on the GPU: what its calls return and
keep, calls on a given stream, and two threads at once.  The values themselves
are held against the oracle elsewhere; here calls are compared with each other,
bit for bit."""

import gc
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def D():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_quantize_amd import decoder
    decoder.native()
    return decoder


def _calls(D, seed=0):
    """name -> (function, arguments) of one small call of each kind."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    b = lambda *s: n(*s).to(torch.bfloat16)  # noqa: E731
    S, H, K, d, page = 5, 8, 2, 64, 16
    lens = torch.tensor([40, 0, 17, 1, 64], **I32)
    table = D.RopeTable(d)
    x, h, w = b(33, 256), b(33, 256), n(256)
    return {
        "norm_fwd": (D.qlora_norm_residual_fwd, dict(x=x, h=h, w_pre=w, w_post=w, gate=w)),
        "norm_bwd": (D.qlora_norm_residual_bwd, dict(dxo=x, dn=h, xo=x, h=h, w_pre=w, w_post=w, gate=w,
                                                     need_gains=True)),
        "rope": (D.qlora_rope, dict(q=b(S, H, d), k=b(S, K, d), table=table, positions=lens)),
        "write": (D.qlora_rope_cache_write, dict(
            q=b(S, H, d), k=b(S, K, d), v=b(S, K, d), table=table, positions=lens,
            slots=torch.tensor([3, -1, 17, 40, 319], **I32), k_cache=b(20, K, page, d), v_cache=b(20, K, page, d))),
        "plan": (D.qlora_paged_plan, dict(
            cached_lens=lens, new_lens=torch.ones(S, **I32), free_pages=torch.arange(10, 20, **I32),
            block_table=torch.arange(5 * S, **I32).view(S, 5) % 20, page_size=page, tokens=S + 2)),
        "attention": (D.qlora_paged_attention, dict(
            q=b(S, H, d), k_cache=b(20, K, page, d), v_cache=b(20, K, page, d),
            block_table=torch.arange(4 * S, **I32).view(S, 4), lengths=lens)),
    }


NAMES = ("norm_fwd", "norm_bwd", "rope", "write", "plan", "attention")


def _flat(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


def _same(a, b):
    a, b = _flat(a), _flat(b)
    return len(a) == len(b) and all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
def test_nothing_is_kept(D, name):
    """No reference to an argument or a result outlives its call, and refused
    calls keep none either."""
    f, kw = _calls(D)[name]
    tensors = [t for t in kw.values() if isinstance(t, torch.Tensor)]
    f(**kw)
    torch.cuda.synchronize()
    gc.collect()
    counts, memory = [sys.getrefcount(t) for t in tensors], torch.cuda.memory_allocated()
    for _ in range(50):
        f(**kw)
    for key, t in kw.items():
        if isinstance(t, torch.Tensor):
            for bad in (3, t.cpu(), t.double() if t.dtype != torch.int32 else t.long()):
                with pytest.raises((TypeError, ValueError)):
                    f(**{**kw, key: bad})
    del t, bad
    gc.collect()
    assert [sys.getrefcount(t) for t in tensors] == counts
    assert torch.cuda.memory_allocated() == memory


def test_given_tensors_are_returned(D):
    calls = _calls(D)
    f, kw = calls["norm_fwd"]
    xo, n = torch.empty_like(kw["x"]), torch.empty_like(kw["x"])
    r = f(**kw, xo=xo, n=n)
    assert r[0] is xo and r[1] is n and _same(r, f(**kw))
    r = f(kw["x"], w_pre=kw["w_pre"])
    assert r[0] is kw["x"]
    assert f(kw["x"], kw["h"])[1] is None
    f, kw = calls["norm_bwd"]
    dx, dh = torch.empty_like(kw["xo"]), torch.empty_like(kw["xo"])
    r = f(**kw, dx=dx, dh=dh)
    assert r.dx is dx and r.dh is dh and _same(r, f(**kw))
    r = f(**{**kw, "need_gains": False, "need_dh": False})
    assert r.dh is None and r.dw_pre is None and r.dw_post is None and r.dgate is None
    f, kw = calls["rope"]
    q, k = torch.empty_like(kw["q"]), torch.empty_like(kw["k"])
    r = f(**kw, q_out=q, k_out=k)
    assert r[0] is q and r[1] is k and _same(r, f(**kw))
    assert f(**{**kw, "q": None})[0] is None and f(**{**kw, "k": None})[1] is None
    f, kw = calls["write"]
    q = torch.empty_like(kw["q"])
    assert f(**kw, q_out=q) is q and _same(q, f(**kw)) and f(**{**kw, "q": None}) is None
    f, kw = calls["plan"]
    table = kw["block_table"].clone()
    first = f(**kw)
    kw["block_table"].copy_(table)
    out = D.PagedPlan(*(torch.empty_like(t) for t in first))
    assert f(**kw, out=out) is out and _same(out, first)
    f, kw = calls["attention"]
    o, lse = torch.empty_like(kw["q"]), torch.empty(kw["q"].shape[:2], device="cuda")
    assert f(**kw, out=o, lse=lse) is o and _same(o, f(**kw))


@pytest.mark.parametrize("name", NAMES)
def test_a_given_stream_is_used(D, name):
    """The call waits for what its stream holds, not for the current one, and the
    current stream stays what it was."""
    f, kw = _calls(D)[name]
    want = f(**kw)
    kw = _calls(D)[name][1]
    torch.cuda.synchronize()
    side, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    held = torch.empty(64 << 20, device="cuda")
    first = next(k for k in kw if isinstance(kw[k], torch.Tensor))
    right = kw[first].clone()
    kw[first].zero_()
    side.wait_stream(cur)
    with torch.cuda.stream(side):
        for _ in range(20):
            held.add_(1.0)
        kw[first].copy_(right)       # late on the side stream
    got = f(**kw, stream=side)
    assert torch.cuda.current_stream() == cur
    side.synchronize()
    assert _same(got, want)
    with torch.cuda.stream(side):
        again = f(**_calls(D)[name][1], stream=side)
    side.synchronize()
    assert _same(again, want)


def test_two_threads(D):
    """The module lets other threads run while it launches; two of them, each on
    a stream of its own, give what one gives."""
    want = {}
    for name, (f, kw) in _calls(D).items():
        want[name] = f(**kw)
    torch.cuda.synchronize()
    wrong = []

    def work():
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    for name, (f, kw) in _calls(D).items():
                        got = f(**kw)
                        stream.synchronize()
                        if not _same(got, want[name]):
                            wrong.append(name)
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_statuses_become_errors(D):
    """What the library refuses raises its error, with its message, and the next
    call works."""
    from bit_nf4_quantized_quantize_amd import binding as B
    for name, bad in (("norm_fwd", dict(eps=-1.0)), ("norm_bwd", dict(eps=-1.0)), ("attention", dict(scale=float("nan")))):
        f, kw = _calls(D)[name]
        with pytest.raises(B.QLoraError, match="qlora_"):
            f(**kw, **bad)
        f(**kw)
    f, kw = _calls(D)["write"]
    odd = D.RopeTable(64)
    odd.rot_dim, odd.turns = 66, torch.zeros(33, dtype=torch.float64, device="cuda")
    with pytest.raises(B.QLoraError, match="qlora_"):
        f(**{**kw, "table": odd})
    torch.cuda.synchronize()
