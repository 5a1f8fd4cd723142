"""The fused block decoding from an 8-bit cache and behind a prefix that its
sequences share: prefill_shared, prefill and decode together, against the block's
own forward over whole sequences.

The cached calls round what the forward keeps in fp32 (keys, values and weights in
bfloat16: 2e-2 of the output, as the decoder's other tests have it).  Rows in 8
bits are off by half a step of codes, at most 1/254 of a row's largest size in
whole numbers and 2^-4 of an element in E4M3; the attention's output is a weighted
mean of such rows and one part of the output among three (the stream and two
branches), so it adds at most 1e-2 (a largest size of 2.6 root mean squares) and
2^-4."""

import numpy as np
import pytest
import torch

from oracle import kvcache as ok

pytestmark = pytest.mark.gpu

HIDDEN, MLP, HEADS, R = 256, 512, 4, 8
D_HEAD = HIDDEN // HEADS
KINDS = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOL = {"bf16": 2e-2, "int8": 2e-2 + 1e-2, "e4m3": 2e-2 + 2.0 ** -4}


@pytest.fixture(scope="module")
def BL():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_quantize_amd import block, kvcache
    kvcache.native()
    return block


def _block(BL, rot=None, inter=False, **extras):
    from bit_nf4_quantized_quantize_amd import RopeTable
    g = torch.Generator().manual_seed(4)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    shapes = BL.linear_shapes(HIDDEN, MLP)
    W = {n: rn(*sh) * 0.05 for n, sh in shapes.items()}
    A = {n: rn(shapes[n][1], R) * 0.05 for n in BL.LINEARS}
    Bm = {n: rn(R, shapes[n][0]) * 0.05 for n in BL.LINEARS}
    rope = None if rot is None else RopeTable(rot, interleaved=inter)
    return BL.QLoraBlock(W, A, Bm, 1 + 0.1 * rn(HIDDEN), 1 + 0.1 * rn(HIDDEN), 2.0, HEADS, rope=rope, fused=True, **extras)


def _x(*shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, HIDDEN, generator=g).cuda()


def _rel(a, b):
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("rot,inter,seqs,prefix,prompt,more", [
    (64, False, 3, 37, 5, 19),       # 3 rows to a key head: narrow workgroups
    (32, True, 40, 70, 3, 4),        # 40 rows: wide ones
    (None, False, 2, 16, 0, 18),     # no prompts of their own, a whole page of prefix
])
def test_decoding_behind_a_shared_prefix(BL, kind, rot, inter, seqs, prefix, prompt, more):
    blk = _block(BL, rot, inter)
    shared, own = _x(prefix, seed=1), _x(seqs, prompt + more, seed=2)
    whole = torch.cat((shared.expand(seqs, -1, -1), own), 1)
    want = blk(whole).detach()
    cache = blk.cache(num_pages=8 + seqs * 3, page_size=16, max_seqs=seqs, max_len=48, dtype=KINDS[kind], max_prefix=80)
    first = blk.prefill_shared(shared, cache)
    assert cache.host_prefix == prefix and cache.prefix_len.tolist() == [prefix] and cache.used == -(-prefix // 16)
    out = []
    if prompt:
        out.append(blk.prefill(own[:, :prompt].contiguous(), cache))
    for i in range(prompt, prompt + more):
        out.append(blk.decode(own[:, i].contiguous(), cache)[:, None])
    got = torch.cat(out, 1)
    assert cache.host_lens == [prompt + more] * seqs
    assert _rel(first, want[0, :prefix]) < 2e-2          # the prefix attends to what is not yet coded
    assert _rel(got, want[:, prefix:]) < TOL[kind]
    for i in range(prompt + more):
        assert _rel(got[:, i], want[:, prefix + i]) < 1.5 * TOL[kind], i


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_what_an_8_bit_cache_holds(BL, kind):
    """Beside a bfloat16 cache filled by the same calls: the values are its values
    coded, the keys within half a step and a rounding to bfloat16 (2^-8)."""
    blk = _block(BL, 64)
    caches = {k: blk.cache(12, 16, 3, 48, KINDS[k]) for k in ("bf16", kind)}
    x = _x(3, 20)
    ys = {}
    for k, c in caches.items():
        ys[k] = [blk.prefill(x[:, :14].contiguous(), c)] + [blk.decode(x[:, i].contiguous(), c)[:, None] for i in range(14, 20)]
    full, rows = caches["bf16"], caches[kind].rows
    assert torch.equal(full.table, caches[kind].table)
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    for s in range(3):
        for i in range(20):
            page, at = int(full.table[s, i // 16]), i % 16
            codes, scale = ok.encode(n(full.v[page, :, at]), kind)
            assert np.array_equal(n(rows.v[page, :, at]), codes)
            assert np.array_equal(rows.v_scale[page, :, at].cpu().numpy(), scale)
            ref, sc, c = n(full.k[page, :, at]), n(rows.k_scale[page, :, at])[:, None], n(rows.k[page, :, at])
            top = np.abs(ref).max(-1, keepdims=True)
            assert (np.abs(c * sc - ref) <= ok.half_step(c, kind) * sc + 2.0 ** -7 * top).all()
    assert torch.equal(ys[kind][0], ys["bf16"][0])        # prompts attend to what is not yet coded
    assert _rel(torch.cat(ys[kind], 1), torch.cat(ys["bf16"], 1)) < TOL[kind]


def test_refusals_leave_the_cache(BL):
    blk = _block(BL, 64)
    cache = blk.cache(6, 16, 2, 32, torch.int8, max_prefix=40)
    state = lambda: (cache.lens.tolist(), list(cache.host_lens), cache.prefix_len.tolist(), cache.host_prefix, cache.used)  # noqa: E731
    empty = state()
    for bad in (_x(0), _x(41), _x(2, 3), _x(5)[:, :64].contiguous(), _x(5).double()):
        with pytest.raises(ValueError):
            blk.prefill_shared(bad, cache)
        assert state() == empty
    with pytest.raises(ValueError, match="pages needed"):
        blk.prefill_shared(_x(20), blk.cache(1, 16, 2, 32, torch.int8, max_prefix=40))
    with pytest.raises(ValueError, match="max_prefix"):
        blk.prefill_shared(_x(1), blk.cache(6, 16, 2, 32))
    broken = _block(BL, 64, post1=torch.ones(HIDDEN, dtype=torch.bfloat16, device="cuda"))   # a gain of another type
    with pytest.raises(Exception):
        broken.prefill_shared(_x(20), cache)
    assert state() == empty
    graph = torch.cuda.CUDAGraph()
    x = _x(20)
    y = x * 2
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        z = x * 2
        with pytest.raises(RuntimeError, match="captured"):
            blk.prefill_shared(x, cache)
    graph.replay()
    torch.cuda.synchronize()
    assert state() == empty and torch.equal(y, z)
    blk.prefill_shared(x, cache)
    with pytest.raises(ValueError, match="once"):
        blk.prefill_shared(x, cache)
    blk.decode(_x(2), cache)
    assert state() == ([1, 1], [1, 1], [20], 20, 4)
    with pytest.raises(Exception):
        broken.decode(_x(2), cache)
    assert state() == ([1, 1], [1, 1], [20], 20, 4)
    other = blk.cache(6, 16, 2, 32, torch.int8, max_prefix=40)
    blk.decode(_x(2), other)
    with pytest.raises(ValueError, match="before"):
        blk.prefill_shared(x, other)
