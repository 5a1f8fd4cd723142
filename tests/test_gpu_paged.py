"""GPU parity: attention of one new token over the paged cache, and the plan of
a batch, against the fp64 oracle.

Tolerance of the attention: a score is a sum of at most 256 exact bfloat16
products in fp32, so it is off by e = (d + 8) u scale sum |q_i k_i| (u = 2^-24)
and its weight by a relative e plus 8 u of the exponential and of the score's
own size; a weight enters the product with V as a bfloat16 number and the bfloat16
remainder (half a step of each, 2^-16) and n terms are added, so with W = sum p_i
|v_i|
    |err| <= (2^-16 + 2 e + (n + 256) u) W + 2^-8 |out|,
the last for the rounding of the output.  The log-sum-exp carries e + (n + 64)
u and its own rounding."""

import math
import sys

import numpy as np
import pytest
import torch

from oracle import decoder as od

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = torch.bfloat16


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


def _setup(S, H, KV, d, page, cols, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: (spread * torch.randn(*s, generator=g, device="cuda")).to(BF)  # noqa: E731
    pages = S * cols + 2
    table = torch.randperm(pages, generator=g, device="cuda")[:S * cols].view(S, cols).to(torch.int32)
    return r(S, H, d), r(pages, KV, page, d), r(pages, KV, page, d), table




def _check(D, q, kc, vc, table, lengths, scale=None):
    S, H, d = q.shape
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    lse = torch.empty(S, H, device="cuda")
    out = D.qlora_paged_attention(q, kc, vc, table, lens, scale=scale, lse=lse)
    sc = 1 / math.sqrt(d) if scale is None else scale
    tb = table.cpu().numpy()
    ref, rlse, wt = od.paged_attention(_n(q), _n(kc), _n(vc), tb, lengths, sc)
    n = max(max(lengths), 0)
    qa = np.abs(_n(q)).max(-1)                                         # a score's terms: |q| |k| d at most
    kmax = float(np.abs(_n(kc)[np.isfinite(_n(kc))]).max())
    e = ((d + 8) * U * abs(sc) * (np.abs(_n(q)).sum(-1) * kmax) + 8 * U * abs(sc) * qa * kmax * d)
    tol = (2.0 ** -16 + 2 * e[..., None] + (n + 256) * U) * wt + 2.0 ** -8 * np.abs(ref)
    err = np.abs(_n(out) - ref)
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))
    got = _n(lse)
    none = np.isneginf(rlse)
    assert np.array_equal(np.isneginf(got), none)
    ok = np.abs(got[~none] - rlse[~none]) <= (e + (n + 64) * U)[~none] + 4 * U * np.abs(rlse[~none])
    assert ok.all()
    assert not _n(out)[none].any()
    plain = D.qlora_paged_attention(q, kc, vc, table, lens, scale=scale)
    assert torch.equal(plain, out)
    return out


SHAPES = [  # S, q heads, kv heads, head_dim, page, columns, lengths
    (1, 1, 1, 8, 16, 1, [1]), (1, 32, 32, 128, 16, 40, [512]), (3, 4, 2, 64, 16, 9, [0, 1, 144]),
    (2, 8, 1, 128, 32, 5, [31, 33]), (5, 6, 2, 80, 16, 12, [15, 16, 17, 100, 191]), (2, 16, 1, 96, 64, 4, [255, 256]),
    (2, 34, 2, 64, 128, 3, [384, 200]), (1, 40, 1, 128, 16, 80, [1279]), (4, 7, 7, 256, 16, 20, [320, 3, 64, 65]),
    (2, 64, 8, 128, 64, 33, [2111, 700]), (1, 2, 2, 32, 1024, 2, [1500]), (70, 4, 4, 64, 16, 8, list(range(0, 70))),
    (2, 3, 1, 40, 16, 30, [470, 479]), (1, 8, 8, 192, 16, 20, [300]), (1, 20, 1, 16, 16, 20, [299]),
    (1, 4, 4, 128, 16, 520, [8311]), (1, 2, 1, 64, 64, 1100, [70000]), (2, 3, 1, 128, 16, 2000, [31999, 700])]


@pytest.mark.parametrize("S,H,KV,d,page,cols,lengths", SHAPES)
def test_attention(D, S, H, KV, d, page, cols, lengths):
    _log(f"paged attention S={S} H={H} KV={KV} d={d} page={page} lengths={lengths[:8]}")
    q, kc, vc, table = _setup(S, H, KV, d, page, cols, seed=S * 1000 + d)
    _check(D, q, kc, vc, table, lengths)


def test_lengths_around_tiles(D):
    """Every length up to 300, in one batch of heads shared by 4 and by 1."""
    for H, KV in ((8, 2), (2, 2)):
        lengths = list(range(300))
        _log(f"paged attention lengths 0..299 H={H}")
        q, kc, vc, table = _setup(300, H, KV, 64, 16, 19, seed=H)
        _check(D, q, kc, vc, table, lengths)


@pytest.mark.parametrize("H,KV,d,page", [(4, 4, 128, 16), (8, 1, 64, 32), (32, 2, 128, 64), (3, 3, 256, 16)])
def test_what_lies_behind_the_length_is_not_used(D, H, KV, d, page):
    """NaN and infinities in the slots behind the last token, in pages of no
    sequence, and in table entries behind the length."""
    _log(f"paged attention garbage H={H} KV={KV} d={d} page={page}")
    cols = 256 // page
    q, kc, vc, table = _setup(4, H, KV, d, page, cols, seed=7)
    lengths = [1, page - 1, 101, 250]
    ref = _check(D, q, kc, vc, table, lengths)
    used = torch.zeros(kc.shape[0], page, dtype=torch.bool)
    for s, n in enumerate(lengths):
        for i in range(n):
            used[int(table[s, i // page]), i % page] = True
    dead = ~used.cuda()
    kc.transpose(1, 2)[dead] = float("nan")
    vc.transpose(1, 2)[dead] = float("inf")
    t2 = table.clone()
    for s, n in enumerate(lengths):
        t2[s, -(-n // page):] = 2 ** 31 - 1
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    got = D.qlora_paged_attention(q, kc, vc, t2, lens)
    assert torch.equal(got, ref)


def test_missing_pages_and_wild_lengths(D):
    """Pages outside the cache take no part; lengths are cut to the table."""
    _log("paged attention missing pages")
    q, kc, vc, table = _setup(5, 4, 2, 64, 16, 20, seed=11)
    pages = kc.shape[0]
    table[0, 3], table[0, 4], table[1, 0], table[3, :] = -1, pages, -2 ** 31, 2 ** 31 - 1
    table[2, 19] = pages + 5
    out = _check(D, q, kc, vc, table, [320, 300, 320, 200, 17])
    assert not out[3].any()
    lens = torch.tensor([2 ** 31 - 1, -1, -2 ** 31, 5, 320], dtype=torch.int32, device="cuda")
    ref = torch.tensor([320, 0, 0, 5, 320], dtype=torch.int32, device="cuda")
    a = D.qlora_paged_attention(q, kc, vc, table, lens)
    assert torch.equal(a, D.qlora_paged_attention(q, kc, vc, table, ref))


def test_large_scores(D):
    """Scores far apart: weights that underflow, and a maximum that arrives
    late or early in the sequence."""
    _log("paged attention large scores")
    q, kc, vc, table = _setup(2, 4, 4, 64, 16, 40, seed=13, spread=4.0)
    _check(D, q, kc, vc, table, [640, 600])
    for at in (0, 639, 300):
        k2 = kc.clone()
        k2[int(table[0, at // 16]), :, at % 16] = q[0] * 8
        _check(D, q, k2, vc, table, [640, 600])
    _check(D, q, kc, vc, table, [640, 600], scale=0.0)
    _check(D, q, kc, vc, table, [640, 600], scale=-0.3)


def test_strided_queries(D):
    _log("paged attention strided q")
    q, kc, vc, table = _setup(6, 4, 2, 64, 16, 9, seed=17)
    full = torch.zeros(6, 8 * 64 + 8, dtype=BF, device="cuda")
    view = full[:, :4 * 64].view(6, 4, 64)
    view.copy_(q)
    lens = torch.tensor([5, 60, 144, 0, 99, 1], dtype=torch.int32, device="cuda")
    out = torch.full((6, 4, 64), 3.0, dtype=BF, device="cuda")
    got = D.qlora_paged_attention(view, kc, vc, table, lens, out=out)
    assert got is out and torch.equal(out, D.qlora_paged_attention(q, kc, vc, table, lens))


def test_cache_beyond_32_bits(D):
    """Elements of the cache whose offset passes 2^32."""
    _log("paged attention 64-bit offsets")
    KV, page, d = 8, 64, 128
    pages = (2 ** 32 + 2 ** 28) // (KV * page * d)
    kc = torch.zeros(pages, KV, page, d, dtype=BF, device="cuda")
    vc = torch.zeros(pages, KV, page, d, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(19)
    cols = 6
    top = torch.arange(pages - 2 * cols, pages, device="cuda")[torch.randperm(2 * cols, generator=g, device="cuda")]
    for p in top.tolist():
        kc[p] = torch.randn(KV, page, d, generator=g, device="cuda").to(BF)
        vc[p] = torch.randn(KV, page, d, generator=g, device="cuda").to(BF)
    q = torch.randn(2, 16, d, generator=g, device="cuda").to(BF)
    table = top.to(torch.int32).view(2, cols)
    lens = torch.tensor([383, 129], dtype=torch.int32, device="cuda")
    lo = pages - 2 * cols
    small = D.qlora_paged_attention(q, kc[lo:].clone(), vc[lo:].clone(), table - lo, lens)
    assert small.any() and torch.equal(D.qlora_paged_attention(q, kc, vc, table, lens), small)
    # and the write of a token there
    k, v = torch.randn(1, KV, d, device="cuda").to(BF), torch.randn(1, KV, d, device="cuda").to(BF)
    slot = torch.tensor([pages * page - 1], dtype=torch.int32, device="cuda")
    D.qlora_rope_cache_write(None, k, v, None, None, slot, kc, vc)
    assert torch.equal(kc[-1, :, -1], k[0]) and torch.equal(vc[-1, :, -1], v[0])


def test_other_stream_and_graph(D):
    """Two calls at once on two streams, and a graph replayed with other lengths
    and eager work between."""
    _log("paged attention stream and graph")
    q, kc, vc, table = _setup(3, 8, 2, 128, 16, 70, seed=23)
    q2 = torch.flip(q, (0,)).contiguous()
    lens = torch.tensor([1100, 3, 700], dtype=torch.int32, device="cuda")
    ref, ref2 = (D.qlora_paged_attention(z, kc, vc, table, lens) for z in (q, q2))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a = D.qlora_paged_attention(q, kc, vc, table, lens, stream=s1)
        b = D.qlora_paged_attention(q2, kc, vc, table, lens, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a, ref) and torch.equal(b, ref2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = D.qlora_paged_attention(q, kc, vc, table, lens)
    for n in ([1100, 3, 700], [0, 1120, 16], [5, 6, 7]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        ref = D.qlora_paged_attention(q, kc, vc, table, lens)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref), n


def test_no_sequences(D):
    q, kc, vc, table = _setup(2, 4, 2, 64, 16, 3, seed=29)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    assert D.qlora_paged_attention(q[:0], kc, vc, table[:0], e).shape == (0, 4, 64)
    lens = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    out = D.qlora_paged_attention(q, kc, vc, torch.empty(2, 0, dtype=torch.int32, device="cuda"), lens)
    assert out.shape == (2, 4, 64) and not out.any()


# -------------------------------------------------------------------- plan

def _plan_case(rng, S, page, chigh, nhigh, spare, cols=None):
    cached, new = rng.integers(0, chigh + 1, S), rng.integers(0, nhigh + 1, S)
    need = int(sum(-(-(c + n) // page) + c // -page for c, n in zip(cached, new)))
    have = [-(-int(c) // page) for c in cached]
    if cols is None:
        cols = max([-(-int(c + n) // page) for c, n in zip(cached, new)], default=0) + 1
    ids = rng.permutation(sum(have) + max(need + spare, 0))
    table = np.full((S, cols), -7)
    at = 0
    for s, n in enumerate(have):
        w = min(n, cols)
        table[s, :w] = ids[at:at + w]
        at += n
    return cached, new, ids[at:], table


def _dev(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _check_plan(D, cached, new, free, table, page, tokens, out=None):
    t = _dev(table)
    p = D.qlora_paged_plan(_dev(cached), _dev(new), _dev(free), t, page, tokens, out=out)
    ref = od.paged_plan(cached, new, free, table, page, tokens)
    got = (t, p.total_lens, p.starts, p.slots, p.positions, p.pages_needed)
    for g, r, name in zip(got, ref, ("table", "total_lens", "starts", "slots", "positions", "pages_needed")):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(r).reshape(-1)), name
    return p


@pytest.mark.parametrize("page", [1, 7, 16, 128])
@pytest.mark.parametrize("S,chigh,nhigh", [(1, 0, 1), (1, 50, 300), (16, 100, 1), (63, 40, 5), (64, 0, 90), (65, 33, 33),
                                           (513, 20, 9), (1500, 64, 3), (4096, 17, 2)])
def test_plan(D, S, chigh, nhigh, page):
    _log(f"plan S={S} cached<={chigh} new<={nhigh} page={page}")
    rng = np.random.default_rng(S * 7 + page)
    cached, new, free, table = _plan_case(rng, S, page, chigh, nhigh, 3)
    total = int(new.sum())
    _check_plan(D, cached, new, free, table, page, total)
    _check_plan(D, cached, new, free, table, page, total + 37)
    if total > 2:
        _check_plan(D, cached, new, free, table, page, total // 2)


def test_plan_short_of_pages_and_columns(D):
    _log("plan short")
    rng = np.random.default_rng(3)
    for spare, cols in ((-5, None), (-10 ** 6, None), (2, 2), (-4, 3)):
        cached, new, free, table = _plan_case(rng, 40, 8, 30, 20, spare, cols)
        p = _check_plan(D, cached, new, free, table, 8, int(new.sum()))
        if spare < 0 and cols is None:
            assert int(p.pages_needed) > len(free)
    # a cached page that is missing: its tokens' slots are missing
    _check_plan(D, [5, 3], [2, 4], [9, 8], [[-1, -1], [4, -1]], 8, 6)


def test_plan_odd_lengths(D):
    _log("plan negative lengths, no sequences, no tokens")
    _check_plan(D, [-4, 3, -1], [2, -5, 0], [1, 2, 3], [[0, 0]] * 3, 2, 5)
    _check_plan(D, [0, 0], [0, 0], [], [[0, 0]] * 2, 2, 4)
    _check_plan(D, [3], [2], [7], [[5, 0, 0]], 2, 0)
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    p = D.qlora_paged_plan(z, z, z, torch.empty(0, 3, dtype=torch.int32, device="cuda"), 16, 3)
    assert p.starts.tolist() == [0] and p.slots.tolist() == [-1] * 3 and p.pages_needed.tolist() == [0]


def test_plan_lengths_beyond_31_bits(D):
    """Lengths that make no sense: sums stop at 2^31 - 1, the rows that exist are
    planned as far as the table goes."""
    _log("plan lengths beyond 31 bits")
    big = 2 ** 31 - 1
    t = _dev([[-7] * 3] * 4)
    p = D.qlora_paged_plan(_dev([0, 3, big, big]), _dev([big, 7, big, 1]), _dev([5, 6, 7, 8]), t, 16, 40)
    assert p.starts.tolist() == [0, big, big, big, big] and p.total_lens.tolist() == [big, 10, big, big]
    assert p.positions.tolist() == list(range(40))
    assert p.slots.tolist() == [80 + i for i in range(16)] + [96 + i for i in range(16)] + [112 + i for i in range(8)]
    assert t.tolist() == [[5, 6, 7]] + [[-7] * 3] * 3 and p.pages_needed.tolist() == [3]
    t = _dev([[4, -7, -7]])
    p = D.qlora_paged_plan(_dev([big - 2]), _dev([5]), _dev([5, 6]), t, 16, 6)
    assert p.slots.tolist() == [-1] * 6 and p.positions.tolist() == [big - 2, big - 1, big, big, big, 0]
    assert t.tolist() == [[4, -7, -7]]


def test_plan_into_given_buffers(D):
    _log("plan out=")
    rng = np.random.default_rng(11)
    cached, new, free, table = _plan_case(rng, 20, 16, 50, 30, 5)
    T = int(new.sum()) + 4
    e = lambda n: torch.full((n,), -9, dtype=torch.int32, device="cuda")  # noqa: E731
    out = D.PagedPlan(e(20), e(21), e(T), e(T), e(1))
    assert _check_plan(D, cached, new, free, table, 16, T, out=out) is out
    with pytest.raises(ValueError):
        D.qlora_paged_plan(_dev(cached), _dev(new), _dev(free), _dev(table), 16, T, out=out._replace(slots=e(T - 1)))
    for page, tokens in ((0, T), (-1, T), (2 ** 32 + 16, T), (16, -1)):
        with pytest.raises(ValueError):
            D.qlora_paged_plan(_dev(cached), _dev(new), _dev(free), _dev(table), page, tokens)


def test_plan_graph(D):
    _log("plan graph")
    rng = np.random.default_rng(5)
    cached, new, free, table = _plan_case(rng, 50, 16, 90, 40, 400)
    c, n, f, t = _dev(cached), _dev(new), _dev(free), _dev(table)
    t0 = t.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p = D.qlora_paged_plan(c, n, f, t, 16, 2500)
    for k in range(3):
        n.copy_(_dev(rng.permutation(new)))
        t.copy_(t0)
        ref = D.qlora_paged_plan(c, n, f, t, 16, 2500)
        want = t.clone()
        t.copy_(t0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(t, want) and all(torch.equal(a, b) for a, b in zip(p, ref)), k


def test_decode_steps_together(D):
    """Plan, write and attend, token by token for three sequences that join at
    different times: every step equals attention over the tokens' own history
    held apart in fp64."""
    _log("decode steps together")
    S, H, KV, d, page, cols = 3, 6, 2, 64, 16, 4
    g = torch.Generator(device="cuda").manual_seed(31)
    pages = S * cols
    kc = torch.full((pages, KV, page, d), float("nan"), dtype=BF, device="cuda")
    vc = kc.clone()
    free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((S, cols), -1, dtype=torch.int32, device="cuda")
    cached = torch.zeros(S, dtype=torch.int32, device="cuda")
    tab = D.RopeTable(32, base=1000.0, device="cuda")
    f, _ = od.rope_frequencies(32, base=1000.0)
    ks, vs = [[] for _ in range(S)], [[] for _ in range(S)]
    for step in range(40):
        new = torch.tensor([13 if step == 0 else 1, int(step >= 5), int(step % 2)], dtype=torch.int32)
        T = int(new.sum()) + 2   # two padded rows
        p = D.qlora_paged_plan(cached, new.cuda(), free, table, page, T)
        q, k, v = (torch.randn(T, h, d, generator=g, device="cuda").to(BF) for h in (H, KV, KV))
        qo = D.qlora_rope_cache_write(q, k, v, tab, p.positions, p.slots, kc, vc)
        last = (p.starts[1:] - 1).clamp(min=0).long()
        lens = torch.where(new.cuda() > 0, p.total_lens, torch.zeros_like(p.total_lens))
        out = D.qlora_paged_attention(qo[last].contiguous(), kc, vc, table, lens)
        free = free[int(p.pages_needed):].contiguous()
        cached = p.total_lens
        pos = p.positions.cpu().numpy()
        kr = od.rope(_n(k), pos, f)
        for s in range(S):
            for r in range(int(p.starts[s]), int(p.starts[s + 1])):
                ks[s].append(kr[r])
                vs[s].append(_n(v)[r])
            if int(new[s]) == 0:
                assert not out[s].any()
                continue
            K, V = np.array(ks[s]), np.array(vs[s])
            qr = od.rope(_n(q), pos, f)[int(last[s])]
            for h in range(H):
                j = h // (H // KV)
                sc = K[:, j] @ qr[h] / math.sqrt(d)
                w = np.exp(sc - sc.max())
                w /= w.sum()
                # q and k are rounded to bfloat16 (2^-8 each way in a score of size |q||k|/8), weights and
                # the output once more
                e = 2 * 2.0 ** -8 * np.linalg.norm(qr[h]) * np.linalg.norm(K[:, j], axis=1).max() / math.sqrt(d)
                err = np.abs(_n(out[s, h]) - w @ V[:, j])
                assert (err <= (np.expm1(2 * e) + 2.0 ** -7) * (w @ np.abs(V[:, j])) + 1e-6).all()
