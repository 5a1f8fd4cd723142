"""GPU parity: attention of one new token per sequence over an 8-bit cache and
over a prefix that the sequences share, against the fp64 oracle.

Tolerance.  The oracle takes the numbers that the codes stand for.  A score is a
sum of at most 256 exact products in fp32, each addition off by at most a whole
step (2 u, u = 2^-24), times a scale of its row and of the softmax: off by e = 2
(d + 8) u |scale| sum |q_i k_i|, its weight by a relative e plus 16 u of the
exponential and of the size of the score.  A weight is rounded once with the
value's scale and enters the products with all its bits, over a prefix of more
than 32 rows with at least 16 (2^-16); n terms are added and parts joined, (2 n +
256) u.  With W = sum p_i |v_i|
    |err| <= (2^-16 + 2 e + (2 n + 256) u) W + 2^-8 |out| + n 2^-126 max |v|,
the second for the rounding of the output to bfloat16, the third for weights that
are no normal fp32 numbers: exp of a score 88 or more below the row's largest is
under 2^-126 of the largest weight, which is 1 and part of the sum, and may count
as nothing or as up to that.  The log-sum-exp carries e + (2 n + 64) u and its own
rounding."""

import math

import numpy as np
import pytest
import torch

from oracle import kvcache as ok

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = torch.bfloat16
KINDS = {"bf16": BF, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_quantize_amd import kvcache
    kvcache.native()
    return kvcache


def _n(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _cache(K, pages, KV, page, d, kind, g):
    """A cache full of rows of different sizes."""
    c = K.KVCache.zeros(pages, KV, page, d, KINDS[kind])
    z = [torch.randn(pages * page, KV, d, generator=g, device="cuda") *
         torch.exp(0.5 * torch.randn(pages * page, KV, 1, generator=g, device="cuda")) for _ in "kv"]
    K.qlora_kv_write(None, z[0].to(BF), z[1].to(BF), None, None,
                     torch.arange(pages * page, dtype=torch.int32, device="cuda"), c)
    return c


def _setup(K, S, H, KV, d, page, cols, pcols, kind, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = S * cols + pcols + 1
    c = _cache(K, pages, KV, page, d, kind, g)
    q = torch.randn(S, H, d, generator=g, device="cuda").to(BF)
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    return q, c, ids[:S * cols].view(S, cols).clone(), ids[S * cols:S * cols + pcols].clone()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _check(K, q, cache, table, lengths, ptable=None, plen=0, scale=None, values=None):
    """Runs the call (with a prefix if ptable is given) and checks it."""
    S, H, d = q.shape
    lse = torch.full((S, H), 7.0, device="cuda")
    if ptable is None:
        f = lambda **kw: K.qlora_kv_attention(q, cache, table, _i32(lengths), scale=scale, **kw)  # noqa: E731
    else:
        f = lambda **kw: K.qlora_prefix_attention(q, cache, ptable, _i32([plen]), table, _i32(lengths),  # noqa: E731
                                                  scale=scale, **kw)
    out = f(lse=lse)
    sc = 1 / math.sqrt(d) if scale is None else scale
    if values is None:
        values = [ok.values(_n(c), None if s is None else _n(s)) for c, s in ((cache.k, cache.k_scale),
                                                                             (cache.v, cache.v_scale))]
    ref, rlse, wt = ok.attention(_n(q), *values, table.cpu().numpy(), lengths, sc,
                                 () if ptable is None else ptable.tolist(), plen)
    page = cache.k.shape[2]
    n = max(max(lengths, default=0), 0) + max(plen, 0) if table.shape[1] else max(plen, 0)
    kmax = float(np.abs(values[0][np.isfinite(values[0])]).max())
    qsum = np.abs(_n(q)).sum(-1)
    e = 2 * (d + 8) * U * abs(sc) * qsum * kmax + 16 * U * (1 + abs(sc) * qsum * kmax)
    vmax = float(np.abs(values[1][np.isfinite(values[1])]).max())
    tol = (2.0 ** -16 + 2 * e[..., None] + (2 * n + 256) * U) * wt + 2.0 ** -8 * np.abs(ref) + n * 2.0 ** -126 * vmax
    err = np.abs(_n(out) - ref)
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()), page)
    got, none = _n(lse), np.isneginf(rlse)
    assert np.array_equal(np.isneginf(got), none) and not _n(out)[none].any()
    assert (np.abs(got[~none] - rlse[~none]) <= (e + (2 * n + 64) * U)[~none] + 4 * U * np.abs(rlse[~none])).all()
    assert torch.equal(f(), out)          # and again the same, bit for bit
    return out


OWN = [  # S, H, KV, d, page, cols, lengths
    (1, 1, 1, 16, 16, 1, [1]),
    (2, 4, 4, 128, 16, 5, [80, 0]),
    (3, 8, 2, 64, 16, 9, [1, 144, 33]),
    (2, 21, 3, 80, 32, 6, [190, 31]),                       # seven heads to a kv head, heads of 80
    (2, 40, 2, 96, 16, 4, [17, 64]),                        # twenty heads to one
    (2, 16, 1, 256, 64, 3, [129, 15]),
    (4, 4, 2, 112, 128, 12, [1500, 1, 0, 777]),             # split and joined
    (3, 8, 1, 128, 16, 70, [1100, 500, 1120]),
    (1, 2, 2, 240, 16, 60, [959]),
]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("S,H,KV,d,page,cols,lengths", OWN)
def test_own_tokens(K, S, H, KV, d, page, cols, lengths, kind):
    q, c, table, _ = _setup(K, S, H, KV, d, page, cols, 0, kind)
    _check(K, q, c, table, lengths)


SHARED = [  # S, H, KV, d, page, cols, pcols, lengths (high), prefix
    (1, 1, 1, 16, 16, 1, 1, 1, 1),
    (2, 4, 4, 128, 16, 2, 3, 20, 48),
    (5, 6, 2, 64, 16, 3, 9, 40, 130),                       # 15 rows
    (4, 16, 4, 128, 16, 2, 63, 30, 1000),                   # 16
    (17, 2, 2, 128, 32, 1, 11, 32, 345),                    # 17
    (8, 32, 8, 80, 16, 4, 20, 60, 311),                     # 32
    (11, 9, 3, 96, 16, 2, 33, 17, 513),                     # 33
    (16, 8, 2, 128, 64, 2, 10, 100, 600),                   # 64
    (43, 6, 2, 64, 16, 1, 30, 16, 465),                     # 129
    (32, 16, 4, 128, 16, 3, 65, 48, 1030),                  # 128
    (65, 4, 1, 128, 128, 1, 9, 128, 1100),                  # 260
    (20, 8, 1, 256, 16, 2, 20, 31, 300),                    # 160 rows, heads of 256
    (12, 40, 2, 112, 16, 1, 40, 9, 640),                    # 240, twenty heads to one
    (3, 20, 1, 240, 32, 2, 30, 50, 950),
    (130, 4, 2, 64, 16, 48, 10, 700, 150),                  # long own lengths of many sequences: joined where they end
    (17, 12, 2, 64, 16, 64, 12, 1000, 190),                 # of few: cut, and joined by themselves
]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("S,H,KV,d,page,cols,pcols,high,prefix", SHARED)
def test_shared_prefix(K, S, H, KV, d, page, cols, pcols, high, prefix, kind):
    q, c, table, ptable = _setup(K, S, H, KV, d, page, cols, pcols, kind, seed=S)
    lengths = [high * i // max(S - 1, 1) for i in range(S)]
    _check(K, q, c, table, lengths, ptable, prefix)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("S", [3, 40])
def test_lengths_of_zero_and_beyond(K, S, kind):
    """No prefix, no own tokens, neither, lengths and tables that make no sense."""
    q, c, table, ptable = _setup(K, S, 4, 2, 64, 16, 2, 6, kind)
    own = [(7 * i) % 33 for i in range(S)]
    _check(K, q, c, table, own, ptable, 0)
    _check(K, q, c, table, own, ptable[:0], 0)
    _check(K, q, c, table, [0] * S, ptable, 90)
    _check(K, q, c, table, [0] * S, ptable, 0)
    _check(K, q, c, table[:, :0], [5] * S, ptable, 33)
    _check(K, q, c, table[:, :0], [5] * S, ptable[:0], 3)
    _check(K, q, c, table, [-5, 1000] + own[2:], ptable, 2 ** 31 - 1)
    _check(K, q, c, table, own, ptable, -1)
    # the prefix alone is what its tokens are as own ones
    alone = K.qlora_prefix_attention(q, c, ptable, _i32([90]), table, _i32([0] * S))
    same = K.qlora_kv_attention(q, c, ptable[None].repeat(S, 1), _i32([90] * S))
    assert (alone.float() - same.float()).abs().max() <= 2.0 ** -7 * same.float().abs().max()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("S", [2, 40])
def test_pages_that_are_none(K, S, kind):
    """Tokens of pages outside the cache take no part, also inside a tile."""
    q, c, table, ptable = _setup(K, S, 4, 2, 64, 16, 3, 12, kind)
    pages = c.k.shape[0]
    table[0, 1], table[1, 0], table[1, 1], table[1, 2] = -1, pages, 2 ** 31 - 1, -2 ** 31
    ptable[0], ptable[3], ptable[4], ptable[5], ptable[11] = -1, pages, -7, 2 ** 31 - 1, pages + 5
    _check(K, q, c, table, [48] * S, ptable, 12 * 16)
    _check(K, q, c, table, [41] * S, ptable, 100)
    _check(K, q, c, table, [48] * S)
    ptable.fill_(-1)
    table.fill_(pages)
    _check(K, q, c, table, [48] * S, ptable, 12 * 16)     # nothing is left


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("S", [2, 40])
def test_what_lies_behind_a_length_is_not_used(K, S, kind):
    """NaN, infinities and codes that are no numbers behind the lengths, in the
    rest of the last pages and in pages of nobody."""
    q, c, table, ptable = _setup(K, S, 4, 2, 64, 16, 3, 5, kind)
    lengths, prefix = [17 + i % 20 for i in range(S)], 70
    before = K.qlora_prefix_attention(q, c, ptable, _i32([prefix]), table, _i32(lengths))
    live = np.zeros((c.k.shape[0], 16), bool)
    for row, n in [(ptable.tolist(), prefix)] + [(table[s].tolist(), lengths[s]) for s in range(S)]:
        for i in range(n):
            live[row[i // 16], i % 16] = True
    dead = torch.tensor(~live, device="cuda")[:, None, :]
    for t in (c.k, c.v):
        bad = dead[..., None].expand(t.shape)
        if kind == "bf16":
            t[bad] = math.inf
            t[..., ::2][bad[..., ::2]] = math.nan
        else:
            t.view(torch.uint8)[bad] = 0x7F          # no number in E4M3
    for t in (c.k_scale, c.v_scale):
        if t is not None:
            t[dead.expand(t.shape)] = math.nan
            t[:, 0][dead[:, 0]] = math.inf
    assert torch.equal(K.qlora_prefix_attention(q, c, ptable, _i32([prefix]), table, _i32(lengths)), before)
    assert torch.isfinite(K.qlora_kv_attention(q, c, table, _i32(lengths))).all()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("S", [2, 40])
def test_a_row_that_could_not_be_held_spoils_its_own_head(K, S, kind):
    q, c, table, ptable = _setup(K, S, 4, 2, 64, 16, 2, 5, kind)
    lengths = [20] * S
    before = K.qlora_prefix_attention(q, c, ptable, _i32([70]), table, _i32(lengths))
    c.v_scale[ptable[1], 0, 3] = math.nan
    got = K.qlora_prefix_attention(q, c, ptable, _i32([70]), table, _i32(lengths))
    assert torch.isnan(got[:, :2]).all() and torch.equal(got[:, 2:], before[:, 2:])
    c.v_scale[ptable[1], 0, 3] = 1.0
    c.k_scale[table[1, 0], 1, 2] = math.nan
    got = K.qlora_prefix_attention(q, c, ptable, _i32([70]), table, _i32(lengths))
    assert torch.isnan(got[1, 2:]).all() and torch.isfinite(got[0]).all() and torch.isfinite(got[1, :2]).all()


@pytest.mark.parametrize("S", [2, 40])
def test_an_infinity_among_the_values_stays_one(K, S):
    q, c, table, ptable = _setup(K, S, 4, 2, 64, 16, 2, 5, "bf16")
    c.v[ptable[2], 1, 5, 7] = math.inf
    c.v[ptable[0], 0, 1, 9] = -math.inf
    got = K.qlora_prefix_attention(q, c, ptable, _i32([70]), table, _i32([20] * S)).float()
    assert (got[:, 2:, 7] == math.inf).all() and (got[:, :2, 9] == -math.inf).all()
    got[:, 2:, 7], got[:, :2, 9] = 0, 0
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("S", [4, 48])
def test_scales_strides_and_given_outputs(K, S, kind):
    H, KV, d = 6, 2, 64
    q0, c, table, ptable = _setup(K, S, H, KV, d, 16, 2, 5, kind)
    wide = torch.zeros(S, 3 * H * d, dtype=BF, device="cuda")
    q = wide[:, 64:64 + H * d].unflatten(1, (H, d))
    q.copy_(q0)
    lengths, n = _i32([(5 * i) % 33 for i in range(S)]), _i32([77])
    for scale in (0.0, -0.3, 2.0, 30.0):
        _check(K, q, c, table, lengths.tolist(), ptable, 77, scale=scale)
    ref = K.qlora_prefix_attention(q0, c, ptable, n, table, lengths)
    out = torch.empty(S, H, d, dtype=BF, device="cuda")
    got = K.qlora_prefix_attention(q, c, ptable, n, table, lengths, out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, ref)
    assert K.qlora_prefix_attention(q[:0], c, ptable, n, table[:0], lengths[:0]).shape == (0, H, d)


@pytest.mark.parametrize("kind", list(KINDS))
def test_large_scores(K, kind):
    """Scores far beyond the range of the exponential: all weight on one token."""
    q, c, table, ptable = _setup(K, 40, 4, 2, 64, 16, 2, 8, kind)
    _check(K, q * 30, c, table, [20] * 40, ptable, 120, scale=1.0)
    _check(K, q[:2] * 30, c, table[:2], [20] * 2, ptable, 120, scale=1.0)


def test_offsets_beyond_32_bits(K):
    """Pages behind 2^31 elements of the cache, as own tokens and as a prefix."""
    KV, page, d = 2, 1024, 256
    pages = 2 ** 31 // (KV * page * d) + 3
    g = torch.Generator(device="cuda").manual_seed(1)
    for kind in ("int8", "bf16"):
        c = K.KVCache.zeros(pages, KV, page, d, KINDS[kind])
        small = _cache(K, 3, KV, page, d, kind, g)
        for big, few in zip(c, small):
            if big is not None:
                big[-3:] = few
        for S in (2, 40):
            q = torch.randn(S, 4, d, generator=g, device="cuda").to(BF)
            t, p = _i32([[1]] * S), _i32([2, 0])
            n, own = _i32([1500]), _i32([100] * S)
            ref = K.qlora_prefix_attention(q, small, p, n, t, own)
            assert torch.equal(K.qlora_prefix_attention(q, c, p + (pages - 3), n, t + (pages - 3), own), ref)
            ref = K.qlora_kv_attention(q, small, t, own)
            assert torch.equal(K.qlora_kv_attention(q, c, t + (pages - 3), own), ref)
        del c


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("S", [3, 40])
def test_graphs_and_streams(K, S, kind):
    """A captured write, read and attention replayed with other contents between
    eager calls; two streams at once."""
    H, KV, d = 4, 2, 64
    q, c, table, ptable = _setup(K, S, H, KV, d, 16, 3, 40, kind)
    k, v = torch.randn(S, KV, d, device="cuda").to(BF), torch.randn(S, KV, d, device="cuda").to(BF)
    own, n = _i32([20 + i % 20 for i in range(S)]), _i32([600])
    slots = torch.stack([table[s, (int(own[s]) - 1) // 16] * 16 + (int(own[s]) - 1) % 16 for s in range(S)]).to(torch.int32)

    def step():
        K.qlora_kv_write(None, k, v, None, None, slots, c)
        a = K.qlora_prefix_attention(q, c, ptable, n, table, own)
        return a, K.qlora_kv_attention(q, c, table, own), K.qlora_kv_read(c, slots)[0]
    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for i in range(4):
        q.copy_(torch.randn(S, H, d, device="cuda"))
        k.copy_(torch.randn(S, KV, d, device="cuda"))
        n.fill_(600 - 37 * i)
        graph.replay()
        got = [t.clone() for t in kept]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), i
    ref = step()[0]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for st in (side, torch.cuda.current_stream()):
            with torch.cuda.stream(st):
                outs.append(K.qlora_prefix_attention(q, c, ptable, n, table, own))
    outs.append(K.qlora_prefix_attention(q, c, ptable, n, table, own, stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_what_is_written_counts_as_changed(K):
    q, c, table, ptable = _setup(K, 2, 4, 2, 64, 16, 2, 5, "int8")
    before = [t._version for t in c]
    z = torch.zeros(2, 2, 64, dtype=BF, device="cuda")
    K.qlora_kv_write(None, z, z, None, None, _i32([0, 1]), c)
    assert all(t._version > b for t, b in zip(c, before))
    out, lse = torch.empty_like(q), torch.empty(2, 4, device="cuda")
    a, b, n = out._version, lse._version, [t._version for t in c]
    K.qlora_prefix_attention(q, c, ptable, _i32([9]), table, _i32([1, 2]), out=out, lse=lse)
    assert out._version > a and lse._version > b and [t._version for t in c] == n
