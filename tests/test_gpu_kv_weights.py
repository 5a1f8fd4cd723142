"""What a weight of the attention over a paged cache keeps, for every kernel that
may take a row: one sequence's own tokens, a prefix behind few rows and behind
many.  Values are made to cancel, so that the rounding of the output hides
nothing."""
import math

import pytest
import torch

from test_gpu_kv_attention import BF, KINDS, U, _i32

pytestmark = pytest.mark.gpu

PATHS = ["own", "few", "many"]


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_quantize_amd import kvcache
    kvcache.native()
    return kvcache


def _attend(K, path, q, cache, n, scale=None, lse=None):
    """q [S, H, d] over tokens 0 .. n - 1 of the cache's pages in order. More than 32
    rows of a kv head and a table with room for more than 2^18 tokens times kv
    heads times tiles of 16 rows: the kernels for many rows."""
    S, H, _ = q.shape
    pages, KV, page, _ = cache.k.shape
    table, none = torch.arange(pages, dtype=torch.int32, device="cuda"), _i32([[0]] * S)
    if path == "own":
        return K.qlora_kv_attention(q, cache, table[None].repeat(S, 1), _i32([n] * S), scale=scale, lse=lse)
    if path == "many":
        assert S * H // KV > 32
        room = 2 ** 18 // (-(-S * H // (16 * KV)) * KV * page) + 1
        table = torch.cat((table, table.new_full((max(0, room - pages),), -1)))
    return K.qlora_prefix_attention(q, cache, table, _i32([n]), none, _i32([0] * S), scale=scale, lse=lse)


def _sequences(path, S):
    return 8 if path == "few" else S


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("path", PATHS)
def test_scales_enter_with_all_their_bits(K, path, kind):
    """Two tokens of equal scores, values a and -b with scales of 24 bits: weights of
    one, so every product is exact and (a - b) / 2 is the result before its rounding."""
    KV, d, S = 8, 16, _sequences(path, 12)
    c = K.KVCache.zeros(1, KV, 16, d, KINDS[kind])
    g = torch.Generator().manual_seed(3)
    a, b = ((1 + torch.randint(0, 2 ** 23, (KV,), generator=g).double() * 2.0 ** -23) for _ in "ab")
    a[0], b[0] = 1 + 2.0 ** -8 + 2.0 ** -16, 1 + 2.0 ** -8
    a[1], b[1] = 1 + 2.0 ** -8 + 2.0 ** -16 + 2.0 ** -23, 1 + 2.0 ** -8 + 2.0 ** -16
    b[2:5] = a[2:5] - torch.tensor([2.0 ** -23, 2.0 ** -18, 2.0 ** -15])
    c.v[0, :, 0], c.v[0, :, 1] = torch.ones(KV, d).to(KINDS[kind]).cuda(), (-torch.ones(KV, d)).to(KINDS[kind]).cuda()
    c.v_scale[0, :, 0], c.v_scale[0, :, 1] = a.float().cuda(), b.float().cuda()
    got = _attend(K, path, torch.zeros(S, 4 * KV, d, dtype=BF, device="cuda"), c, 2)
    want = ((a - b) / 2).to(BF).cuda().repeat_interleave(4)[None, :, None].expand(got.shape)
    assert torch.equal(got, want)


@pytest.mark.parametrize("path", PATHS)
def test_weights_enter_with_all_their_bits(K, path):
    """A token of weight p = exp(s) with value 1, and three of weight 1 whose values are
    the bfloat16 parts of -p, other ones in the column of each row: nothing is left.
    The score and its exponential are off by 2 u and 2 u of p, the sums of at most
    eight numbers under 2 by 2 u each: 20 u in all, with twice that for the order of
    the additions within the products, 40 u; two parts of a weight leave up to 128 u."""
    S, H, d = _sequences(path, 32), 4, 128
    s = -(torch.arange(128).double() * 37 % 128 + 1) / 256 * 1.375     # four bits or so of -0.005 to -0.69
    s = s.to(BF)
    p, rows = torch.exp(s.double()), S * H
    c = K.KVCache.zeros(1, 1, 16, d)
    c.k[0, 0, 0, 0], c.v[0, 0, 0] = 1.0, 1.0
    left = -p
    for t in (1, 2, 3):
        part = left.to(BF)
        c.v[0, 0, t] = part.cuda()
        left = left - part.double()
    assert left.abs().max() < U / 2
    q = torch.zeros(rows, d, dtype=BF)
    q[:, 0] = s[:rows]
    out = _attend(K, path, q.view(S, H, d).cuda(), c, 4, scale=1.0).double().cpu().view(rows, d)
    off = out[torch.arange(rows), torch.arange(rows)].abs() * (p[:rows] + 3)
    assert (off <= 40 * U).all(), float(off.max() / U)
    # and not because nothing is read: another row's column holds what the values there make
    want = (p[:rows, None] - p[None, :]) / (p[:rows, None] + 3)
    assert ((out - want).abs() <= 2.0 ** -8 * want.abs() + 40 * U).all()
    assert math.isfinite(float(out.abs().max())) and float(out.abs().max()) > 0.05


@pytest.mark.parametrize("size", [1.5 * 2.0 ** 126, 1.0, 2.0 ** -95])
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("path,S,d", [("own", 3, 64), ("few", 8, 64), ("many", 12, 64), ("many", 70, 128), ("many", 12, 256)])
def test_values_of_any_size(K, path, S, d, kind, size):
    """A token late in the line weighs 2^7 times as much as those before it: its weight
    times its value must not pass the largest number on the way, nor lose bits below
    the smallest normal one.  Weights are off by 16 u, the 128 sums by 2 u each; the
    output is rounded by 2^-8 at most."""
    n, late = 128, 69
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.zeros(n, 1, d, dtype=BF, device="cuda")
    k[late, 0, 0] = 7.0
    v = torch.randn(n, 1, d, generator=g, device="cuda") * 2.0 ** -9
    v[late] = torch.where(v[late] < 0, -1.0, 1.0)
    v = (v.double() * size).to(BF)
    c = K.KVCache.zeros(n // 16, 1, 16, d, KINDS[kind])
    K.qlora_kv_write(None, k, v, None, None, torch.arange(n, dtype=torch.int32, device="cuda"), c)
    q = torch.zeros(S, 4, d, dtype=BF, device="cuda")
    q[..., 0] = 1.0
    got = _attend(K, path, q, c, n, scale=math.log(2.0)).double()
    values = c.v.double() if kind == "bf16" else c.v.float().double() * c.v_scale.double()[..., None]
    values = values[:, 0].reshape(n, d)
    p = torch.ones(n, dtype=torch.float64, device="cuda")
    p[late] = 2.0 ** 7
    want, wt = p @ values / p.sum(), p @ values.abs() / p.sum()
    assert torch.isfinite(want).all() and (want.abs() > 0.4 * size).all()
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 272 * U * wt).all()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("path", PATHS)
def test_scales_of_either_sign(K, path, kind):
    """A row's numbers are code times scale, also for a scale of -0 or below it, and
    for a weight of 0.  Tolerance: a score's products and their sum are off by 2 (d + 8)
    u of their sizes' sum, the weight by that and 16 u more, 48 sums by 2 u each; the
    output is rounded by 2^-8.  A weight under 2^-126 of the largest is no normal fp32
    number and may count as nothing: where one token has all the weight and a value of
    0 the result is made of such ones alone."""
    n, KV, d, S = 48, 2, 64, _sequences(path, 20)
    g = torch.Generator(device="cuda").manual_seed(6)
    c = K.KVCache.zeros(n // 16, KV, 16, d, KINDS[kind])
    z = [torch.randn(n, KV, d, generator=g, device="cuda").to(BF) for _ in "kv"]
    K.qlora_kv_write(None, *z, None, None, torch.arange(n, dtype=torch.int32, device="cuda"), c)
    for t in (c.k_scale, c.v_scale):
        t[:, :, 3::5] *= -1.0
    c.v_scale[:, :, 4::6], c.k_scale[1, :, 2] = -0.0, -0.0
    c.k_scale[2, 0, 5] *= 400.0           # one token takes all of a row's weight, or none of it
    q = torch.randn(S, 4, d, generator=g, device="cuda").to(BF)
    got = _attend(K, path, q, c, n).double()
    k, v = ((t.float().double() * s.double()[..., None]).transpose(1, 2).reshape(n, KV, d)
            for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
    for h in range(4):
        score = q[:, h].double() @ k[:, h // 2].t().contiguous() / math.sqrt(d)
        p = torch.softmax(score, -1)
        want, wt = p @ v[:, h // 2], p @ v[:, h // 2].abs()
        size = (q[:, h].double().abs() @ k[:, h // 2].abs().t().contiguous()).amax(-1, keepdim=True) / math.sqrt(d)
        e = (2 * (d + 8) + 16) * U * (1 + size)
        assert ((got[:, h] - want).abs() <= 2.0 ** -8 * want.abs() + (2 * e + 112 * U) * wt +
                n * 2.0 ** -126 * float(v.abs().max())).all(), h
    assert (q[:, 0].double() @ k[:, 0].t().contiguous()).abs().max() / 8 > 100
