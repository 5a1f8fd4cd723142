"""GPU parity of the paged attention where single weights and values show: what
a weight carries into the product with V, against exact arithmetic in fp64."""

import sys

import pytest
import torch

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


def _three_tokens(delta):
    """Caches of len(delta) sequences of three tokens in a page of 16, one head of
    8: scores 0, 0 and -delta (a single product each), and values c1, c2, -1
    in the first column with c1 + c2 the two bfloat16 numbers next to the weight
    w = exp(-delta), so that out = (c1 + c2 - w) / (2 + w).  Returns (q, k_cache,
    v_cache, table, lengths, w, out) with w and out in fp64."""
    S = delta.numel()
    w = torch.exp(-delta.double())
    c1 = w.to(BF)
    c2 = (w - c1.double()).to(BF)
    q = torch.zeros(S, 1, 8, dtype=BF, device="cuda")
    q[:, 0, 0] = 1
    kc = torch.zeros(S, 1, 16, 8, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    kc[:, 0, 2, 0] = -delta
    vc[:, 0, 0, 0], vc[:, 0, 1, 0], vc[:, 0, 2, 0] = c1, c2, -1
    table = torch.arange(S, dtype=torch.int32, device="cuda").view(S, 1)
    lens = torch.full((S,), 3, dtype=torch.int32, device="cuda")
    return q, kc, vc, table, lens, w, (c1.double() + c2.double() - w) / (2 + w)


def test_a_weight_enters_the_product_with_all_its_bits(D):
    """The scores are exact.  Their product with the fp32 factor log2(e) is off by 2
    u |score| <= 2 u, the exponential by 2 u (1 ulp): the weight by 4 u w.  The
    first two tokens' weights are 1.  The sum of c1, c2 and the weight's parts takes
    six additions of numbers below 1, 2 u each at most; the division and the
    rounding of the output are relative to the result.  So
        |err| <= (4 + 12) u / (2 + w) + 2^-8 |out|,
    where a weight cut to 16 bits is off by up to 64 u / (2 + w)."""
    _log("paged attention: the bits of a weight")
    delta = (torch.arange(1, 2049, device="cuda") / 2048.0).to(BF).unique()
    q, kc, vc, table, lens, w, ref = _three_tokens(delta)
    out = D.qlora_paged_attention(q, kc, vc, table, lens, scale=1.0)[:, 0].double()
    assert not out[:, 1:].any()
    assert ref.abs().max() > 20 * U            # the case is what it says: bits behind the 16th show
    assert ((out[:, 0] - ref).abs() <= 16 * U / (2 + w) + 2.0 ** -8 * ref.abs()).all()


@pytest.mark.parametrize("S,H,KV,d,page,lengths", [
    (3, 4, 2, 64, 16, [40, 1, 300]), (2, 8, 8, 128, 32, [70, 900]), (1, 34, 2, 80, 16, [1500]), (2, 2, 1, 256, 64, [33, 700])])
def test_infinities_among_the_attended_values(D, S, H, KV, d, page, lengths):
    """A column of V with infinities of one sign gives that infinity, with both
    signs or a NaN gives NaN; the other columns, heads and sequences are, bit for
    bit, what they were.  The scores are small (|q . k| / sqrt(d) below 10), so no
    weight is zero."""
    _log(f"paged attention: infinities S={S} H={H} KV={KV} d={d} lengths={lengths}")
    g = torch.Generator(device="cuda").manual_seed(d)
    cols = -(-max(lengths) // page)
    pages = S * cols
    q = torch.randn(S, H, d, generator=g, device="cuda").to(BF)
    kc, vc = (torch.randn(pages, KV, page, d, generator=g, device="cuda").to(BF) for _ in range(2))
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(S, cols)
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    lse = torch.empty(S, H, device="cuda")
    want = D.qlora_paged_attention(q, kc, vc, table, lens, lse=lse).clone()
    want_lse = lse.clone()
    inf, nan, G = float("inf"), float("nan"), H // KV
    for s, n in enumerate(lengths):
        j = s % KV
        for c, (at, value) in enumerate([(0, inf), (n - 1, -inf), (n // 2, inf), (n // 3, nan)]):
            vc[int(table[s, at // page]), j, at % page, 2 * c] = value
            want[s, j * G:(j + 1) * G, 2 * c] = value
        if n > 2:
            vc[int(table[s, (n - 1) // page]), j, (n - 1) % page, 4] = inf    # a second one, of the same sign
            c = d - 1                                                       # both signs
            vc[int(table[s, 0]), j, 0, c], vc[int(table[s, 1 // page]), j, 1, c] = inf, -inf
            want[s, j * G:(j + 1) * G, c] = nan
    got = D.qlora_paged_attention(q, kc, vc, table, lens, lse=lse)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[~got.isnan()], want[~want.isnan()])
    assert torch.equal(lse, want_lse)


@pytest.mark.parametrize("which", ["q", "k"])
def test_a_nan_score_spoils_its_own_heads_only(D, which):
    """A NaN in a query gives that head NaN, one in an attended key the heads of its
    kv head in its sequence; the rest is, bit for bit, what it was."""
    _log(f"paged attention: NaN in {which}")
    g = torch.Generator(device="cuda").manual_seed(5)
    S, H, KV, d, page, cols = 3, 8, 2, 64, 16, 50
    q = torch.randn(S, H, d, generator=g, device="cuda").to(BF)
    kc, vc = (torch.randn(S * cols, KV, page, d, generator=g, device="cuda").to(BF) for _ in range(2))
    table = torch.randperm(S * cols, generator=g, device="cuda").to(torch.int32).view(S, cols)
    lens = torch.tensor([700, 5, 33], dtype=torch.int32, device="cuda")
    lse = torch.empty(S, H, device="cuda")
    want, want_lse = D.qlora_paged_attention(q, kc, vc, table, lens, lse=lse), lse.clone()
    spoilt = torch.zeros(S, H, dtype=torch.bool, device="cuda")
    for s, at in ((0, 650), (2, 0)):
        if which == "q":
            q[s, 3, 7] = float("nan")
            spoilt[s, 3] = True
        else:
            kc[int(table[s, at // page]), 1, at % page, 9] = float("nan")
            spoilt[s, H // KV:] = True
    got = D.qlora_paged_attention(q, kc, vc, table, lens, lse=lse)
    assert got[spoilt].isnan().all() and lse[spoilt].isnan().all()
    assert torch.equal(got[~spoilt], want[~spoilt]) and torch.equal(lse[~spoilt], want_lse[~spoilt])
