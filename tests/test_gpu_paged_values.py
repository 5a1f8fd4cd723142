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
