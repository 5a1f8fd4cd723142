"""GPU parity of the paged attention's workgroups of eight waves, which calls of
large capacity take, against fp64: one part per sequence and several, every head
size class, ragged lengths from 0, a missing page, and NaN and infinities behind
the lengths.

Tolerance: a score is a sum of d exact bfloat16 products in fp32 and is off by
e <= (d + 16) u scale sum_i |q_i| max|k| (u = 2^-24; 16 for the product with the
scale in base 2, the exponent's own rounding and the exponential), so a weight by a
relative 2 e, the running maxima's factors among it; a sum of n weighted values
adds n + 256 roundings (with those of the joins), and the output is rounded once:
    |err| <= (2 e + (n + 256) u) sum_i p_i |v_i| + 2^-8 |out|."""

import ctypes
import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = torch.bfloat16


@pytest.fixture(scope="module")
def D():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_quantize_amd import decoder
    decoder.lib()
    return decoder


def _eight_waves(S, H, KV, d, page, cols):
    """The rule of the launcher: 128 tiles of 32 tokens per CU, heads up to 128."""
    return S * KV * -(-H // KV // 16) * -(-cols * page // 32) >= 128 * 256 and d <= 128


def _reference(q, kc, vc, table, n, scale):
    """(out, lse, weight) [H, d] of one sequence in fp64; table: its row on the host."""
    H, d = q.shape
    pages, KV, page, _ = kc.shape
    at = [(p, i) for p, i in ((int(table[i // page]), i % page) for i in range(n)) if 0 <= p < pages]
    if not at:
        z = torch.zeros(H, d, dtype=torch.float64, device="cuda")
        return z, torch.full((H,), -math.inf, dtype=torch.float64, device="cuda"), z
    p, o = (torch.tensor(c, device="cuda") for c in zip(*at))
    out, lse, wt = [], [], []
    for j in range(KV):
        k, v = kc[p, j, o].double(), vc[p, j, o].double()
        s = scale * (q[j * (H // KV):(j + 1) * (H // KV)].double() @ k.t().contiguous())
        w = torch.softmax(s, -1)
        out.append(w @ v)
        wt.append(w @ v.abs())
        lse.append(torch.logsumexp(s, -1))
    return torch.cat(out), torch.cat(lse), torch.cat(wt)


CASES = [  # q heads, kv heads, head_dim, page, columns, lengths; one part per sequence, then several
    (16, 16, 64, 16, 64, [0, 1, 1024, 15, 16, 17, 31, 32, 33, 1023] + [i * 16 + i for i in range(54)], 1),
    (32, 32, 80, 32, 40, [1280, 0, 1, 255, 256, 257, 1279] + [41 * i for i in range(25)], 1),
    (64, 16, 128, 64, 16, [1024, 1, 0, 64, 63, 65, 512, 513] + [16 * i + 3 for i in range(56)], 1),
    (1024, 64, 96, 16, 65, [1040, 0, 1, 511, 1039, 700, 64, 65, 33, 2, 900, 128, 129, 130, 131, 132], 1),
    (64, 8, 128, 16, 1100, [17600, 0, 1, 512, 513, 9000, 4111, 31], 2),
    (136, 8, 64, 64, 256, [16384, 70, 0, 3001], 2),
    (4, 4, 96, 64, 1400, [89600, 1, 0], 2),
    (8, 8, 40, 128, 130, [16640, 600, 0, 12345, 1, 127, 128, 129], 2),
]


@pytest.mark.parametrize("H,KV,d,page,cols,lengths,parts", CASES)
def test_eight_waves(D, H, KV, d, page, cols, lengths, parts):
    S = len(lengths)
    print(f"paged attention, eight waves: S={S} H={H} KV={KV} d={d} page={page} capacity={cols * page}", flush=True)
    sys.stdout.flush()
    assert _eight_waves(S, H, KV, d, page, cols)
    ws = ctypes.c_int64()
    assert D.lib().qlora_paged_attention_workspace(S, H, KV, d, cols, page, ctypes.byref(ws)) == 0
    assert (ws.value > 0) == (parts > 1)
    g = torch.Generator(device="cuda").manual_seed(d * S)
    # pages 0 .. full - 1 are anybody's, full + s is the last page of sequence s, the one behind is spoilt
    full = 96
    pages = full + S + 1
    q = torch.randn(S, H, d, generator=g, device="cuda").to(BF)
    kc, vc = (torch.randn(pages, KV, page, d, generator=g, device="cuda").to(BF) for _ in range(2))
    table = torch.randint(0, full, (S, cols), generator=g, device="cuda").cpu()
    kmax = float(kc.abs().max())
    kc[-1], vc[-1] = float("nan"), float("inf")
    missing = max(range(S), key=lambda s: lengths[s])
    for s, n in enumerate(lengths):
        used = -(-n // page)
        table[s, used:] = pages - 1 if s % 2 else 2 ** 31 - 1
        if used:
            table[s, used - 1] = full + s
            kc[full + s, :, (n - 1) % page + 1:] = float("nan")
            vc[full + s, :, (n - 1) % page + 1:] = float("-inf")
    table[missing, lengths[missing] // page // 2] = -1
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    lse = torch.empty(S, H, device="cuda")
    dev = table.to(torch.int32).cuda()
    out = D.qlora_paged_attention(q, kc, vc, dev, lens, lse=lse)
    scale = 1 / math.sqrt(d)
    for s, n in enumerate(lengths):
        ref, rl, wt = _reference(q[s], kc, vc, table[s].tolist(), n, scale)
        e = (d + 16) * U * scale * q[s].double().abs().sum(-1, keepdim=True) * kmax
        err = (out[s].double() - ref).abs()
        assert (err <= (2 * e + (n + 256) * U) * wt + 2.0 ** -8 * ref.abs()).all(), (s, n, float(err.max()))
        if n == 0:
            assert not out[s].any() and torch.equal(lse[s].double(), rl)
        else:
            assert ((lse[s].double() - rl).abs() <= 2 * e[:, 0] + (n + 256) * U + 4 * U * rl.abs()).all(), (s, n)
    again = D.qlora_paged_attention(q, kc, vc, dev, lens)
    assert torch.equal(again, out)


def test_lengths_beyond_the_table(D):
    """Cut to the table, in calls of eight waves too."""
    H = KV = 16
    S, d, page, cols = 64, 64, 16, 64
    assert _eight_waves(S, H, KV, d, page, cols)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(S, H, d, generator=g, device="cuda").to(BF)
    kc, vc = (torch.randn(50, KV, page, d, generator=g, device="cuda").to(BF) for _ in range(2))
    table = torch.randint(0, 50, (S, cols), generator=g, device="cuda").to(torch.int32)
    lens = torch.full((S,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    lens[1], lens[2] = -1, -2 ** 31
    cut = lens.clamp(0, cols * page)
    a, b = (D.qlora_paged_attention(q, kc, vc, table, n) for n in (lens, cut))
    assert torch.equal(a, b) and not a[1].any() and not a[2].any() and a[0].any()
