"""The attention of QLoraBlock.decode against a plain one over the numbers that its
cache holds (in 8 bits far from the keys and values that were written, so a forward
over those says little), and the block's output with either.  Both attentions are
rounded to bfloat16, by 2^-9 at most each, and their rotated queries are the same but
where the two round to other neighbours, which moves a score by 2^-8 of one of its
products: 2^-7 in all.  The output differs by that in one of its three parts and by
the rounding of the two linears behind it, 2^-8 each.

The plain attention, on the CPU, takes mistakes on request; each has to show."""
import math

import pytest
import torch

from test_gpu_block_kv import BL, D_HEAD, HEADS, HIDDEN, KINDS, _block, _rel, _x  # noqa: F401

pytestmark = pytest.mark.gpu

TOL, TOL_OUT = 2.0 ** -7, 4 * 2.0 ** -8


def _turned(q, position, rot, inter):
    """q [sequences, heads, d] at one position, fp64, rounded to bfloat16."""
    if rot is None:
        return q
    f = position * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    c, s, z = f.cos(), f.sin(), q.double().clone()
    a, b = (z[..., 0:rot:2].clone(), z[..., 1:rot:2].clone()) if inter else (z[..., :rot // 2].clone(), z[..., rot // 2:rot].clone())
    if inter:
        z[..., 0:rot:2], z[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        z[..., :rot // 2], z[..., rot // 2:rot] = a * c - b * s, a * s + b * c
    return z.to(torch.bfloat16)


def _plain(q, position, prefix, own, rot, inter, mistake=None):
    """Attention of one token per sequence over the prefix's rows [tokens, heads, d] and
    its own [sequences, tokens, heads, d]; all on the CPU."""
    S, n = q.shape[0], prefix[0].shape[0]
    q = _turned(q, position - (n if mistake == "no offset" else 0), rot, inter).double()
    k, v = (torch.cat((p.expand(S, -1, -1, -1), o), 1).double() for p, o in zip(prefix, own))
    score = torch.einsum("shd,snhd->shn", q, k) / math.sqrt(D_HEAD)
    if mistake == "no prefix":
        score[..., :n] = -math.inf
    if mistake == "one token less":
        score[..., -1] = -math.inf
    if mistake == "even weights":
        score.zero_()
    if mistake == "other heads":
        v = v.roll(1, 2)
    return torch.einsum("shn,snhd->shd", score.softmax(-1), v).reshape(S, HIDDEN).to(torch.bfloat16)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("rot,inter,seqs,prefix,prompt,more", [
    (64, False, 3, 37, 5, 6), (32, True, 40, 70, 3, 4), (None, False, 2, 16, 0, 6),
])
def test_decode_is_attention_over_what_the_cache_holds(BL, kind, rot, inter, seqs, prefix, prompt, more):  # noqa: F811
    from bit_nf4_quantized_quantize_amd import qlora_kv_read
    blk = _block(BL, rot, inter)
    shared, own = _x(prefix, seed=1), _x(seqs, prompt + more, seed=2)
    cache = blk.cache(num_pages=8 + seqs * 3, page_size=16, max_seqs=seqs, max_len=48, dtype=KINDS[kind], max_prefix=80)
    blk.prefill_shared(shared, cache)
    if prompt:
        blk.prefill(own[:, :prompt].contiguous(), cache)
    before = [z.cpu() for z in qlora_kv_read(cache.rows, cache.prefix_slots, dtype=torch.float32)]
    seen, fused, least = {}, blk._fused, {}

    def recorded(x, attend):
        def kept(q, k, v):
            seen["q"], seen["k"], seen["o"] = q.cpu(), k.cpu(), attend(q, k, v)
            return seen["o"]
        return fused(x, kept)

    for i in range(prompt, prompt + more):
        x = own[:, i].contiguous()
        blk._fused = recorded
        got = blk.decode(x, cache)
        blk._fused = fused
        t = torch.arange(i + 1, device="cuda")
        slots = (cache.table[:, t // 16] * 16 + t % 16).to(torch.int32).flatten()
        mine = [z.view(seqs, i + 1, HEADS, D_HEAD).cpu() for z in qlora_kv_read(cache.rows, slots, dtype=torch.float32)]
        o, want = seen["o"].cpu().float(), _plain(seen["q"], prefix + i, before, mine, rot, inter)
        assert o.shape == want.shape and _rel(o, want.float()) < TOL, i
        # the key it stored: half a step of codes off, and at its place behind the prefix
        key = _turned(seen["k"], prefix + i, rot, inter).float()
        assert _rel(mine[0][:, i], key) < 2.0 ** -4 + 2.0 ** -8, i
        if rot is not None:
            assert _rel(mine[0][:, i], _turned(seen["k"], i, rot, inter).float()) > 4 * 2.0 ** -4, i
        with torch.no_grad():
            assert _rel(got, fused(x, lambda q, k, v: want.cuda())) < TOL_OUT, i
        for m in ("no offset", "no prefix", "one token less", "even weights", "other heads"):
            if m != "no offset" or rot is not None:
                off = _plain(seen["q"], prefix + i, before, mine, rot, inter, m).float()
                least[m] = min(least.get(m, math.inf), _rel(off, want.float()))
    assert all(off > 4 * TOL for off in least.values()), least
