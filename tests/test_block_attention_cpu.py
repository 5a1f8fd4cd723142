"""block.causal_attention, the attention of prompts, on the CPU: rows in turns give
what all at once give, and never more scores than asked for."""
import math

import numpy as np
import pytest
import torch

from bit_nf4_quantized_quantize_amd import block


def _reference(q, k, v, heads, prefix):
    """The definition in fp64."""
    b, t, hd = q.shape
    d = hd // heads
    q, k, v = (z.double().numpy().reshape(b, t, heads, d) for z in (q, k, v))
    out = np.zeros((b, t, heads, d))
    for s in range(b):
        for h in range(heads):
            for i in range(t):
                kk, vv = k[s, :i + 1, h], v[s, :i + 1, h]
                if prefix is not None:
                    kk = np.concatenate((prefix[0][:, h].double().numpy(), kk))
                    vv = np.concatenate((prefix[1][:, h].double().numpy(), vv))
                w = kk @ q[s, i, h] / math.sqrt(d)
                w = np.exp(w - w.max())
                out[s, i, h] = w @ vv / w.sum()
    return out.reshape(b, t, hd)


@pytest.mark.parametrize("b,t,heads,d,prefix", [(1, 61, 2, 8, 0), (2, 33, 3, 16, 0), (2, 40, 2, 8, 77), (3, 1, 2, 8, 50),
                                                (1, 7, 1, 8, 400)])
@pytest.mark.parametrize("most", [2 ** 28, 11000, 1500, 1])
def test_rows_in_turns(b, t, heads, d, prefix, most, monkeypatch):
    monkeypatch.setattr(block, "MOST_SCORES", most, raising=False)
    g = torch.Generator().manual_seed(t)
    q, k, v = (torch.randn(b, t, heads * d, generator=g) for _ in "qkv")
    before = [torch.randn(prefix, heads, d, generator=g) for _ in "kv"] if prefix else None
    sizes, call = [0], torch.matmul
    monkeypatch.setattr(torch, "matmul", lambda x, y: sizes.append(call(x, y).numel()) or call(x, y))
    with torch.no_grad():
        got = block.causal_attention(q, k, v, heads, before).double().numpy()
    monkeypatch.setattr(torch, "matmul", call)
    # the outputs of the products are scores, and rows of d
    assert max(sizes) <= max(most, heads * max(t + prefix, b * t * d))
    want = _reference(q, k, v, heads, before)
    assert np.abs(got - want).max() <= 2.0 ** -24 * 4 * (d + t + prefix + 32) * max(1.0, np.abs(want).max())
    if most == 2 ** 28:      # and the form that gradients go through
        again = block.causal_attention(q, k, v, heads, before).double().numpy()
        assert np.array_equal(got, again)


def test_gradients_go_through_one_form(monkeypatch):
    monkeypatch.setattr(block, "MOST_SCORES", 1, raising=False)
    q, k, v = (torch.randn(2, 9, 16, generator=torch.Generator().manual_seed(i), requires_grad=True) for i in range(3))
    block.causal_attention(q, k, v, 2).square().sum().backward()
    assert all(torch.isfinite(z.grad).all() and z.grad.abs().sum() > 0 for z in (q, k, v))
