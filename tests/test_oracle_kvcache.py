"""Pins of the oracle of the 8-bit and the shared key-value cache."""

import numpy as np
import pytest
import torch

from oracle import decoder as od
from oracle import kvcache as ok


def test_e4m3_sizes_are_the_formats():
    bits = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ok.E4M3, bits)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_nearest_code(kind):
    """Against all codes by distance; ties go to the even one."""
    codes = np.arange(128.0) if kind == "int8" else ok.E4M3
    rng = np.random.default_rng(3)
    y = np.concatenate([rng.uniform(-ok.MOST[kind], ok.MOST[kind], 2000), (codes[1:] + codes[:-1]) / 2, codes, -codes])
    got = ok.nearest(y, kind)
    dist = np.abs(np.abs(y)[:, None] - codes[None])
    assert np.array_equal(np.abs(np.abs(y) - np.abs(got)), dist.min(1))
    tie = np.sort(dist, 1)[:, 0] == np.sort(dist, 1)[:, 1]
    assert tie.any() and (np.searchsorted(codes, np.abs(got[tie])) % 2 == 0).all()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_rows(kind):
    z = np.random.default_rng(4).normal(size=(5, 64)).astype(np.float32)
    z[1] = 0
    z[2, 3], z[3, 4] = np.nan, -np.inf
    codes, scale = ok.encode(z, kind)
    assert np.isnan(scale[2:4]).all() and not codes[2:4].any() and scale[1] == 0 and not codes[1].any()
    good = [0, 4]
    err = np.abs(ok.values(codes, scale)[good] - z[good])
    assert (err <= ok.half_step(codes[good], kind) * scale[good, None] * (1 + 2.0 ** -22)).all()
    assert (np.abs(codes[good]).max(-1) == ok.MOST[kind]).all()


def test_a_prefix_is_tokens_before_the_own():
    """Prefix and own tokens together are one sequence of the paged attention."""
    rng = np.random.default_rng(5)
    q, k, v = rng.normal(size=(2, 4, 16)), rng.normal(size=(6, 2, 4, 16)), rng.normal(size=(6, 2, 4, 16))
    got = ok.attention(q, k, v, np.array([[0, 1], [4, -1]]), [5, 0], 0.25, [2, 5], 8)
    ref = od.paged_attention(q, k, v, np.array([[2, 5, 0, 1], [2, 5, 0, 0]]), [13, 8], 0.25)
    for a, b in zip(got, ref):
        assert np.allclose(a, b, atol=1e-14)
