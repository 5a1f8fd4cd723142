"""GPU parity of rotary angles at far positions with ordinary frequencies, against
exact rational arithmetic on the table the call was given."""

import math
import sys
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FAR = [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 977, 2 ** 30 + 1, 1234567891, -2 ** 31, -2 ** 31 + 1, -1999999973, 16777217, 1, 0]


@pytest.fixture(scope="module")
def D():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_quantize_amd import decoder
    decoder.lib()
    return decoder


def _trig(position, turns):
    """cos and sin of 2 pi position turns: the whole turns are taken off exactly."""
    f = Fraction(position) * Fraction(turns)
    x = 2 * math.pi * float(f - round(f))
    return math.cos(x), math.sin(x)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("scaling", ["none", "yarn"])
def test_far_angles(D, scaling, inverse):
    """q = (1, 0) becomes (cos, sin), through no rounding but those of the cosine
    and sine themselves: the functions to 2 ulp (4 u of the value), the remainder of
    the angle in fp32 put back to first order (one rounding, u of the value, and
    terms of (2 pi 2^-25)^2 < 2^-44), the factor 1 or mscale (u):
        |err| <= 6 u |value| + 2^-44."""
    rot = 64
    tab = D.RopeTable(rot, scaling=scaling, factor=4.0 if scaling == "yarn" else 1.0, original_len=4096, device="cuda")
    print("far angles", scaling, inverse, flush=True)
    sys.stdout.flush()
    pos = torch.tensor(FAR, dtype=torch.int32, device="cuda")
    q = torch.zeros(len(FAR), 1, rot, device="cuda")
    q[..., :rot // 2] = 1
    out, _ = D.qlora_rope(q, None, tab, pos, inverse=inverse)
    turns, sign = tab.turns.tolist(), -1.0 if inverse else 1.0
    ref = np.array([[_trig(p, t) for t in turns] for p in FAR]) * tab.mscale   # [positions, pairs, 2]
    got = out[:, 0].double().cpu().numpy()
    for part, want in ((got[:, :rot // 2], ref[..., 0]), (got[:, rot // 2:], sign * ref[..., 1])):
        err = np.abs(part - want)
        assert (err <= 6 * U * np.abs(want) + 2.0 ** -44).all(), float((err / (U * np.abs(want) + 2.0 ** -60)).max())


def test_far_angles_into_the_cache(D):
    """The same from the form that writes the cache, in bfloat16: the value's own
    rounding, 2^-8, and the above."""
    rot, T = 64, len(FAR)
    tab = D.RopeTable(rot, interleaved=True, device="cuda")
    pos = torch.tensor(FAR, dtype=torch.int32, device="cuda")
    k = torch.zeros(T, 1, rot, dtype=torch.bfloat16, device="cuda")
    k[..., ::2] = 1
    kc = torch.zeros(1, 1, 16, rot, dtype=torch.bfloat16, device="cuda")
    D.qlora_rope_cache_write(None, k, k, tab, pos, torch.arange(T, dtype=torch.int32, device="cuda"), kc, kc.clone())
    ref = np.array([[_trig(p, t) for t in tab.turns.tolist()] for p in FAR]).reshape(T, rot)
    err = np.abs(kc[0, 0, :T].double().cpu().numpy() - ref)
    assert (err <= (2.0 ** -8 + 8 * U) * np.abs(ref) + 2.0 ** -44).all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("scaling", ["none", "yarn"])
def test_cosines_and_sines_are_rounded_once(D, scaling, inter):
    """Through q = (1, 0), in float32: the fp64 value times mscale, in one rounding of
    u of the value at most.  The fp64 functions and product add 2^-50 of it, the
    angle 2^-52."""
    print("trig", scaling, inter, flush=True)
    rot, T = 128, 500
    tab = D.RopeTable(rot, scaling=scaling, factor=16.0 if scaling == "yarn" else 1.0, original_len=4096,
                      interleaved=inter, device="cuda")
    pos = (torch.arange(T, device="cuda") * 777 - 1000).to(torch.int32)
    q = torch.zeros(T, 1, rot, device="cuda")
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    q[..., a] = 1
    out, _ = D.qlora_rope(q, None, tab, pos)
    ref = np.array([[_trig(p, t) for t in tab.turns.tolist()] for p in pos.tolist()]) * tab.mscale
    got = out[:, 0].double().cpu().numpy()
    for part, want in ((got[:, a], ref[..., 0]), (got[:, b], ref[..., 1])):
        assert (np.abs(part - want) <= U * (1 + 2.0 ** -20) * np.abs(want) + 2.0 ** -48).all()
