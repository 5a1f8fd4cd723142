"""GPU parity of the 8-bit key-value cache: rows written and read back, against
the fp64 oracle.

Values are held as they come, so their codes and scales are the oracle's bit for
bit.  A rotated key is off by the roundings of its cosine, sine, two products and
sum, r = 4 u m (|a| + |b|) (u = 2^-24, m the table's factor), its scale by that of
the row's largest and its own rounding, so the number held is within half a step
of codes, taken at the scale, plus 2 r + 2^-22 of its size.  Reading back rounds
code * scale once: to fp32 by u, to bfloat16 by 2^-8 (and u before it)."""

import math

import numpy as np
import pytest
import torch

from oracle import decoder as od
from oracle import kvcache as ok

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = torch.bfloat16
KINDS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_quantize_amd import kvcache
    kvcache.native()
    return kvcache


def _n(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _bits(t):
    return t.view(torch.uint8).cpu().numpy().copy()


def _gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s, std=1.0: (std * torch.randn(*s, generator=g, device="cuda")).to(BF)


def _used(K, pages, KV, page, d, kind, seed=9):
    """A cache with other contents."""
    c = K.KVCache.zeros(pages, KV, page, d, KINDS[kind])
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in (c.k, c.v):
        t.view(torch.uint8).copy_(torch.randint(0, 120, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in (c.k_scale, c.v_scale):
        t.copy_(torch.rand(t.shape, generator=g, device="cuda"))
    return c


def _at(t, slots, page):
    s = torch.as_tensor(slots, device=t.device).long()
    return t[s // page, :, s % page] if t.dim() == 3 else t.view(torch.uint8)[s // page, :, s % page].view(t.dtype)


def _check_values(K, cache, slots, v, kind):
    """The rows of v [T, KV, d] in their slots, bit for bit."""
    codes, scale = ok.encode(_n(v), kind)
    page = cache.v.shape[2]
    got_s = _at(cache.v_scale, slots, page).cpu().numpy()
    assert np.array_equal(got_s, scale, equal_nan=True)
    assert np.array_equal(_n(_at(cache.v, slots, page)), codes)


SHAPES = [  # T, H, KV, d, rot, page, interleaved, scaling
    (1, 1, 1, 16, 16, 1, False, "none"),
    (1, 8, 8, 128, 128, 16, False, "none"),
    (5, 6, 2, 64, 64, 16, True, "ntk"),
    (16, 64, 8, 128, 128, 16, False, "yarn"),
    (33, 4, 4, 80, 32, 32, True, "none"),        # half a head or less, three lanes of eight without elements
    (7, 2, 1, 96, 96, 64, False, "linear"),
    (40, 4, 2, 64, 40, 16, False, "none"),       # pairs that are no whole pieces
    (40, 4, 2, 112, 6, 16, True, "none"),
    (9, 3, 3, 256, 256, 128, False, "none"),
    (9, 0, 2, 256, 0, 16, False, "none"),        # nothing to rotate, no queries
    (1100, 4, 2, 128, 128, 16, False, "none"),   # several tokens per workgroup
    (1031, 2, 2, 32, 32, 1024, True, "yarn"),
]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("T,H,KV,d,rot,page,inter,scaling", SHAPES)
def test_write_and_read(K, T, H, KV, d, rot, page, inter, scaling, kind):
    from bit_nf4_quantized_quantize_amd import decoder as D
    r = _gen(T + d)
    pages = -(-T // page) + 3
    cache = _used(K, pages, KV, page, d, kind)
    old = {n: _bits(t) for n, t in cache._asdict().items()}
    q, k, v = (r(T, H, d) if H else None), r(T, KV, d), r(T, KV, d)
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32).cuda()
    pos = torch.randint(0, 100000, (T,), generator=g).to(torch.int32).cuda()
    table = D.RopeTable(rot, scaling=scaling, factor=1.0 if scaling == "none" else 8.0, original_len=4096,
                        interleaved=inter) if rot else None
    out = K.qlora_kv_write(q, k, v, table, pos if rot else None, slots, cache)
    if H:
        ref = D.qlora_rope(q, None, table, pos)[0] if rot else q
        assert torch.equal(out, ref)      # the queries are those of the rotary call
    else:
        assert out is None
    _check_values(K, cache, slots, v, kind)
    if rot:
        freq = table.turns.cpu().numpy() * 2 * math.pi
        ref = od.rope(_n(k), _n(pos), freq, table.mscale, inter)
        size = np.abs(_n(k))
        pair = size.copy()
        if inter:
            pair[..., 0:rot:2] = pair[..., 1:rot:2] = size[..., 0:rot:2] + size[..., 1:rot:2]
        else:
            h = rot // 2
            pair[..., :h] = pair[..., h:rot] = size[..., :h] + size[..., h:rot]
        off = 4 * U * table.mscale * pair
        got_s = _n(_at(cache.k_scale, slots, page))
        top = np.abs(ref).max(-1) / ok.MOST[kind]
        assert (np.abs(got_s - top) <= 2 * U * top + off.max(-1) / ok.MOST[kind]).all()
        codes = _n(_at(cache.k, slots, page))
        tol = ok.half_step(codes, kind) * got_s[..., None] + 2 * off + 2.0 ** -22 * np.abs(ref)
        assert (np.abs(codes * got_s[..., None] - ref) <= tol).all()
    else:
        codes, scale = ok.encode(_n(k), kind)
        assert np.array_equal(_n(_at(cache.k, slots, page)), codes)
        assert np.array_equal(_at(cache.k_scale, slots, page).cpu().numpy(), scale)
    # rows that no token names are as they were
    named = np.zeros(pages * page, bool)
    named[slots.cpu().numpy()] = True
    for n, t in cache._asdict().items():
        now = _bits(t).reshape(pages, KV, page, -1).transpose(0, 2, 1, 3).reshape(pages * page, -1)
        was = old[n].reshape(pages, KV, page, -1).transpose(0, 2, 1, 3).reshape(pages * page, -1)
        assert np.array_equal(now[~named], was[~named]), n
    # read back: any order, a slot twice, slots outside
    ask = torch.cat([slots.flip(0), slots[:1], torch.tensor([-1, pages * page, 2 ** 31 - 1, -2 ** 31], device="cuda",
                                                            dtype=torch.int32)])
    for dtype, half in ((torch.float32, U), (BF, 2.0 ** -8 + U)):
        got = K.qlora_kv_read(cache, ask, dtype=dtype)
        for z, c, s in ((got[0], cache.k, cache.k_scale), (got[1], cache.v, cache.v_scale)):
            assert z.dtype == dtype and z.shape == (len(ask), KV, d)
            ref = ok.read(ok.values(_n(c), _n(s)), ask.tolist())
            assert (np.abs(_n(z) - ref) <= half * np.abs(ref)).all()


@pytest.mark.parametrize("kind", list(KINDS))
def test_rows_that_are_hard_to_hold(K, kind):
    """Zeros, subnormal and huge sizes, ties between codes, NaN and infinities."""
    d, KV = 64, 1
    r = _gen(1)
    rows = [torch.zeros(d), r(d).cpu().float() * 2.0 ** -126, r(d).cpu().float() * 2.0 ** -130,
            r(d).cpu().float() * 2.0 ** 100, torch.full((d,), 3.3e38),
            torch.cat([torch.tensor([127.0 / 64]), (torch.arange(d - 1) + 0.5) / 64]),   # ties in whole numbers
            torch.cat([torch.tensor([3.5]), (torch.arange(d - 1) + 0.5) / 64])]
    for bad in (math.nan, math.inf, -math.inf):
        z = r(d).cpu().float()
        z[17] = bad
        rows.append(z)
    rows.append(torch.cat([torch.tensor([2.0 ** -133]), torch.zeros(d - 1)]))            # the smallest bfloat16
    v = torch.stack(rows).to(BF).cuda()[:, None]
    T = v.shape[0]
    cache = _used(K, 2, KV, 16, d, kind)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    K.qlora_kv_write(None, v, v, None, None, slots, cache)
    _check_values(K, cache, slots, v, kind)
    for a, b in ((cache.k, cache.v), (cache.k_scale, cache.v_scale)):   # keys that are not rotated alike
        assert np.array_equal(_bits(a[0, 0, :T]), _bits(b[0, 0, :T]))
    back = K.qlora_kv_read(cache, slots, dtype=torch.float32)[1].cpu()
    spoilt = ~torch.isfinite(v.float().cpu()).all(-1)
    assert torch.isnan(back[spoilt]).all() and torch.isfinite(back[~spoilt]).all()


@pytest.mark.parametrize("kind", list(KINDS))
def test_every_quotient_is_rounded_to_the_nearest_code(K, kind):
    """All pairs of a largest size and another one of 8 bits: the quotients next
    to the border of two codes among them."""
    d = 256
    top = 1.0 + torch.arange(128) / 128.0
    rows = torch.cat([torch.arange(1, 256).float() / 256.0, torch.zeros(1)])[None].repeat(128, 1) * 2.0 ** -1
    rows = torch.minimum(rows * 2, top[:, None])
    rows[:, -1] = top
    v = rows.to(BF).cuda()[:, None]
    cache = K.KVCache.zeros(8, 1, 16, d, KINDS[kind])
    slots = torch.arange(128, dtype=torch.int32, device="cuda")
    K.qlora_kv_write(None, v, v, None, None, slots, cache)
    _check_values(K, cache, slots, v, kind)


@pytest.mark.parametrize("kind", list(KINDS))
def test_strides_places_and_slots_outside(K, kind):
    """Tokens strided, queries rotated in place, some slots outside the cache."""
    from bit_nf4_quantized_quantize_amd import decoder as D
    r = _gen(2)
    T, H, KV, d, page = 20, 4, 2, 64, 16
    table, pos = D.RopeTable(d), torch.arange(T, dtype=torch.int32, device="cuda")
    for pad in (8, 3 * d, 4):   # the last: rows off the 16-byte grid, element by element
        wide = r(T, (H + 2 * KV) * d + pad)
        q, k, v = (wide[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, H), (H, H + KV), (H + KV, H + 2 * KV)))
        slots = torch.arange(T, dtype=torch.int32, device="cuda")
        slots[3], slots[4], slots[5] = -1, 2 * page, 2 ** 31 - 1
        cache, dense = (_used(K, 2, KV, page, d, kind) for _ in range(2))
        ref = K.qlora_kv_write(q.contiguous(), k.contiguous(), v.contiguous(), table, pos, slots, dense)
        out = K.qlora_kv_write(q, k, v, table, pos, slots, cache, q_out=q)
        assert out.data_ptr() == q.data_ptr() and torch.equal(q, ref)
        for a, b in zip(cache, dense):
            assert np.array_equal(_bits(a), _bits(b))
        live = [i for i in range(T) if i not in (3, 4, 5)]
        _check_values(K, cache, slots[live], v[live], kind)
        got = K.qlora_kv_read(cache, slots)
        assert not got[0][3:6].any() and not got[1][3:6].any()


def test_bfloat16_cache_is_the_decoders(K):
    from bit_nf4_quantized_quantize_amd import decoder as D
    r = _gen(3)
    T, H, KV, d, page = 21, 4, 2, 72, 16
    q, k, v, table = r(T, H, d), r(T, KV, d), r(T, KV, d), D.RopeTable(d)
    pos, slots = torch.arange(T, dtype=torch.int32, device="cuda"), torch.randperm(32, device="cuda")[:T].to(torch.int32)
    a = K.KVCache.zeros(2, KV, page, d)
    kc, vc = a.k.clone(), a.v.clone()
    assert torch.equal(K.qlora_kv_write(q, k, v, table, pos, slots, a),
                       D.qlora_rope_cache_write(q, k, v, table, pos, slots, kc, vc))
    assert torch.equal(a.k, kc) and torch.equal(a.v, vc)
    got = K.qlora_kv_read(a, slots)
    assert torch.equal(got[1], v)
    s = slots.long()
    assert torch.equal(K.qlora_kv_read(a, slots, dtype=torch.float32)[0], kc[s // page, :, s % page].float())


def test_given_outputs_and_empty_calls(K):
    cache = _used(K, 2, 2, 16, 32, "int8")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    z = torch.empty(0, 2, 32, dtype=BF, device="cuda")
    was = [_bits(t) for t in cache]
    assert K.qlora_kv_write(z, z, z, None, None, none, cache).shape == (0, 2, 32)
    assert all(np.array_equal(a, _bits(b)) for a, b in zip(was, cache))
    assert K.qlora_kv_read(cache, none)[0].shape == (0, 2, 32)
    slots = torch.tensor([3, 30], dtype=torch.int32, device="cuda")
    ko, vo = (torch.empty(2, 2, 32, device="cuda") for _ in range(2))
    got = K.qlora_kv_read(cache, slots, torch.float32, k_out=ko, v_out=vo)
    assert got[0].data_ptr() == ko.data_ptr() and got[1].data_ptr() == vo.data_ptr()
    ref = K.qlora_kv_read(cache, slots, torch.float32)
    assert torch.equal(ko, ref[0]) and torch.equal(vo, ref[1])


def test_offsets_beyond_32_bits(K):
    """A cache of more than 2^31 elements: its last rows."""
    KV, page, d = 2, 1024, 256
    pages = 2 ** 31 // (KV * page * d) + 3
    r = _gen(5)
    v = r(4, KV, d)
    for kind in KINDS:
        cache = K.KVCache.zeros(pages, KV, page, d, KINDS[kind])
        slots = torch.tensor([pages * page - 1, 0, (pages - 1) * page, 7], dtype=torch.int32, device="cuda")
        K.qlora_kv_write(None, v, v, None, None, slots, cache)
        _check_values(K, cache, slots, v, kind)
        codes, scale = ok.encode(_n(v), kind)
        got = K.qlora_kv_read(cache, slots, dtype=torch.float32)
        ref = ok.values(codes, scale)
        for z in got:
            assert (np.abs(_n(z) - ref) <= U * np.abs(ref)).all()
        del cache
