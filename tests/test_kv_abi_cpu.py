"""Checks of the 8-bit and the shared key-value cache that need no GPU: every
declared function is exported and bound, workspace sizes, and refusals of the C
ABI and of the compiled module, all on the host before anything is enqueued (the
pointers passed here are never dereferenced)."""

import ctypes
import os
import re
import sys

import pytest
import torch

import bit_nf4_quantized_quantize_amd as pkg
from bit_nf4_quantized_quantize_amd import binding as B
from bit_nf4_quantized_quantize_amd import decoder as D
from bit_nf4_quantized_quantize_amd import kvcache as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, MIS, MIS4 = 0x10000, 0x10004, 0x10002   # aligned, not to 16, not to 4
OK, BAD, DT, WS, AL = (B.QLORA_OK, B.QLORA_ERR_INVALID_ARG, B.QLORA_ERR_UNSUPPORTED_DTYPE,
                       B.QLORA_ERR_WORKSPACE_TOO_SMALL, B.QLORA_ERR_MISALIGNED)
BF16, INT8, E4M3 = 0, 1, 2
CACHE = dict(k=P, v=P, k_scale=P, v_scale=P, num_pages=4, page_size=16, kv_heads=2, head_dim=64, type=INT8)


def _caller(name, order, base):
    """Calls the C function with `base`, some of it changed; names of the cache's
    fields change the cache."""
    L = K.lib()

    def call(**kw):
        unknown = set(kw) - set(order) - {f"c_{n}" for n in CACHE}
        assert not unknown, unknown
        fields = {**CACHE, **{n[2:]: v for n, v in kw.items() if n.startswith("c_")}}
        if fields["type"] == BF16 and not any(n.endswith("_scale") for n in kw):
            fields["k_scale"] = fields["v_scale"] = None
        c = K.KVCacheStruct(**fields)
        args = [kw.get(n, base.get(n)) for n in order]
        args[order.index("cache")] = kw.get("cache", ctypes.byref(c))
        return getattr(L, name)(*args)
    return call


def test_exports_match_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "qlora_kvcache.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*int\s+(qlora_\w+)\s*\(", text, flags=re.M)))
    assert sorted(K.EXPORTED) == names == sorted(K._SIG)
    for n in names:
        assert hasattr(K.lib(), n)
    types = dict(re.findall(r"QLORA_CACHE_(\w+) = (\d)", text))
    assert types == {"BF16": "0", "INT8": "1", "E4M3": "2"}
    assert K.CACHE_TYPES == {torch.bfloat16: 0, torch.int8: 1, torch.float8_e4m3fn: 2}
    fields = re.search(r"typedef struct qlora_kv_cache \{(.*?)\}", text, flags=re.S).group(1)
    assert re.findall(r"(\w+);", fields) == [n for n, _ in K.KVCacheStruct._fields_]


def _descriptor_refusals(f, page_min=1):
    assert f(cache=None) == BAD
    assert f(c_type=3) == DT and f(c_type=-1) == DT
    for d in (0, -16, 8, 24, 72, 272, 2 ** 30):
        assert f(c_head_dim=d) == BAD, d
    assert f(c_type=BF16, c_head_dim=60) == BAD and f(c_type=BF16, c_head_dim=264) == BAD
    for p in (0, -16, 3, 24, 2048):
        assert f(c_page_size=p) == BAD, p
    if page_min > 1:
        assert f(c_page_size=8) == BAD
    assert f(c_kv_heads=0) == BAD and f(c_kv_heads=5000) == BAD
    assert f(c_num_pages=0) == BAD and f(c_num_pages=-1) == BAD and f(c_num_pages=2 ** 27) == BAD
    assert f(c_num_pages=2 ** 62) == BAD and f(c_num_pages=2 ** 26, c_kv_heads=2, c_head_dim=256) == BAD


def _buffer_refusals(f):
    for n in ("k", "v", "k_scale", "v_scale"):
        assert f(**{f"c_{n}": None}) == BAD and f(**{f"c_{n}": MIS}) == AL, n
        assert n in K.lib().qlora_last_error().decode()
    assert f(c_type=BF16, c_k_scale=P, c_v_scale=None) == BAD     # bfloat16 has no scales


WRITE = ("q q_stride q_heads qo qo_stride k k_stride v v_stride T rot positions turns mscale inter slots cache "
         "stream").split()


def test_write_refusals():
    f = _caller("qlora_kv_write", WRITE, dict(q=P, q_stride=256, q_heads=4, qo=P + 4096, qo_stride=256, k=P,
                                              k_stride=128, v=P, v_stride=128, T=2, rot=64, positions=P, turns=P,
                                              mscale=1.0, inter=0, slots=P))
    _descriptor_refusals(f)
    _buffer_refusals(f)
    assert f(T=-1) == BAD and f(T=2 ** 24) == BAD and f(rot=65) == BAD and f(rot=66) == BAD and f(rot=-2) == BAD
    assert f(q_heads=-1) == BAD and f(q_heads=5000) == BAD and f(inter=2) == BAD
    for n in ("q_stride", "qo_stride", "k_stride", "v_stride"):
        assert f(**{n: 64}) == BAD and f(**{n: 2 ** 60}) == BAD, n
    for n in ("q", "qo", "k", "v", "slots", "positions", "turns"):
        assert f(**{n: None}) == BAD and f(**{n: MIS if n not in ("slots", "positions") else MIS4}) == AL, n
    assert f(q=P, qo=P, qo_stride=512) == BAD                     # in place at another stride
    assert f(T=0, q=None, k=None, v=None, slots=None, c_k=None) == OK
    assert f(c_type=BF16, k=None) == BAD and f(c_type=BF16, T=0, k=None) == OK


READ = "cache slots T dtype k v stream".split()


def test_read_refusals():
    f = _caller("qlora_kv_read", READ, dict(slots=P, T=3, dtype=1, k=P, v=P))
    _descriptor_refusals(f)
    _buffer_refusals(f)
    assert f(dtype=2) == DT and f(dtype=-1) == DT
    assert f(T=-1) == BAD and f(T=2 ** 24) == BAD and f(T=2 ** 23, c_kv_heads=4096, c_head_dim=256) == BAD
    assert f(slots=None) == BAD and f(slots=MIS4) == AL and f(k=MIS) == AL and f(v=MIS) == AL
    assert f(T=0, slots=None) == OK and f(k=None, v=None) == OK


ATTN = "q q_stride S q_heads cache table cols lengths scale out lse ws nws stream".split()
PREFIX = "q q_stride S q_heads cache ptable pcols plen table cols lengths scale out lse ws nws stream".split()
BASE = dict(q=P, q_stride=256, S=2, q_heads=4, ptable=P, pcols=3, plen=P, table=P, cols=2, lengths=P, scale=0.1, out=P,
            lse=P, ws=P, nws=1 << 40)


@pytest.mark.parametrize("name,order", [("qlora_kv_attention", ATTN), ("qlora_prefix_attention", PREFIX)])
def test_attention_refusals(name, order):
    f = _caller(name, order, {k: v for k, v in BASE.items() if k in order})
    _descriptor_refusals(f, 16)
    _buffer_refusals(f)
    assert f(S=-1) == BAD and f(S=65536) == BAD
    assert f(q_heads=0) == BAD and f(q_heads=3) == BAD and f(q_heads=4098) == BAD and f(q_heads=-2) == BAD
    assert f(cols=-1) == BAD and f(cols=2 ** 31) == BAD and f(cols=2 ** 27) == BAD and f(cols=2 ** 62) == BAD
    for bad in (float("nan"), float("inf")):
        assert f(scale=bad) == BAD
    assert f(q_stride=255) == BAD and f(q_stride=260) == BAD and f(q_stride=2 ** 60) == BAD
    for n in ("q", "out", "lengths", "table"):
        assert f(**{n: None}) == BAD and f(**{n: MIS if n in ("q", "out") else MIS4}) == AL, n
    assert f(lse=MIS4) == AL
    assert f(S=0, q=None, out=None, lengths=None, table=None, **({"plen": None, "ptable": None} if "plen" in order
                                                                 else {})) == OK
    if "plen" in order:
        assert f(pcols=-1) == BAD and f(pcols=2 ** 27) == BAD and f(pcols=2 ** 27 - 1) == BAD
        assert f(S=2 ** 15, q_heads=2048, q_stride=2 ** 20) == BAD
        assert f(plen=None) == BAD and f(plen=MIS4) == AL and f(ptable=None) == BAD and f(ptable=MIS4) == AL


@pytest.mark.parametrize("typ", [BF16, INT8, E4M3])
def test_workspaces(typ):
    n = ctypes.c_int64()
    own = _caller("qlora_kv_attention_workspace", "cache S q_heads cols n".split(), dict(n=ctypes.byref(n)))
    both = _caller("qlora_prefix_attention_workspace", "cache S q_heads pcols cols n".split(), dict(n=ctypes.byref(n)))
    assert own(c_type=typ, S=2, q_heads=4, cols=4) == OK and n.value == 0             # one launch
    assert own(c_type=typ, S=2, q_heads=4, cols=4096) == OK and n.value > 0
    need = n.value
    f = _caller("qlora_kv_attention", ATTN, {k: v for k, v in BASE.items() if k in ATTN})
    assert f(c_type=typ, cols=4096, nws=need - 1) == WS and f(c_type=typ, cols=4096, nws=need, ws=None) == BAD
    assert f(c_type=typ, cols=4096, nws=need, ws=MIS) == AL
    assert own(c_type=typ, S=0, q_heads=4, cols=4096) == OK and n.value == 0
    assert both(c_type=typ, S=0, q_heads=4, pcols=64, cols=4) == OK and n.value == 0
    assert both(c_type=typ, S=2, q_heads=4, pcols=0, cols=4) == OK and n.value == 0   # no prefix
    f = _caller("qlora_prefix_attention", PREFIX, BASE)
    for S, pcols in ((2, 3), (2, 4096), (200, 64), (4096, 1000)):
        assert both(c_type=typ, S=S, q_heads=4, pcols=pcols, cols=4) == OK
        need = n.value
        assert need >= 2 * S * 4 * 66 * 4, "the parts of the prefix and of the own tokens"
        assert f(c_type=typ, S=S, pcols=pcols, cols=4, nws=need - 1) == WS
        assert f(c_type=typ, S=S, pcols=pcols, cols=4, nws=need, ws=None) == BAD
    for g in (own, both):
        assert g(c_type=typ, S=1, q_heads=4, cols=1, pcols=1, n=None) == BAD if g is both else \
            g(c_type=typ, S=1, q_heads=4, cols=1, n=None) == BAD


# ------------------------------------------------------------------ the module

I32, BF = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)


def _calls(dtype=torch.int8):
    q, kv = torch.zeros(2, 4, 32, **BF), torch.zeros(2, 2, 32, **BF)
    cache = K.KVCache.zeros(3, 2, 16, 32, dtype, device="cpu")
    ids, lens, cols = torch.zeros(2, **I32), torch.ones(2, **I32), torch.zeros(2, 2, **I32)
    t = D.RopeTable.__new__(D.RopeTable)
    t.turns, t.rot_dim, t.mscale, t.interleaved = torch.zeros(16, dtype=torch.float64), 32, 1.0, False
    attn = dict(q=q, cache=cache, block_table=cols, lengths=lens, out=q.clone(), lse=torch.zeros(2, 4))
    return {
        "write": (K.qlora_kv_write, dict(q=q, k=kv, v=kv, table=t, positions=ids, slots=ids, cache=cache,
                                         q_out=q.clone())),
        "read": (K.qlora_kv_read, dict(cache=cache, slots=ids, k_out=kv.clone(), v_out=kv.clone())),
        "attention": (K.qlora_kv_attention, attn),
        "prefix": (K.qlora_prefix_attention, dict(attn, prefix_table=ids, prefix_len=lens[:1].clone())),
    }


@pytest.mark.parametrize("dtype", list(K.CACHE_TYPES))
@pytest.mark.parametrize("name", list(_calls()))
def test_host_tensors_are_refused(name, dtype):
    f, kw = _calls(dtype)[name]
    with pytest.raises(ValueError, match="HIP device"):
        f(**kw)


@pytest.mark.parametrize("name", list(_calls()))
def test_every_tensor_argument_is_checked(name):
    """Each tensor argument in turn, those of the cache among them: not a tensor,
    another type, one more dimension, every second element."""
    f, kw = _calls()[name]
    spots = [(n, None) for n, t in kw.items() if isinstance(t, torch.Tensor)] + [("cache", i) for i in range(4)]
    for n, i in spots:
        t = kw[n] if i is None else kw[n][i]
        put = (lambda b: {**kw, n: b}) if i is None else (  # noqa: E731
            lambda b: {**kw, n: K.KVCache(*kw[n][:i], b, *kw[n][i + 1:])})
        with pytest.raises(TypeError, match=n if i is None else K.KVCache._fields[i]):
            f(**put(3))
        for bad in (t.to(torch.float16), t[None], t.repeat_interleave(2, -1)[..., ::2]):
            if bad.shape == (1,) and bad.dtype == t.dtype:
                continue      # every second element of one is that one
            with pytest.raises(ValueError) as e:
                f(**put(bad))
            assert "HIP device" not in str(e.value), (n, i, bad.shape, bad.dtype)


def test_caches_that_do_not_fit_together():
    f, kw = _calls()["read"]
    c, b = kw["cache"], _calls(torch.bfloat16)["read"][1]["cache"]
    for bad in (K.KVCache(c.k, c.v, None, None), K.KVCache(c.k, c.v, c.k_scale, None),
                K.KVCache(b.k, b.v, c.k_scale, c.v_scale), K.KVCache(c.k, b.v, c.k_scale, c.v_scale),
                K.KVCache(c.k, c.v[:2], c.k_scale, c.v_scale), K.KVCache(c.k, c.v, c.k_scale[:2], c.v_scale),
                K.KVCache(c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)):
        with pytest.raises(ValueError) as e:
            f(**{**kw, "cache": bad})
        assert "HIP device" not in str(e.value)
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        K.KVCache.zeros(2, 2, 16, 32, torch.float16, device="cpu")
    with pytest.raises(ValueError, match="dtype"):
        f(**kw, dtype=torch.float16)
    f, kw = _calls()["prefix"]
    for n in ("prefix_table", "prefix_len"):
        with pytest.raises(TypeError):
            f(**{**kw, n: None})
    with pytest.raises(TypeError):
        f(**kw, scale="1")
    f, kw = _calls()["write"]
    with pytest.raises(ValueError, match="heads"):
        f(**{**kw, "k": torch.zeros(2, 3, 32, **BF)})
    with pytest.raises(TypeError):
        K.native().read(kw["k"])


def test_a_missing_module_is_reported(monkeypatch):
    monkeypatch.setattr(K, "_native", None)
    monkeypatch.setitem(sys.modules, "bit_nf4_quantized_quantize_amd._kvcache", None)
    monkeypatch.delattr(pkg, "_kvcache", raising=False)
    f, kw = _calls()["read"]
    with pytest.raises(B.QLoraLibraryError, match="build it"):
        f(**kw)


# ---------------------------------------------------------------- the block's cache

@pytest.mark.parametrize("bad", [
    dict(dtype=torch.float16), dict(dtype=torch.int8, head_dim=72), dict(dtype=torch.float8_e4m3fn, head_dim=8),
    dict(max_prefix=-1), dict(max_prefix=2 ** 31), dict(max_prefix=2 ** 31 - 100, max_len=64)])
def test_caches_that_the_block_does_not_make(bad, monkeypatch):
    from bit_nf4_quantized_quantize_amd import block as BL
    good = dict(num_pages=2, page_size=16, heads=2, head_dim=64, max_seqs=3, max_len=32, device="cpu")
    for t in K.CACHE_TYPES:
        c = BL.PagedCache(**good, dtype=t, max_prefix=20)
        assert c.k.dtype == t and (c.rows.k_scale is None) == (t == torch.bfloat16) and c.prefix_table.shape == (2,)
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: pytest.fail("allocated"))
    with pytest.raises(ValueError):
        BL.PagedCache(**{**good, **bad})
