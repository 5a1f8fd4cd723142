"""C-ABI checks of the decoder-block operators that need no GPU: every declared
function is exported and bound, host queries, and refusals, all of which
happen on the host before anything is enqueued (the pointers passed here are
never dereferenced)."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

from bit_nf4_quantized_quantize_amd import binding as B
from bit_nf4_quantized_quantize_amd import decoder as D
from oracle import decoder as od

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, MIS, MIS4 = 0x10000, 0x10004, 0x10002   # aligned, not to 16, not to 4
OK, BAD, DT, WS, AL = (B.QLORA_OK, B.QLORA_ERR_INVALID_ARG, B.QLORA_ERR_UNSUPPORTED_DTYPE,
                       B.QLORA_ERR_WORKSPACE_TOO_SMALL, B.QLORA_ERR_MISALIGNED)
F32, BF16 = B.QLORA_DTYPE_F32, B.QLORA_DTYPE_BF16


def _caller(name, order, base):
    L = D.lib()

    def call(**kw):
        unknown = set(kw) - set(order)
        assert not unknown, unknown
        return getattr(L, name)(*[kw.get(k, base[k]) for k in order])
    return call


def test_exports_match_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "qlora_decoder.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*int\s+(qlora_\w+)\s*\(", text, flags=re.M)))
    assert sorted(D.EXPORTED) == names == sorted(D._SIG)
    for n in names:
        assert hasattr(D.lib(), n)
    macros = dict(re.findall(r"#define (QLORA_\w+) (\d+)", text))
    assert int(macros["QLORA_NORM_MAX_WIDTH"]) == D.NORM_MAX_WIDTH
    assert int(macros["QLORA_PLAN_MAX_SEQS"]) == D.PLAN_MAX_SEQS


FWD = ("x xt h ht T D w_post gate alpha w_pre eps xo n stream").split()


def test_norm_forward_refusals():
    f = _caller("qlora_norm_residual_fwd", FWD, dict(x=P, xt=BF16, h=P, ht=BF16, T=2, D=64, w_post=P, gate=P,
                                                     alpha=1.0, w_pre=P, eps=1e-6, xo=P, n=P, stream=None))
    assert f(xt=BF16, ht=F32) == DT and f(xt=2) == DT and f(ht=-1) == DT
    assert f(T=-1) == BAD and f(T=2 ** 31) == BAD and f(D=0) == BAD and f(D=16385) == BAD
    assert f(eps=-1.0) == BAD and f(eps=float("nan")) == BAD and f(eps=float("inf")) == BAD
    assert f(xo=None, n=None) == BAD and f(w_pre=None) == BAD and f(h=None) == BAD and f(x=None) == BAD
    for k in ("x", "h", "w_post", "gate", "w_pre", "xo", "n"):
        assert f(**{k: MIS}) == AL, k
        assert k in D.lib().qlora_last_error().decode()
    assert f(T=0, x=None, h=None, w_post=None, gate=None) == OK


BWD = ("dxo xo xt dn h ht T D w_post gate alpha w_pre eps dx dh dw_post dgate dw_pre ws nws stream").split()


def test_norm_backward_refusals():
    f = _caller("qlora_norm_residual_bwd", BWD,
                dict(dxo=P, xo=P, xt=F32, dn=P, h=P, ht=BF16, T=2, D=64, w_post=P, gate=P, alpha=1.0, w_pre=P,
                     eps=1e-6, dx=P, dh=P, dw_post=P, dgate=P, dw_pre=P, ws=P, nws=1 << 20, stream=None))
    assert f(xt=BF16, ht=F32) == DT and f(T=-1) == BAD and f(D=20000) == BAD
    assert f(w_post=None) == BAD and f(dn=None) == BAD and f(w_pre=None) == BAD and f(h=None) == BAD
    assert f(w_post=None, dw_post=None, h=None) == BAD          # the gate's gradient needs h
    assert f(xo=None) == BAD and f(dx=None) == BAD
    for k in ("dxo", "xo", "dn", "h", "w_post", "gate", "w_pre", "dx", "dh", "dw_post", "dgate", "dw_pre", "ws"):
        assert f(**{k: MIS}) == AL, k
    n = ctypes.c_int64()
    g = D.lib().qlora_norm_residual_bwd_workspace
    assert g(2, 64, F32, BF16, 3, ctypes.byref(n)) == OK and n.value >= 2 * 64 * 4
    assert f(nws=n.value - 1) == WS and f(ws=None) == BAD
    assert g(2, 64, F32, BF16, 0, ctypes.byref(n)) == OK and n.value == 0
    assert g(0, 64, F32, BF16, 3, ctypes.byref(n)) == OK and n.value == 0
    assert g(2, 64, F32, BF16, 4, ctypes.byref(n)) == BAD and g(2, 64, F32, BF16, 3, None) == BAD
    assert g(2, 64, BF16, F32, 3, ctypes.byref(n)) == DT
    assert f(T=0, dw_post=None, dgate=None, dw_pre=None, xo=None, dx=None) == OK


ROPE = ("q qs qh qo qos k ks kh ko kos T d rot dt pos turns m inter inv stream").split()


def test_rope_refusals():
    f = _caller("qlora_rope", ROPE, dict(q=P, qs=256, qh=4, qo=P + 4096, qos=256, k=P, ks=128, kh=2, ko=P + 4096,
                                         kos=128, T=3, d=64, rot=64, dt=BF16, pos=P, turns=P, m=1.0, inter=0, inv=0,
                                         stream=None))
    assert f(dt=2) == DT and f(T=-1) == BAD and f(T=2 ** 24) == BAD
    assert f(d=0) == BAD and f(d=1025) == BAD and f(rot=63) == BAD and f(rot=66) == BAD and f(rot=-2) == BAD
    assert f(qh=-1) == BAD and f(kh=5000) == BAD and f(inter=2) == BAD and f(inv=-1) == BAD
    for k in ("qs", "qos", "ks", "kos"):
        assert f(**{k: 127}) == BAD, k
        assert f(**{k: 2 ** 62}) == BAD, k
    for k in ("q", "qo", "k", "ko", "turns"):
        assert f(**{k: None}) == BAD and f(**{k: MIS}) == AL, k
    assert f(pos=None) == BAD and f(pos=MIS4) == AL
    assert f(qo=P, qos=512) == BAD and f(ko=P, kos=512) == BAD     # in place with other strides
    assert f(T=0, q=None) == OK and f(qh=0, kh=0, q=None, k=None) == OK


def test_rope_frequencies():
    out, m = (ctypes.c_double * 512)(), ctypes.c_float()
    f = D.lib().qlora_rope_frequencies
    good = (64, 1e4, 0, 1.0, 0.0, 32.0, 1.0)
    assert f(*good, out, ctypes.byref(m)) == OK
    for i, vals in enumerate([(0, 63, 1026, -2), (1.0, -1.0, float("inf"), float("nan")), (-1, 4),
                              (0.5, float("nan"), float("inf"))]):
        for v in vals:
            a = list(good)
            a[i] = v
            assert f(*a, out, ctypes.byref(m)) == BAD, (i, v)
    assert f(2, 1e4, 2, 2.0, 0.0, 32.0, 1.0, out, ctypes.byref(m)) == BAD        # NTK of one pair
    assert f(64, 1e4, 3, 2.0, 0.0, 32.0, 1.0, out, ctypes.byref(m)) == BAD       # YaRN without its length
    assert f(64, 1e4, 3, 2.0, 4096.0, 1.0, 1.0, out, ctypes.byref(m)) == BAD
    assert f(*good, None, ctypes.byref(m)) == BAD and f(*good, out, None) == BAD
    for scaling, factor in (("none", 1.0), ("linear", 3.0), ("ntk", 8.0), ("yarn", 16.0)):
        kw = dict(base=10000.0, scaling=scaling, factor=factor, original_len=4096)
        t, ms = D.qlora_rope_frequencies(128, **kw)
        fr, mr = od.rope_frequencies(128, **kw)
        assert np.allclose(np.array(t) * 2 * np.pi, fr, rtol=1e-14, atol=0) and abs(ms - mr) <= 2.0 ** -24 * mr
    with pytest.raises(ValueError):
        D.qlora_rope_frequencies(64, scaling="cubic")
    with pytest.raises(B.QLoraError):
        D.qlora_rope_frequencies(-2)


WRITE = ("q qs qh qo qos k ks v vs kh T d rot pos turns m inter slots kc vc pages page stream").split()


def test_cache_write_refusals():
    f = _caller("qlora_rope_cache_write", WRITE,
                dict(q=P, qs=256, qh=4, qo=P, qos=256, k=P, ks=128, v=P, vs=128, kh=2, T=3, d=64, rot=64, pos=P,
                     turns=P, m=1.0, inter=0, slots=P, kc=P, vc=P, pages=4, page=16, stream=None))
    assert f(T=-1) == BAD and f(kh=0) == BAD and f(d=0) == BAD and f(rot=66) == BAD and f(inter=2) == BAD
    for v in (0, 3, 24, -16, 2048):
        assert f(page=v) == BAD, v
    for v in (0, -1, 2 ** 27, 2 ** 62):
        assert f(pages=v) == BAD, v
    for k in ("qs", "qos", "ks", "vs"):
        assert f(**{k: 127}) == BAD and f(**{k: 2 ** 62}) == BAD, k
    for k in ("q", "qo", "k", "v", "turns", "kc", "vc"):
        assert f(**{k: None}) == BAD and f(**{k: MIS}) == AL, k
    for k in ("pos", "slots"):
        assert f(**{k: None}) == BAD and f(**{k: MIS4}) == AL, k
    assert f(qos=512) == BAD
    assert f(T=0, k=None) == OK


PLAN = ("cached new S page free nfree table cols T total starts slots pos need stream").split()


def test_plan_refusals():
    f = _caller("qlora_paged_plan", PLAN, dict(cached=P, new=P, S=3, page=16, free=P, nfree=5, table=P, cols=4, T=9,
                                               total=P + 64, starts=P, slots=P, pos=P, need=P, stream=None))
    assert f(total=P) == BAD            # in place of the lengths
    assert f(S=-1) == BAD and f(S=4097) == BAD and f(page=0) == BAD
    for k in ("nfree", "cols", "T"):
        assert f(**{k: -1}) == BAD and f(**{k: 2 ** 31}) == BAD, k
    for k in ("cached", "new", "free", "table", "total", "starts", "slots", "pos", "need"):
        assert f(**{k: None}) == BAD and f(**{k: MIS4}) == AL, k


ATTN = ("q qs S H KV d kc vc pages page table cols lens scale out lse ws nws stream").split()


def test_attention_refusals():
    f = _caller("qlora_paged_attention", ATTN,
                dict(q=P, qs=256, S=2, H=4, KV=2, d=64, kc=P, vc=P, pages=8, page=16, table=P, cols=4, lens=P,
                     scale=1.0, out=P, lse=P, ws=P, nws=1 << 30, stream=None))
    assert f(S=-1) == BAD and f(S=65536) == BAD and f(H=3) == BAD and f(KV=0) == BAD and f(H=0) == BAD
    for v in (0, 4, 65, 264, 512, -8):
        assert f(d=v, qs=4096) == BAD, v
    for v in (8, 1, 0, 17, 2048, -16):
        assert f(page=v) == BAD, v
    assert f(cols=-1) == BAD and f(cols=2 ** 27) == BAD and f(cols=2 ** 62) == BAD
    assert f(pages=0) == BAD and f(pages=2 ** 27) == BAD
    assert f(scale=float("nan")) == BAD and f(scale=float("inf")) == BAD
    assert f(qs=255) == BAD and f(qs=260) == BAD and f(qs=2 ** 62) == BAD
    for k in ("q", "kc", "vc", "out"):
        assert f(**{k: None}) == BAD and f(**{k: MIS}) == AL, k
    for k in ("table", "lens"):
        assert f(**{k: None}) == BAD and f(**{k: MIS4}) == AL, k
    assert f(lse=MIS4) == AL
    n = ctypes.c_int64()
    g = D.lib().qlora_paged_attention_workspace
    assert g(2, 4, 2, 64, 4, 16, ctypes.byref(n)) == OK and n.value >= 0
    assert g(2, 4, 3, 64, 4, 16, ctypes.byref(n)) == BAD and g(2, 4, 2, 64, 4, 16, None) == BAD
    assert g(1, 32, 32, 128, 4096, 16, ctypes.byref(n)) == OK
    if n.value:
        big = dict(S=1, H=32, KV=32, d=128, qs=4096, cols=4096)
        assert f(**big, nws=n.value - 1) == WS and f(**big, ws=None) == BAD and f(**big, ws=MIS) == AL
    assert f(S=0, q=None, out=None) == OK


def test_binding_refuses_what_is_not_on_a_device_or_not_laid_out():
    x, w = torch.zeros(2, 8), torch.ones(8)
    with pytest.raises(ValueError, match="HIP device"):
        D.qlora_norm_residual_fwd(x, x, w_pre=w)
    for bad in (dict(x=x.t()), dict(x=x.half()), dict(h=torch.zeros(2, 7)), dict(w_pre=w.double()),
                dict(gate=torch.ones(7)), dict(h=x, n_dtype=torch.bfloat16), dict(n_dtype=torch.float16)):
        with pytest.raises(ValueError):
            D.qlora_norm_residual_fwd(**{**dict(x=x, w_pre=w), **bad})
    with pytest.raises(ValueError):
        D.qlora_norm_residual_bwd(x, x.bfloat16(), x, x)
    q = torch.zeros(3, 2, 8, dtype=torch.bfloat16)
    i3 = torch.zeros(3, dtype=torch.int32)
    kc = torch.zeros(2, 2, 16, 8, dtype=torch.bfloat16)
    for bad in (dict(lengths=i3.long()), dict(lengths=i3[:2]), dict(block_table=i3), dict(block_table=i3.view(1, 3)),
                dict(k_cache=kc[0]), dict(v_cache=kc[:1]), dict(k_cache=kc.float()), dict(q=q.float()),
                dict(q=q.transpose(0, 1)), dict(q=torch.zeros(3, 2, 16, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            D.qlora_paged_attention(**{**dict(q=q, k_cache=kc, v_cache=kc, block_table=i3.view(3, 1), lengths=i3),
                                       **bad})
    with pytest.raises(ValueError):
        D.qlora_paged_plan(i3, i3.long(), i3, i3.view(3, 1), 16, 3)
    with pytest.raises(ValueError):
        D.qlora_paged_plan(i3, i3, i3, i3.view(1, 3), 16, 3)
    tab = D.RopeTable(8, device="cpu")
    assert tab.turns.dtype == torch.float64 and tab.turns.numel() == 4
    for bad in (dict(q=q.half()), dict(q=None, k=None), dict(positions=i3.long()), dict(positions=i3[:2]),
                dict(k=q.float()), dict(q=q[0])):
        with pytest.raises(ValueError):
            D.qlora_rope(**{**dict(q=q, k=q, table=tab, positions=i3), **bad})
    with pytest.raises(ValueError):
        D.qlora_rope_cache_write(q, q[:, :1], q, tab, i3, i3, kc, kc)
