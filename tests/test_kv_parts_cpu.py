"""How the own tokens of a batch behind a shared prefix are cut, told from the
workspaces that the calls ask for (a row of head_dim + 2 fp32 numbers for each
part, none for a single one)."""

import ctypes

import pytest

from bit_nf4_quantized_quantize_amd import kvcache as K

PAGE, D = 32, 128


def _parts(S, H, KV, own, prefix, typ):
    n = ctypes.c_int64()
    c = K.KVCacheStruct(k=None, v=None, k_scale=None, v_scale=None, num_pages=4096, page_size=PAGE, kv_heads=KV,
                        head_dim=D, type=typ)
    if prefix is None:
        assert K.lib().qlora_kv_attention_workspace(ctypes.byref(c), S, H, own // PAGE, ctypes.byref(n)) == 0
    else:
        assert K.lib().qlora_prefix_attention_workspace(ctypes.byref(c), S, H, prefix // PAGE, own // PAGE,
                                                        ctypes.byref(n)) == 0
    per = S * H * (D + 2) * 4
    assert n.value % per == 0
    return max(n.value // per, 1)


def _own(S, H, KV, own, typ, prefix=8000):
    return _parts(S, H, KV, own, prefix, typ) - _parts(S, H, KV, 0, prefix, typ) + 1


@pytest.mark.parametrize("typ", [0, 1, 2])
@pytest.mark.parametrize("S,H,KV", [(32, 32, 8), (64, 32, 8), (32, 64, 8), (40, 64, 16)])
def test_long_own_tokens_are_cut_behind_a_prefix_too(S, H, KV, typ):
    """From 256 workgroups on they stay whole only up to the length that this was
    measured to pay at."""
    for own in (2048, 4096, 16384, 65536):
        assert _own(S, H, KV, own, typ) == _parts(S, H, KV, own, None, typ) > 1, own
    for own in (32, 512, 768, 1024):
        assert _own(S, H, KV, own, typ) == 1, own


@pytest.mark.parametrize("typ", [0, 1, 2])
@pytest.mark.parametrize("S,KV", [(40, 8), (40, 16), (63, 16)])
def test_one_query_head_per_key_head_is_cut_as_without_a_prefix(S, KV, typ):
    """Whole own tokens are for workgroups that join the prefix's parts, which those
    of one row do not."""
    for own in (32, 512, 768, 1024, 4096, 16384):
        assert _own(S, KV, KV, own, typ) == _parts(S, KV, KV, own, None, typ), own
