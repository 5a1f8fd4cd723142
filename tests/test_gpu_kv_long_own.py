"""Long own tokens behind a shared prefix that the kernels for many rows take, on
both sides of the length up to which they stay whole and join the prefix's parts:
the checks of test_gpu_kv_attention, even lengths and one long among short ones."""
import pytest
import torch

from test_gpu_kv_attention import KINDS, _check, _setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_quantize_amd import kvcache
    kvcache.native()
    return kvcache


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("room", [1024, 1056, 4096])
@pytest.mark.parametrize("S,H,KV,d", [(40, 16, 8, 32), (40, 8, 8, 32)])
def test_long_own_tokens(K, S, H, KV, d, room, kind):
    q, c, table, ptable = _setup(K, S, H, KV, d, 32, room // 32, 3, kind, seed=room)
    ptable = torch.cat((ptable, ptable.new_full((2 ** 18 // (KV * 32) + 1,), -1)))     # room for many tokens
    _check(K, q, c, table, [room if s == 7 else s % 40 for s in range(S)], ptable, 83)
    if room < 2000:
        _check(K, q, c, table, [room - s for s in range(S)], ptable, 83)
