"""Attention behind a shared prefix by the kernels for many rows, which long
prefixes take (csrc/kv_prefix.hip): the checks of test_gpu_kv_attention, with
tables of the prefix that have room for many more tokens, none of them there. And
the sizes around the rule that chooses between the kernels."""
import pytest
import torch

import test_gpu_kv_attention as base
from test_gpu_kv_attention import KINDS, SHARED, _check, _i32, _setup

pytestmark = pytest.mark.gpu


class Roomy:
    """The kvcache module, the prefix's table filled up to more than 2^18 tokens
    times kv heads times tiles of 16 rows."""

    def __init__(self, module):
        self.module = module

    def __getattr__(self, name):
        return getattr(self.module, name)

    def qlora_prefix_attention(self, q, cache, prefix_table, *args, **kw):
        KV, page = cache.k.shape[1:3]
        tiles = -(-q.shape[0] * q.shape[1] // (16 * KV))
        more = max(0, 2 ** 18 // (max(tiles, 1) * KV * page) + 1 - prefix_table.shape[0])
        table = torch.cat((prefix_table, prefix_table.new_full((more,), -1)))
        return self.module.qlora_prefix_attention(q, cache, table, *args, **kw)


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_quantize_amd import kvcache
    kvcache.native()
    return Roomy(kvcache)


MANY = [c for c in SHARED if c[0] * c[1] // c[2] > 32] + [
    (40, 2, 2, 128, 16, 2, 35, 25, 550),                    # a row to a sequence and kv head
    (140, 4, 4, 64, 32, 1, 9, 32, 270),                     # of enough sequences for whole own parts
    (70, 8, 4, 128, 16, 2, 40, 32, 630),                    # two rows, 140 in all
    (150, 4, 2, 128, 16, 1, 40, 16, 639),                   # 300
]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("S,H,KV,d,page,cols,pcols,high,prefix", MANY)
def test_shared_prefix(K, S, H, KV, d, page, cols, pcols, high, prefix, kind):
    base.test_shared_prefix(K, S, H, KV, d, page, cols, pcols, high, prefix, kind)


@pytest.mark.parametrize("kind", list(KINDS))
def test_lengths_of_zero_and_beyond(K, kind):
    base.test_lengths_of_zero_and_beyond(K, 40, kind)


@pytest.mark.parametrize("kind", list(KINDS))
def test_pages_that_are_none(K, kind):
    base.test_pages_that_are_none(K, 40, kind)


@pytest.mark.parametrize("kind", list(KINDS))
def test_what_lies_behind_a_length_is_not_used(K, kind):
    base.test_what_lies_behind_a_length_is_not_used(K, 40, kind)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_a_row_that_could_not_be_held_spoils_its_own_head(K, kind):
    base.test_a_row_that_could_not_be_held_spoils_its_own_head(K, 40, kind)


def test_an_infinity_among_the_values_stays_one(K):
    base.test_an_infinity_among_the_values_stays_one(K, 40)


@pytest.mark.parametrize("kind", list(KINDS))
def test_scales_strides_and_given_outputs(K, kind):
    base.test_scales_strides_and_given_outputs(K, 48, kind)


@pytest.mark.parametrize("kind", list(KINDS))
def test_large_scores(K, kind):
    base.test_large_scores(K, kind)


def test_offsets_beyond_32_bits(K):
    base.test_offsets_beyond_32_bits(K)


@pytest.mark.parametrize("kind", list(KINDS))
def test_graphs_and_streams(K, kind):
    base.test_graphs_and_streams(K, 40, kind)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("S,H,KV,d,pcols", [
    (1024, 1, 1, 16, 4), (1025, 1, 1, 16, 4),               # rows
    (16, 16, 4, 64, 1024), (16, 16, 4, 64, 1025),           # 4 tiles of 4 heads: 2^18 tokens of room, and a page more
    (32, 2, 2, 64, 4096), (33, 2, 2, 64, 4096),             # 32 rows are few whatever the room
])
def test_around_the_choice(K, S, H, KV, d, pcols, kind):
    q, c, table, ptable = _setup(K, S, H, KV, d, 16, 1, 20, kind)
    room = torch.cat((ptable, ptable.new_full((max(0, pcols - 20),), -1)))[:pcols]
    n = min(16 * pcols, 317)
    _check(K.module, q, c, table, [(3 * i) % 17 for i in range(S)], room, n)
    # the same tokens whatever the room of the table
    if pcols >= 20:
        a = K.module.qlora_prefix_attention(q, c, room, _i32([n]), table, _i32([9] * S))
        b = K.module.qlora_prefix_attention(q, c, ptable, _i32([n]), table, _i32([9] * S))
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()
