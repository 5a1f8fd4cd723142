"""QLoraBlock.decode behind a prefix that fills little of what the cache has room
for: the same calls, so the same results bit for bit, as from a cache made for it."""
import pytest
import torch

from test_gpu_block_kv import BL, KINDS, _block, _x  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", list(KINDS))
def test_room_for_a_longer_prefix_changes_nothing(BL, kind, monkeypatch):  # noqa: F811
    blk, seqs, prefix = _block(BL, 64), 40, 500
    shared, own = _x(prefix, seed=1), _x(3, seqs, seed=2)
    tables, call = [], BL.K.qlora_prefix_attention
    monkeypatch.setattr(BL.K, "qlora_prefix_attention", lambda *a, **kw: tables.append(a[2]) or call(*a, **kw))
    ys = []
    for most in (512, 32768):
        cache = blk.cache(32 + seqs, 16, seqs, 16, KINDS[kind], max_prefix=most)
        blk.prefill_shared(shared, cache)
        ys.append([blk.decode(x, cache) for x in own])
    assert [t.shape for t in tables] == [(32,)] * 6
    assert torch.isfinite(ys[0][2]).all()
    for a, b in zip(*ys):
        assert torch.equal(a, b)
    # a failed call leaves a table that a shorter prefix takes over
    cache = blk.cache(40, 16, 2, 16, KINDS[kind], max_prefix=512)
    broken = _block(BL, 64, post1=torch.ones(256, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(Exception):
        broken.prefill_shared(shared, cache)
    assert cache.prefix_pages.numel() == 0
    blk.prefill_shared(shared[:17], cache)
    blk.decode(own[0, :2], cache)
    assert tables[-1].shape == (2,)
