"""PagedCache without a GPU: what its operators cannot take is refused when the
cache is made, and wrong counts before anything is enqueued."""

import pytest
import torch

from bit_nf4_quantized_quantize_amd import block as BL
from bit_nf4_quantized_quantize_amd import decoder as D

GOOD = dict(num_pages=2, page_size=16, heads=2, head_dim=64, max_seqs=3, max_len=32, device="cpu")


@pytest.mark.parametrize("bad", [
    dict(max_seqs=0), dict(max_seqs=-1), dict(max_seqs=D.PLAN_MAX_SEQS + 1), dict(num_pages=0), dict(num_pages=2 ** 27),
    dict(heads=0), dict(max_len=0), dict(max_len=2 ** 31)])
def test_sizes_the_operators_do_not_take(bad, monkeypatch):
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: pytest.fail("allocated"))
    with pytest.raises(ValueError):
        BL.PagedCache(**{**GOOD, **bad})


def test_the_most_sequences_are_taken():
    c = BL.PagedCache(**{**GOOD, "max_seqs": D.PLAN_MAX_SEQS})
    assert c.table.shape == (D.PLAN_MAX_SEQS, 2) and len(c.host_lens) == D.PLAN_MAX_SEQS
