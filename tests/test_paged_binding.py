"""Arguments of the paged calls' Python objects that can be left out or be mistaken."""

import pytest


@pytest.fixture(scope="module")
def tq():
    import __graft_entry__
    __graft_entry__.build()
    import compressed_attention_gb300 as m
    return m


def test_most_rows_of_a_sequence_left_out(tq):
    """Offsets without max_q: a bound that holds for any offsets, so that no row is left out."""
    import torch
    lens, cu = torch.tensor([9, 4], dtype=torch.int32), torch.tensor([0, 5, 6], dtype=torch.int32)
    assert tq.PagedBatch(lens, cu, n_tokens=6).c.max_q == 6
    assert tq.PagedBatch(lens, cu, 5, 6).c.max_q == 5
    assert tq.PagedBatch(lens, cu, n_tokens=0).c.max_q == 1
    assert tq.PagedBatch(lens).c.max_q == 1
