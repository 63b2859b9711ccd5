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


def test_pages_in_another_order(tq):
    """The bytes of whole pages are not enough: rows of a head lie together."""
    import torch
    tab = torch.zeros((2, 2), dtype=torch.int32)
    pages = torch.zeros((4, 2, 16, 68), dtype=torch.uint8)
    assert tq.PagedKV(pages, pages, tab, 16, 2).n_pages == 4
    for shape in ((4, 16, 2, 68), (2, 4, 16, 68), (4, 2, 8, 136), (4, 2, 16 * 68), (4 * 2 * 16 * 68,), (1, 4, 2, 16, 68)):
        other = pages.reshape(shape)
        for k, v in ((other, other), (pages, other)):
            with pytest.raises(ValueError):
                tq.PagedKV(k, v, tab, 16, 2)
    one = torch.zeros((3, 1, 16, 68), dtype=torch.uint8)
    with pytest.raises(ValueError):
        tq.PagedKV(pages, one, tab, 16, 2)
    with pytest.raises(ValueError):
        tq.PagedKV(pages[:0], pages[:0], tab, 16, 2)


def test_the_documentation_says_which_layer_may_write_the_lengths_in_place(tq):
    """Every layer's call counts its slots from the lengths that the last layer's may overwrite."""
    import os
    import re
    assert "last layer" in " ".join(tq.tq_paged_tree_keep.__doc__.split())
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "tq.h")
    says = re.search(r"new_lens    device int32(.*?)\*/", open(header).read(), re.S).group(1)
    assert "last layer's call only" in " ".join(says.replace("*", " ").split()).lower()
