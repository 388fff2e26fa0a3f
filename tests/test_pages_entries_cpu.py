"""The host model of qsa_pages_* on table entries that name no page in use, worked
out by hand (CPU only)."""

import torch

from pages_model import Model


def make(refs, table, lengths):
    plane = torch.arange(len(refs)).view(-1, 1, 1, 1).expand(-1, 1, 16, 1).to(torch.uint8).contiguous()
    return Model(torch.tensor(refs), torch.tensor(table), torch.tensor(lengths), 16, [plane]), plane


def test_fork_of_a_last_page_outside_the_pool():
    """"Entries of a parent outside the pool are counted, become -1 in the child
    and are not copied": a full page's, a last page's."""
    m, plane = make([1, 1, 0, 0], [[0, 4, -1], [1, -1, -1], [-1] * 3, [-1] * 3], [20, 5, 0, 0])
    before = plane.clone()
    assert m.fork([0, 1], [2, 3]) == [-1, 2]       # the first takes no page
    assert m.table[2] == [0, -1, -1] and m.table[3] == [2, -1, -1]
    assert m.refs == [2, 1, 1, 0] and m.lengths == [20, 5, 20, 5] and m.errors == 1
    assert torch.equal(plane[[0, 1, 3]], before[[0, 1, 3]]) and plane[2, 0, :5, 0].tolist() == [1] * 5


def test_packing_with_an_entry_on_a_free_page():
    """"Table entries that name no used page are counted and left": 1 is free and
    below the two pages in use, 5 free behind them."""
    m, plane = make([1, 0, 0, 1, 0, 0], [[0, 1, -1], [3, 5, -1]], [20, 20])
    assert m.compact() == 2
    assert m.table == [[0, 1, -1], [1, 5, -1]] and m.refs == [1, 1, 0, 0, 0, 0] and m.errors == 2
    assert plane[1, 0, 0, 0] == 3
