"""qsa_pages_* where table entries name pages that nobody holds."""

import pytest
import torch

from learned_sparse_attention_gb300 import qsa as Q
from tests.test_pages import I32, empty

pytestmark = pytest.mark.gpu


def put(b, r, k, page):
    b.table[r, k] = page
    b.model.table[r][k] = page


@pytest.mark.parametrize("kind", ["none", "kv", "block"])
def test_packing_counts_entries_on_free_pages(kind):
    """Sequences 0, 2 and 4 leave; entries of those that stay then name pages that
    nobody holds: below the pages in use, where another sequence's tokens arrive,
    behind them, and outside.  They are counted and left."""
    b = empty(20, 6, 4, 16, kind)
    b.extend([40, 20, 33, 64, 16, 48])       # 3 2 3 4 1 3 pages: 0 .. 15
    holes = [p for r in (0, 2, 4) for p in b.model.table[r] if p >= 0]
    b.free([0, 2, 4])
    live = sum(r > 0 for r in b.model.refs)
    assert live == 9 and holes[0] < live <= holes[-1]
    for r, k, page in ((1, 1, holes[0]), (3, 0, holes[1]), (3, 2, holes[-1]), (5, 1, 19), (5, 2, 20)):
        b.model.refs[b.model.table[r][k]] -= 1
        put(b, r, k, page)
    b.refs.copy_(torch.tensor(b.model.refs))
    before = [list(t) for t in b.model.table]
    live = torch.zeros(1, **I32)
    ws = torch.full((Q.pages_workspace_bytes(b.pool),), 0xAB, dtype=torch.uint8, device="cuda")
    Q.pages_compact(b.pool, live, ws)
    assert b.model.compact() == live.item() == 4 and b.model.errors == 5
    b.same("compact")
    for r, k in ((1, 1), (3, 0), (3, 2), (5, 1), (5, 2)):
        assert b.table[r, k] == before[r][k]
    assert (b.refs[:4] > 0).all() and not b.refs[4:].any()
    b.compact()                               # (again: nothing moves)


@pytest.mark.parametrize("blocks", [3, 4097, 40003])
def test_every_free_page_is_known(blocks):
    """A table row over the whole pool, every other page of which is free, from
    odd and even ones on."""
    for odd in (0, 1):
        b = empty(blocks, 2, blocks, 16, "none")
        refs = [(p + odd) % 2 for p in range(blocks)]
        b.refs.copy_(torch.tensor(refs))
        b.model.refs = list(refs)
        b.table[0].copy_(torch.arange(blocks))
        b.model.table[0] = list(range(blocks))
        b.lengths[0] = b.model.lengths[0] = 16 * blocks
        b.compact()


@pytest.mark.parametrize("kind", ["none", "kv", "block"])
@pytest.mark.parametrize("bad", [-1, -7, 20, 1 << 30])
def test_forks_of_a_last_page_outside_the_pool(kind, bad):
    """The child's entry is -1 as well: it takes no page, whose bytes would be
    those of a sequence that has left, and its neighbours get theirs as if it were
    not there."""
    b = empty(20, 8, 4, 16, kind)
    b.extend([40, 20, 32, 5, 0, 0, 0, 0])
    put(b, 0, 2, bad)
    b.fork([1, 0, 3], [4, 5, 6])
    assert b.table[5].tolist() == b.table[0].tolist()[:2] + [-1, -1] and b.lengths[5] == 40
    b.extend([0, 0, 0, 0, 1, 1, 1, 0])     # (a token on that page has no slot)
    b.free([5])
    b.fork([2, 0], [5, 7])


def test_a_bad_last_page_leaves_the_last_free_one():
    b = empty(4, 6, 4, 16)
    b.extend([20, 5, 0, 0, 0, 0])          # three pages of four
    put(b, 0, 1, 99)
    b.fork([0, 1, 1], [2, 3, 4])           # the last free page is the second's, the third is refused
    assert b.lengths.tolist() == [20, 5, 20, 5, 0, 0]


def test_many_forks_some_of_bad_pages():
    """More forks than a planner has threads."""
    reqs = 2600
    b = empty(9000, reqs, 3, 16, "none")
    b.extend([(r * 7) % 41 if r < 600 else 0 for r in range(reqs)])
    for r in range(0, 600, 5):
        n = b.model.lengths[r]
        if n % 16:
            put(b, r, n // 16, -1 if r % 2 else 9000 + r)
    children = list(range(600, reqs))
    b.fork([(7 * c) % 600 for c in children], children)
    b.extend([1] * reqs)
