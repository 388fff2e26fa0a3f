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
