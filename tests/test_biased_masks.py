"""qsa_biased_gqa on GB300: documents and prefixes at the ends of the integers,
beside ordinary rows."""

import numpy as np
import pytest

from learned_sparse_attention_gb300 import qsa as Q
from tests.test_biased_gqa import KINDS, Biased, alibi, some

pytestmark = pytest.mark.gpu

LOW, HIGH = -2 ** 31, 2 ** 31 - 1


def run_with(b, doc, prefix):
    """The call with these values; the batch keeps the equal ones that the check
    can count over (no document below token 0, no prefix at or below it)."""
    b.doc, b.prefix = None if doc is None else doc.astype(np.int32), None if prefix is None else prefix.astype(np.int32)
    out = b.run()
    b.doc = None if doc is None else np.maximum(b.doc, 0)
    b.prefix = None if prefix is None else np.maximum(b.prefix, 0)
    return out


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [3, 60, 1400])
@pytest.mark.parametrize("low", [LOW, LOW + 1, LOW + 255, -1, 0])
def test_lowest_ends(kind, rows, low):
    """Lowest values are no prefix and no document, in a row alone and in all of
    them, with a window and documents beside them."""
    b = Biased([rows + 300], [rows], hq=8, hkv=2, page=16, kind=kind, seed=1)
    b.setup(cap=20.0, slopes=alibi(8), window=250)
    pick = some(rows, 12)
    odd = np.arange(rows) % 7 == 1
    every = np.ones(rows, bool)
    for where in (odd, every):
        doc = np.where(np.arange(rows) % 3 == 2, low, 200)
        prefix = np.where(where, low, np.minimum(b.pos + 40, rows + 300))
        b.check(run_with(b, doc, prefix), pick + [1])
    b.check(run_with(b, None, np.where(odd, low, 290)), pick)
    assert Q.check_errors() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [3, 60, 1400])
@pytest.mark.parametrize("high", [HIGH, HIGH - 255, HIGH - 256])
def test_highest_ends(kind, rows, high):
    """A document that begins there leaves a row nothing, a prefix that ends there
    the table's tokens, the others counted."""
    context = rows + 300 + (-(rows + 300)) % 32  # (the table's last page is full)
    b = Biased([context], [rows], hq=4, hkv=1, page=32, block=32, kind=kind, seed=2)
    b.setup(slopes=alibi(4) * 0.1)
    odd = np.arange(rows) % 5 == 1
    out = run_with(b, np.where(odd, high, 0), None)
    assert Q.check_errors() == 0
    assert (out[odd[:rows].nonzero()[0]] == 0).all()
    b.check(out, [i for i in some(rows, 12) if not odd[i]])
    out = run_with(b, None, np.where(odd, high, 0))
    assert Q.check_errors() > 0
    b.prefix = np.where(odd, context, 0)
    b.check(out, some(rows, 12) + [1])
    # (nothing lies from that document on)
    out = run_with(b, np.where(odd, high, 0), np.where(odd, high, 0))
    assert (out[odd[:rows].nonzero()[0]] == 0).all()
    b.check(out, [i for i in some(rows, 8) if not odd[i]])
    Q.check_errors()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("reqs", [6, 40])
def test_starts_that_step_back_across_the_integers(kind, reqs):
    """Requests whose starts are outside the call are counted and have no rows,
    those beside them theirs; in window calls too."""
    b = Biased([1500] + [16] * (reqs - 2) + [900], [1300] + [0] * (reqs - 2) + [700], hq=8, hkv=1, page=16, kind=kind, seed=3, pad=2)
    b.setup(cap=20.0)
    b.qsl[2], b.qsl[3] = HIGH, -10  # 1300 .. HIGH, HIGH .. -10, -10 .. 1300
    out = b.run()
    assert Q.check_errors() > 0
    b.check(out, some(b.n, 20))
    b.d["out"].fill_(7.0)
    out = b.window(500, 4)
    assert Q.check_errors() > 0
    b.check_window(out, 500, 4, some(b.n, 20))
