"""The tile kernel of qsa_window_gqa on GB300 against float64 rows: sizes at
which `window_plan` (csrc/abi.cu) takes tiles, and the same calls at sizes at
which it takes single rows."""

import numpy as np
import pytest
import torch

from learned_sparse_attention_gb300 import qsa as Q
from oracle import qsa_oracle as O
from tests.attention_bounds import assert_row
from tests.oracle_io import f64
from tests.test_window_gqa import Batch, D

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "block"]


def check_rows(b, out, rows, window, sinks, lost=()):
    """Rows against the tokens they see, those of `lost` left out."""
    for i in rows:
        tok = O.window_tokens(int(b.pos[i]), window, sinks)
        tok = tok[~np.isin(tok, lost)]
        K, V = b.values(int(b.t2r[i]), tok)
        assert_row(out[i], f64(b.q[i]), K, V, None if b.gate is None else f64(b.gate[i]), f"row {i} p {b.pos[i]}")


def some(n, k=24, seed=0):
    return sorted(set(np.random.default_rng(seed).choice(n, min(n, k), replace=False).tolist()) | {0, n - 1})


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [1, 70, 1000])
@pytest.mark.parametrize("first", [5000, 1290])
def test_sinks_of_rows_whose_windows_pass_the_table(kind, rows, first):
    """Tokens past the table are left out and counted; the sinks in it are not
    among them, whether the windows end in the table or begin behind it."""
    b = Batch([320], [rows], kind=kind, page=32, block=32, seed=21, hq=2, hkv=1, gate=False)
    b.pos[:] = first + np.arange(rows)
    out = b.window(1000, 40, max_context=first + rows)
    assert Q.check_errors() > 0
    check_rows(b, out, some(rows), 1000, 40, lost=np.arange(320, first + rows))
