"""qsa_biased_gqa on GB300: batches of many requests against float64 rows, and a
workspace that calls of all sizes share."""

import numpy as np
import pytest
import torch

from learned_sparse_attention_gb300 import qsa as Q
from tests.test_biased_gqa import KINDS, Biased, alibi, some

pytestmark = pytest.mark.gpu


def ragged(reqs, most, seed):
    """Rows and contexts of requests, every fifth of them without rows."""
    rng = np.random.default_rng(seed)
    rows = [0 if i % 5 == 3 else int(rng.integers(1, most + 1)) for i in range(reqs)]
    return [r + int(rng.integers(1, 700 if reqs < 1000 else 100)) for r in rows], rows


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("reqs,most,hq,hkv,page", [
    (33, 130, 8, 2, 16), (70, 90, 6, 1, 48), (150, 40, 16, 1, 32), (1300, 60, 8, 1, 16),  # tiles
    (40, 2, 8, 2, 16), (700, 1, 4, 1, 32), (1300, 3, 32, 2, 16)])                             # single rows
@pytest.mark.parametrize("scores", range(3))
def test_many_requests(kind, reqs, most, hq, hkv, page, scores):
    contexts, rows = ragged(reqs, most, reqs)
    b = Biased(contexts, rows, hq=hq, hkv=hkv, page=page, block=16, kind=kind, seed=scores, pad=3)
    b.setup(**[dict(cap=30.0, prefix=lambda r, p: min(p + 30, contexts[r]) if r >= 0 and r % 2 else 0),
               dict(slopes=alibi(hq), doc=lambda r, p: p // 200 * 200), dict(cap=10.0, slopes=alibi(hq), window=150)][scores])
    out = b.run()
    assert Q.check_errors() == 0
    ends = np.cumsum([r for r in rows if r])
    b.check(out, sorted(set(some(b.n, 30)) | set((ends - 1)[::7].tolist())))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv", [(8, 1), (8, 2)])
def test_one_workspace_for_calls_of_all_sizes(kind, hq, hkv):
    """In a buffer for the largest one, with more behind it that stays as it was,
    calls give what they give in one of their own size, to the bit."""
    b = Biased([4100], [256], hq=hq, hkv=hkv, kind=kind, page=64, block=32, seed=21)
    b.table = b.table.repeat(256, 0)
    d = b.to_gpu()
    slopes = torch.tensor(alibi(hq), dtype=torch.float32, device="cuda") * 0.1

    def args(rows, reqs, context, **kw):
        qsl = torch.arange(reqs + 1, dtype=torch.int32, device="cuda") * (rows // reqs)
        t2r = torch.arange(rows, dtype=torch.int32, device="cuda") // (rows // reqs)
        pos = context - rows // reqs + torch.arange(rows, dtype=torch.int32, device="cuda") % (rows // reqs)
        return Q.biased_args(d["q"][:rows], d["kv"], d["table"], t2r, qsl, pos, torch.empty_like(d["q"][:rows]), context,
                             gate=d["gate"][:rows], scales=b.sc, **kw)

    def run(a, ws):
        a._tensors[7].fill_(float("nan"))
        Q.biased_gqa(b.gcfg(), a, ws)
        return a._tensors[7].clone()

    most, behind = Q.biased_workspace_bytes(b.gcfg(), args(256, 256, 4100, window=100)), 1 << 16
    buffer = torch.full((most + behind,), 0xFF, dtype=torch.uint8, device="cuda")
    whole = torch.full((256,), 300, dtype=torch.int32, device="cuda")
    for rows, reqs in [(256, 256), (256, 64), (256, 1), (64, 64), (64, 2), (48, 1), (16, 16), (8, 8), (5, 5), (4, 1), (1, 1)]:
        for context in (4100, 1100, 300):
            for kw in (dict(softcap=30.0), dict(window=700, slopes=slopes), dict(prefix_end=whole[:rows], window=50, softcap=5.0, slopes=slopes)):
                a = args(rows, reqs, context, **kw)
                own = Q.biased_workspace_bytes(b.gcfg(), a)
                assert own <= most
                first = run(a, buffer[:most])
                alone = torch.full((own + behind,), 0xFF, dtype=torch.uint8, device="cuda")
                second = run(a, alone[:own] if own else None)
                assert torch.isfinite(first.float()).all() and torch.equal(first, second), (rows, reqs, context)
                assert (alone[own:] == 0xFF).all()
    assert (buffer[most:] == 0xFF).all() and Q.check_errors() == 0
