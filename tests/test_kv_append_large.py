"""Large and captured calls of qsa_kv_append on GB300."""

import numpy as np
import pytest
import torch

from learned_sparse_attention_gb300 import qsa as Q
from oracle import qsa_oracle as O
from tests.test_kv_append import Case, D, contiguous_slots

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [Q.DTYPE_BF16, Q.DTYPE_E4M3])
@pytest.mark.parametrize("query", [True, False])
def test_a_prompt_into_plain_caches_matches_the_prepare(dtype, query):
    """16 384 rows, bit for bit."""
    rows, page = 16384, 64
    c = Case(rows, hq=8, hkv=2, blocks=rows // page + 1, mrope=True, seed=1)
    slots = contiguous_slots(c, 17, rows)
    slots[[0, 77, 8000]] = -1
    cfg, gcfg = c.cfg(dtype)
    shape = (c.blocks, c.hkv, page, 2 * D * (2 if dtype == Q.DTYPE_BF16 else 1))
    kv0 = torch.randint(0, 0x7F, shape, generator=torch.Generator().manual_seed(2), dtype=torch.uint8)
    got = []
    for call in (Q.kv_append, Q.main_prepare):
        kv = kv0.cuda().view(torch.bfloat16) if dtype == Q.DTYPE_BF16 else kv0.cuda()
        t = c.tensors(kv, slots, query or call is Q.main_prepare)
        call(cfg, gcfg, Q.main_prep(t), c.positions.cuda(), c.cos_sin.cuda())
        torch.cuda.synchronize()
        got.append((kv.view(torch.uint8), t))
    assert torch.equal(got[0][0], got[1][0])
    if query:
        assert torch.equal(got[0][1]["main_q_out"], got[1][1]["main_q_out"])
        assert torch.equal(got[0][1]["main_gate_out"], got[1][1]["main_gate_out"])
    assert Q.check_errors() == 0


def test_many_rows_captured_twice_and_replayed():
    """Calls of two launches, two in one graph that write one after the other
    into the same cache, replayed on new inputs."""
    rows = 1100
    c = Case(2 * rows, blocks=60, seed=3)
    codes, scales = c.codes.cuda(), c.scales.cuda()
    cfg, gcfg = c.cfg(Q.DTYPE_E4M3_BLOCK)
    slots = contiguous_slots(c, 64 + 5, 2 * rows)
    halves = [c.tensors(codes, slots[lo:lo + rows], True, lo, lo + rows) for lo in (0, rows)]
    pos = [c.positions[lo:lo + rows].cuda() for lo in (0, rows)]
    cs, sc = c.cos_sin.cuda(), Q.kv_scales(scales, c.block)
    preps = [Q.main_prep(t) for t in halves]
    graph = torch.cuda.CUDAGraph()
    Q.kv_append(cfg, gcfg, preps[0], pos[0], cs, scales=sc)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for m, p in zip(preps, pos):
            Q.kv_append(cfg, gcfg, m, p, cs, scales=sc)
    c2 = Case(2 * rows, blocks=60, seed=4)
    for t, p, lo in zip(halves, pos, (0, rows)):
        t["main_qkv"].copy_(c2.qkv[lo:lo + rows])
        p.copy_(c2.positions[lo:lo + rows])
    c2.wq, c2.wk = c.wq, c.wk
    k, v = c2.oracle_kv()
    for _ in range(2):
        codes.copy_(c2.codes)
        scales.copy_(c2.scales)
        graph.replay()
    torch.cuda.synchronize()
    assert Q.check_errors() == 0
    # (the second call begins inside a block that the first wrote: one after the other)
    got_c, got_s = codes.cpu(), scales.cpu()
    want_c, want_s = c2.codes.numpy().copy(), c2.scales.numpy().copy()
    for lo in (0, rows):
        O.append_block_kv(want_c, want_s, slots[lo:lo + rows], k[lo:lo + rows], v[lo:lo + rows], c.page, c.block)
    assert np.array_equal(got_s.numpy(), want_s)
    off = O.e4m3_decode(got_c.numpy()) != O.e4m3_decode(want_c)
    assert off.mean() <= 1e-5 + 2.0 / off.size  # (values within the fp32 error of a midpoint)
