"""Sizes that the block-scaled cache's and the window attention's calls ask
for: tensors that are too small, workspaces over a range of batches (CPU only;
nothing is launched)."""

import ctypes

import pytest
import torch

from learned_sparse_attention_gb300 import build as B
from learned_sparse_attention_gb300 import qsa as Q


@pytest.fixture(scope="module")
def lib():
    B.build_library()
    return Q.load(build_if_missing=False)


class Elsewhere(torch.Tensor):
    """A tensor that says that it is on another GPU."""

    def get_device(self):
        return 1

    @property
    def device(self):
        return torch.device("cuda", 1)


@pytest.mark.parametrize("query", [True, False])
def test_append_refuses_norm_weights_of_another_size_or_device(query):
    """Both are read whole, q's only where q is asked for."""
    g = Q.make_gqa_cfg(2, 1, 16, 3, kv_dtype=Q.DTYPE_E4M3_BLOCK)
    cfg = Q.make_cfg(8, 4, 64, Q.DTYPE_BF16, 4, 10)
    bf = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)  # noqa: E731
    sc = Q.QsaKvScales()
    sc.scales, sc.scale_block, sc._tensors = 256, 16, torch.zeros(6, dtype=torch.uint8)

    def append(**kw):
        t = dict(main_qkv=bf(4, 6 * 128), main_k_norm_w=bf(128), main_q_norm_w=bf(128),
                 kv=torch.zeros((3, 1, 16, 256), dtype=torch.uint8), slot_mapping=torch.zeros(4, dtype=torch.int64))
        if query:
            t.update(main_q_out=bf(4, 2, 128), main_gate_out=bf(4, 2, 128))
        t.update(kw)
        m = Q.QsaMainPrep()
        m._tensors, m._entries = t, Q._main_entries(t)
        Q.kv_append(cfg, g, m, torch.zeros((4, 1, 3), dtype=torch.int64), torch.zeros(10, 64), scales=sc)

    with pytest.raises(ValueError, match="CUDA"):  # (the sizes are right: host tensors all the same)
        append()
    for name in ["main_k_norm_w"] + ["main_q_norm_w"] * query:
        with pytest.raises(ValueError, match=f"{name} has 127 entries"):
            append(**{name: bf(127)})
        with pytest.raises(ValueError, match=f"{name} is on cuda:1"):
            append(**{name: bf(128).as_subclass(Elsewhere)})
    if not query:
        for w in (bf(127), bf(128).as_subclass(Elsewhere), None):
            with pytest.raises(ValueError, match="CUDA"):
                append(main_q_norm_w=w)


GROUPS = [(8, 1), (32, 4), (3, 3), (64, 4), (5, 1), (16, 8)]


@pytest.mark.parametrize("dtype", [Q.DTYPE_BF16, Q.DTYPE_E4M3, Q.DTYPE_E4M3_BLOCK])
@pytest.mark.parametrize("hq,hkv", GROUPS)
def test_window_workspace_of_a_large_batch_serves_smaller_ones(lib, dtype, hq, hkv):
    """The size never falls as rows or tokens grow, and is the same for any
    number of requests.  (64 rows of 4100 tokens and one KV head join without
    scratch, 16 of them need 1 MB.)"""
    g = Q.make_gqa_cfg(hq, hkv, 64, 1000, kv_dtype=dtype)

    def size(rows, reqs, tokens):
        a = Q.QsaWindowArgs()
        a.rows, a.reqs, a.window, a.sinks, a.max_context = rows, reqs, tokens // 2, tokens - tokens // 2, 1 << 20
        n = lib.qsa_window_workspace_bytes(ctypes.byref(g), ctypes.byref(a))
        a.window, a.sinks, a.max_context = 1 << 30, 1 << 30, tokens
        assert lib.qsa_window_workspace_bytes(ctypes.byref(g), ctypes.byref(a)) == n
        return n

    rows = [1, 2, 3, 4, 5, 7, 8, 9, 16, 31, 32, 33, 64, 65, 100, 256, 257, 1000, 5000, 40000]
    tokens = [0, 1, 100, 255, 256, 300, 516, 900, 1300, 2051, 4100, 9000, 32772, 200000]
    table = [[size(r, 1, t) for t in tokens] for r in rows]
    for i, r in enumerate(rows):
        for j, t in enumerate(tokens):
            assert table[i][j] >= max(table[max(i - 1, 0)][j], table[i][max(j - 1, 0)]), (r, t)
            assert {size(r, n, t) for n in (1, 2, r, 10000)} == {table[i][j]}
    assert table[-1][-1] > 0 and max(map(max, table)) < 1 << 26


@pytest.mark.parametrize("hq,hkv", GROUPS)
def test_selection_workspace_of_a_large_batch_serves_smaller_ones(lib, hq, hkv):
    g = Q.make_gqa_cfg(hq, hkv, 64, 1000, kv_dtype=Q.DTYPE_E4M3_BLOCK)

    def size(rows, topk):
        cfg = Q.make_cfg(8, 4, topk, Q.DTYPE_BF16, 4, 1)
        return Q.workspace_bytes(cfg, g, rows, 1, 0)

    rows = [1, 2, 3, 4, 7, 8, 16, 33, 64, 100, 256, 257, 1000, 5000]
    topk = [4, 64, 256, 512, 1024, 2048, 4096, 8192, 100000]
    for i, r in enumerate(rows):
        for j, t in enumerate(topk):
            assert size(r, t) >= max(size(rows[max(i - 1, 0)], t), size(r, topk[max(j - 1, 0)])), (r, t)
