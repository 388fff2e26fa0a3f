"""Sizes that the block-scaled cache's and the window attention's calls ask
for: tensors that are too small, workspaces over a range of batches (CPU only;
nothing is launched)."""

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
