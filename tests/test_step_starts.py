"""A layer step of single rows whose query_start_loc names rows outside the call."""

import numpy as np
import pytest
import torch

from learned_sparse_attention_gb300 import qsa as Q
from learned_sparse_attention_gb300 import workloads as W
from tests.gpu_harness import Step

pytestmark = pytest.mark.gpu

SPECS = {
    "tiny": W.named_spec("tiny_bf16"),
    "e4m3": W.small_spec("starts_e4m3", seed=41, contexts=(1999, 4096, 777, 2500), rows_per_req=(1, 1, 1, 1), n_heads=32,
                         index_dtype=W.DTYPE_E4M3, compress_ratio=4, token_topk=256, hq=32, hkv=4, page=64),
}


@pytest.mark.parametrize("spec", sorted(SPECS))
@pytest.mark.parametrize("start", [2 ** 31 - 1, 1 << 20, -1, -2 ** 31])
def test_starts_outside_the_call_are_counted(spec, start):
    """No key is pooled for such a request; rows of the others are what they were."""
    wl = W.make_workload(SPECS[spec], device="cuda")
    good = Step(wl).run()
    assert Q.check_errors() == 0
    want, packed = good.out.clone(), good.packed.clone()
    wl = W.make_workload(SPECS[spec], device="cuda")
    t = wl.t["query_start_loc"]
    t[1] = start  # request 0 ends and request 1 begins there
    got = Step(wl).run()
    assert Q.check_errors() > 0
    rest = np.arange(2, SPECS[spec].rows)
    assert torch.equal(got.out[rest], want[rest]) and torch.equal(got.packed[rest], packed[rest])
    assert torch.isfinite(got.out.float()).all()
    assert int(t[1]) == start
