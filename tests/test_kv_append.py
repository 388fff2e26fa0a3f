"""qsa_kv_append on GB300 against the oracle: keys and values into caches of
every type, runs and re-encoding of blocks with scales, odd rows."""

import numpy as np
import pytest
import torch

from learned_sparse_attention_gb300 import qsa as Q
from learned_sparse_attention_gb300 import workloads as W
from oracle import qsa_oracle as O
from tests.oracle_io import f64

pytestmark = pytest.mark.gpu

D = 128


class Case:
    """A projection, its positions and slots, and a cache of `blocks` pages."""

    def __init__(self, rows, hq=4, hkv=2, page=64, blocks=6, block=32, mrope=False, seed=0, loud=None):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.hq, self.hkv, self.page, self.blocks, self.block = rows, hq, hkv, page, blocks, block
        self.sections = (8, 12, 12) if mrope else (0, 0, 0)
        self.qkv = torch.randn((rows, (2 * hq + 2 * hkv) * D), generator=g).bfloat16()
        if loud is not None:
            self.qkv *= loud(rows)[:, None]
        self.wq = (torch.randn(D, generator=g) * 0.1).bfloat16()
        self.wk = (torch.randn(D, generator=g) * 0.1).bfloat16()
        self.cos_sin = W.rope_cos_sin(4096, 64)
        pos = torch.randint(0, 4096, (rows, 1, 3), generator=g)
        self.positions = pos
        self.codes = torch.randint(0, 0x7F, (blocks, hkv, page, 2 * D), generator=g, dtype=torch.uint8)
        self.scales = torch.randint(119, 123, (blocks, hkv, page // block, 2), generator=g, dtype=torch.uint8)

    def cfg(self, dtype):
        return (Q.make_cfg(8, 4, 64, Q.DTYPE_BF16, 4, 4096, mrope_section=self.sections),
                Q.make_gqa_cfg(self.hq, self.hkv, self.page, self.blocks, kv_dtype=dtype, k_scale=0.0625, v_scale=0.125))

    def tensors(self, kv, slots, query, lo=0, hi=None):
        hi = self.rows if hi is None else hi
        t = dict(main_qkv=self.qkv[lo:hi].cuda(), main_k_norm_w=self.wk.cuda(), kv=kv,
                 slot_mapping=torch.as_tensor(slots, dtype=torch.int64).cuda())
        if query:
            t.update(main_q_norm_w=self.wq.cuda(),
                     main_q_out=torch.full((hi - lo, self.hq, D), 7.0, dtype=torch.bfloat16, device="cuda"),
                     main_gate_out=torch.full((hi - lo, self.hq, D), 7.0, dtype=torch.bfloat16, device="cuda"))
        return t

    def oracle_kv(self):
        cfg = O.QsaConfig(n_heads=8, head_dim=D, rotary_dim=64, compress_ratio=4, token_topk=64, eps=1e-6, index_dtype=0,
                          mrope_section=self.sections, state_size=8, cpage=4)
        pos, cs = self.positions.numpy().reshape(-1, 3), f64(self.cos_sin)
        k, v = np.empty((self.rows, self.hkv, D)), np.empty((self.rows, self.hkv, D))
        for i in range(self.rows):
            k[i], v[i] = O.prepare_main_row(cfg, f64(self.qkv[i]), pos[i], cs, f64(self.wq), f64(self.wk), 1e-6,
                                            self.hq, self.hkv)[2:]
        return k, v


def run_scaled(c, slots, codes=None, scales=None, query=False, lo=0, hi=None):
    codes = c.codes.cuda() if codes is None else codes
    scales = c.scales.cuda() if scales is None else scales
    cfg, gcfg = c.cfg(Q.DTYPE_E4M3_BLOCK)
    t = c.tensors(codes, slots, query, lo, hi)
    pos = c.positions[lo:c.rows if hi is None else hi].cuda()
    Q.kv_append(cfg, gcfg, Q.main_prep(t), pos, c.cos_sin.cuda(), scales=Q.kv_scales(scales, c.block))
    torch.cuda.synchronize()
    return codes, scales, t


def check_scaled(c, slots, codes, scales, k=None, v=None):
    """The cache against the oracle's: every scale equal; codes equal but for
    values within the fp32 error of a rounding midpoint, one step apart there;
    everything that no run touches as it was."""
    if k is None:
        k, v = c.oracle_kv()
    want_c, want_s = c.codes.numpy().copy(), c.scales.numpy().copy()
    O.append_block_kv(want_c, want_s, np.asarray(slots), k, v, c.page, c.block)
    got_c, got_s = codes.cpu().numpy(), scales.cpu().numpy()
    assert np.array_equal(got_s, want_s)
    a, b = O.e4m3_decode(got_c), O.e4m3_decode(want_c)
    assert np.array_equal(np.isnan(a), np.isnan(b))
    a, b = np.nan_to_num(a), np.nan_to_num(b)
    off = a != b
    # fp32 norm and rotation: a few 2^-24 of the value against steps of 2^-3 or
    # more: under one code in 10^5 may sit that near a midpoint
    assert off.mean() <= 1e-5 + 2.0 / off.size
    step = np.maximum(np.abs(b), 2.0 ** -6) * 2.0 ** -3
    assert (np.abs(a - b)[off] <= step[off] * (1 + 1e-9)).all()


def contiguous_slots(c, first, n):
    return np.arange(first, first + n)


@pytest.mark.parametrize("block,page", [(16, 16), (16, 48), (32, 64), (64, 64), (64, 128), (32, 96)])
@pytest.mark.parametrize("rows,first", [(1, 0), (1, 5), (7, 13), (40, 3), (100, 17)])
def test_runs_of_one_sequence(block, page, rows, first):
    c = Case(rows, page=page, block=block, blocks=10, seed=rows + first)
    slots = contiguous_slots(c, first + page, rows)
    codes, scales, _ = run_scaled(c, slots)
    check_scaled(c, slots, codes, scales)
    assert Q.check_errors() == 0


@pytest.mark.parametrize("hq,hkv,mrope", [(1, 1, False), (16, 1, True), (10, 2, False), (24, 8, True), (9, 9, False)])
def test_heads_and_rotation(hq, hkv, mrope):
    c = Case(37, hq=hq, hkv=hkv, mrope=mrope, seed=hq)
    slots = contiguous_slots(c, 70, 37)
    codes, scales, t = run_scaled(c, slots, query=True)
    check_scaled(c, slots, codes, scales)
    # q and the gate: what the prepare of a bf16 cache gives, bit for bit
    cfg, gcfg = c.cfg(Q.DTYPE_BF16)
    kv = torch.zeros((c.blocks, hkv, c.page, 2 * D), dtype=torch.bfloat16, device="cuda")
    t2 = c.tensors(kv, slots, True)
    Q.main_prepare(cfg, gcfg, Q.main_prep(t2), c.positions.cuda(), c.cos_sin.cuda())
    torch.cuda.synchronize()
    assert torch.equal(t["main_q_out"], t2["main_q_out"])
    assert torch.equal(t["main_gate_out"], t2["main_gate_out"])
    assert Q.check_errors() == 0


@pytest.mark.parametrize("dtype", [Q.DTYPE_BF16, Q.DTYPE_E4M3])
@pytest.mark.parametrize("query", [True, False])
@pytest.mark.parametrize("rows", [1, 33, 1500])
def test_plain_caches_match_the_prepare(dtype, query, rows):
    c = Case(rows, hq=10, hkv=5, blocks=30, seed=rows)
    slots = np.random.default_rng(rows).permutation(30 * 64)[:rows].copy()
    slots[rows // 2] = -1
    cfg, gcfg = c.cfg(dtype)
    kv0 = torch.randint(0, 0x7F, (30, 5, 64, 2 * D * (2 if dtype == Q.DTYPE_BF16 else 1)), dtype=torch.uint8)
    caches = []
    for call in ("append", "prepare"):
        kv = kv0.cuda().view(torch.bfloat16) if dtype == Q.DTYPE_BF16 else kv0.cuda()
        t = c.tensors(kv, slots, query or call == "prepare")
        if call == "append":
            Q.kv_append(cfg, gcfg, Q.main_prep(t), c.positions.cuda(), c.cos_sin.cuda())
        else:
            Q.main_prepare(cfg, gcfg, Q.main_prep(t), c.positions.cuda(), c.cos_sin.cuda())
        torch.cuda.synchronize()
        caches.append((kv.view(torch.uint8), t))
    assert torch.equal(caches[0][0], caches[1][0])
    if query:
        assert torch.equal(caches[0][1]["main_q_out"], caches[1][1]["main_q_out"])
        assert torch.equal(caches[0][1]["main_gate_out"], caches[1][1]["main_gate_out"])
    assert Q.check_errors() == 0


@pytest.mark.parametrize("block", [16, 64])
def test_a_sequence_token_by_token(block):
    """Loudness grows along the sequence, so that blocks are re-encoded again
    and again; the oracle follows call by call."""
    n = 90
    c = Case(n, block=block, seed=3, loud=lambda r: torch.logspace(-3, 3, r).bfloat16())
    k, v = c.oracle_kv()
    codes, scales = c.codes.cuda(), c.scales.cuda()
    want_c, want_s = c.codes.numpy().copy(), c.scales.numpy().copy()
    slots = contiguous_slots(c, 64, n)
    at = 0
    for m in [1] * 20 + [3, 5, 2, 17, 1, 30, 12]:
        run_scaled(c, slots[at:at + m], codes, scales, lo=at, hi=at + m)
        O.append_block_kv(want_c, want_s, slots[at:at + m], k[at:at + m], v[at:at + m], c.page, block)
        at += m
    assert at == n
    assert np.array_equal(scales.cpu().numpy(), want_s)
    a, b = O.e4m3_decode(codes.cpu().numpy()), O.e4m3_decode(want_c)
    off = a != b
    assert off.mean() <= 1e-4  # a flipped code stays flipped through later re-encodings
    assert (np.abs(a - b)[off] <= (np.maximum(np.abs(b), 2.0 ** -6) * 2.0 ** -3)[off] * 2).all()
    # what the cache stands for is near what was appended: half a step of e4m3
    # at the final scale for each rounding, the subnormal step below that
    val = O.dequantise_block_kv(codes.cpu().numpy(), scales.cpu().numpy(), block)
    for i in range(n):
        blk, o = slots[i] // 64, slots[i] % 64
        for h in range(2):
            for w, x in enumerate((k, v)):
                s = float(O.scale_value(scales.cpu().numpy()[blk, h, o // block, w]))
                d = np.abs(val[blk, h, o, w * D:(w + 1) * D] - x[i, h])
                # later re-encodings round only among the subnormals: each adds at most 2^-10 of its
                # scale, and the scales double at the least: twice the last one's in all
                assert (d <= np.abs(x[i, h]) * 2.0 ** -4 * (1 + 2.0 ** -10) + s * 2.0 ** -9).all()


@pytest.mark.parametrize("rows_per_req", [[1] * 40, [4] * 9, [700, 1, 65, 1000], [1024]])
def test_batches(rows_per_req):
    """Requests on their own pages, each at its own place inside a block."""
    rng = np.random.default_rng(len(rows_per_req))
    page, slots, blk = 64, [], 0
    perm = rng.permutation(60)
    for n in rows_per_req:
        start = int(rng.integers(0, 64))
        tok = np.arange(start, start + n)
        need = tok[-1] // page + 1
        slots.append(perm[blk + tok // page] * page + tok % page)
        blk += need
    slots = np.concatenate(slots)
    c = Case(len(slots), blocks=60, hkv=3, hq=3, seed=7)
    codes, scales, _ = run_scaled(c, slots)
    check_scaled(c, slots, codes, scales)
    assert Q.check_errors() == 0


def test_padding_bad_and_repeated_slots():
    c = Case(12, seed=9)
    slots = np.array([70, 71, -1, 72, 6 * 64, 80, 80, 81, -1, 200, 199, 201])
    # 72 and the first 80 begin runs in the block of the last row before them,
    # 6 * 64 is past the cache, the second 80 repeats and 199 steps back: none is
    # written, nor is what goes on with them
    codes, scales, _ = run_scaled(c, slots)
    assert Q.check_errors() == 5
    want = slots.copy()
    want[4] = -1
    k, v = c.oracle_kv()
    check_scaled(c, want, codes, scales, k, v)


def test_gaps_inside_a_block():
    """Ascending slots that are not adjacent are one run."""
    c = Case(5, seed=10)
    slots = np.array([64, 66, 67, 90, 96])
    codes, scales, _ = run_scaled(c, slots)
    check_scaled(c, slots, codes, scales)
    assert Q.check_errors() == 0


def test_zeros_infinities_nan_and_range():
    c = Case(6, hq=1, hkv=1, seed=11)
    v0 = (2 * 1 + 1) * D
    c.qkv[0, v0:] = 0                      # an all-zero V: the smallest scale
    c.qkv[1, v0:v0 + 3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    c.qkv[2, v0:] = 3e38                   # beyond 448 * 2^40: saturates
    c.qkv[3, v0:] = 448.0                  # exactly at a border
    c.qkv[4, v0:] = 450.0
    c.qkv[5, v0:] = 1e-30
    slots = np.arange(6) * 32              # a block each
    codes, scales, _ = run_scaled(c, slots)
    check_scaled(c, slots, codes, scales)
    s = scales.cpu().numpy()[:, 0, :, 1].reshape(-1)[:6]
    assert s[0] == 87 and s[2] == 167 and s[3] == 127 and s[4] == 128 and s[5] == 87
    got = codes.cpu().numpy()[0, 0, 32, D:D + 3]
    assert got[0] == 0x7E and got[1] == 0xFE and got[2] & 0x7F == 0x7F


def test_captured_and_replayed():
    """The same call as a graph, replayed on new inputs."""
    c = Case(40, seed=12)
    codes, scales = c.codes.cuda(), c.scales.cuda()
    cfg, gcfg = c.cfg(Q.DTYPE_E4M3_BLOCK)
    slots = contiguous_slots(c, 64, 40)
    t = c.tensors(codes, slots, True)
    m, sc = Q.main_prep(t), Q.kv_scales(scales, c.block)
    pos, cs = c.positions.cuda(), c.cos_sin.cuda()
    Q.kv_append(cfg, gcfg, m, pos, cs, scales=sc)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.kv_append(cfg, gcfg, m, pos, cs, scales=sc)
    c2 = Case(40, seed=13)
    t["main_qkv"].copy_(c2.qkv)
    pos.copy_(c2.positions)
    codes.copy_(c2.codes)
    scales.copy_(c2.scales)
    graph.replay()
    torch.cuda.synchronize()
    c2.wq, c2.wk = c.wq, c.wk
    check_scaled(c2, slots, codes, scales)


@pytest.mark.parametrize("rows", [40, 1100])
def test_on_another_stream(rows):
    """The call's work, queries included, is done when its stream is."""
    c = Case(rows, blocks=60, seed=14)
    slots = contiguous_slots(c, 32, rows)
    codes, scales = c.codes.cuda(), c.scales.cuda()
    t = c.tensors(codes, slots, True)
    m, sc, pos, cs = Q.main_prep(t), Q.kv_scales(scales, c.block), c.positions.cuda(), c.cos_sin.cuda()
    cfg, gcfg = c.cfg(Q.DTYPE_E4M3_BLOCK)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Q.kv_append(cfg, gcfg, m, pos, cs, scales=sc, stream=s)
    s.synchronize()
    got = t["main_q_out"].clone()
    check_scaled(c, slots, codes, scales)
    codes2, scales2 = c.codes.cuda(), c.scales.cuda()
    t2 = c.tensors(codes2, slots, True)
    Q.kv_append(cfg, gcfg, Q.main_prep(t2), pos, cs, scales=Q.kv_scales(scales2, c.block))
    torch.cuda.synchronize()
    assert torch.equal(got, t2["main_q_out"]) and torch.equal(codes, codes2) and torch.equal(scales, scales2)
    assert Q.check_errors() == 0


@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("hkv", [1, 3])
def test_many_short_runs(block, hkv):
    """1200 rows, most of them runs of their own: one to three rows each in
    some scale block, in any order."""
    rng = np.random.default_rng(block + hkv)
    c = Case(1200, hq=hkv, hkv=hkv, blocks=1200 * block // 64 + 1, block=block, seed=15)
    where = rng.permutation(c.blocks * 64 // block)
    slots, at = [], 0
    while len(slots) < 1200:  # (padding only between runs: inside one it would part it in two)
        n, first = rng.integers(1, 4), rng.integers(0, block - 3)
        slots += [where[at] * block + first + k if at % 30 else -1 for k in range(n)]
        at += 1
    slots = np.array(slots[:1200])
    codes, scales, _ = run_scaled(c, slots)
    check_scaled(c, slots, codes, scales)
    assert Q.check_errors() == 0


@pytest.mark.parametrize("rows", [70, 1100])
def test_padding_inside_a_sequence_is_refused(rows):
    """What follows padding in the block of the row before it is left out and
    counted, in another block it is a run of its own."""
    c = Case(rows, blocks=60, seed=16)
    slots = contiguous_slots(c, 64, rows)
    slots[10:14] = -1              # 74 .. 77: 78 .. 95 follow in the same block of 32
    slots[30:33] = -1              # 94 .. 96: 97 follows in the next one
    codes, scales, _ = run_scaled(c, slots)
    assert Q.check_errors() == 1
    want = slots.copy()
    want[14:30] = -1
    check_scaled(c, want, codes, scales)
