"""The tile kernel of qsa_window_gqa on GB300 against float64 rows: sizes at
which `window_plan` (csrc/abi.cu) takes tiles, and the same calls at sizes at
which it takes single rows."""

import numpy as np
import pytest
import torch

from learned_sparse_attention_gb300 import qsa as Q
from oracle import qsa_oracle as O
from tests.attention_bounds import assert_row, attend_row
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


def far_apart(kind, rows, seed, page=32):
    """One request, half of its rows from position 1000 and half from 20000 on,
    with windows of 1000: nobody sees tokens 1000 + rows // 2 .. 19000."""
    b = Batch([20000 + rows - rows // 2], [rows], kind=kind, page=page, block=16, seed=seed, hq=2, hkv=1, gate=False)
    half = rows // 2
    b.pos[:] = np.r_[1000 + np.arange(half), 20000 + np.arange(rows - half)]
    return b, (1000 + half + page - 1) // page, 19001 // page  # and the first and last + 1 of the unseen pages


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [70, 1001])
def test_pages_between_rows_far_apart_may_be_gone(kind, rows):
    b, p0, p1 = far_apart(kind, rows, 22)
    b.table[0, p0:p1] = -1
    out = b.window(1000, 3)
    assert Q.check_errors() == 0
    check_rows(b, out, some(rows) + [rows // 2 - 1, rows // 2], 1000, 3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [70, 1001])
def test_odd_values_that_no_row_sees_take_no_room(kind, rows):
    """NaN in more than 32 stretches of 128 tokens between two groups of rows,
    and one more that some rows see."""
    b, p0, p1 = far_apart(kind, rows, 23)
    bad = float("nan") if kind == "bf16" else 0x7F
    b.kv[torch.from_numpy(b.table[0, p0:p1].astype(np.int64)), :, :, D:] = bad
    tok = 19000 + rows // 4  # left by the window on the way through the later rows
    b.kv[b.table[0, tok // 32], 0, tok % 32, D + 9] = bad
    out = b.window(1000, 3)
    assert Q.check_errors() == 0
    sees = (b.pos - 1000 < tok) & (tok <= b.pos)
    assert sees.any() and not sees.all()
    assert np.isnan(out[sees][:, :, 9]).all()
    assert np.isfinite(out[sees][:, :, np.arange(D) != 9]).all() and np.isfinite(out[~sees]).all()
    check_rows(b, out, [i for i in some(rows) + [rows // 2 - 1] if not sees[i]], 1000, 3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [60, 2000])
def test_sinks_alone_need_no_other_pages(kind, rows):
    b = Batch([rows], [rows], kind=kind, page=16, block=16, seed=24, hq=2, hkv=1, gate=False)
    b.table[0, 13:] = -1  # tokens from 208 on: 200 are sinks, the rest unseen
    out = b.window(0, 200)
    assert Q.check_errors() == 0
    check_rows(b, out, some(rows), 0, 200)


@pytest.mark.parametrize("kind", KINDS)
def test_bad_pages_in_tiles_are_left_out_and_counted(kind):
    b = Batch([4300], [4000], kind=kind, page=16, block=16, seed=25, hq=2, hkv=1, gate=False)
    b.table[0, 16], b.table[0, 100] = b.blocks + 5, -1
    out = b.window(64, 0)
    assert Q.check_errors() > 0
    near = list(range(40)) + list(range(1595 - 300, 1685 - 300, 3))
    check_rows(b, out, near + some(4000), 64, 0, lost=np.r_[256:272, 1600:1616])


@pytest.mark.parametrize("kind", KINDS)
def test_odd_values_in_tiles_reach_only_rows_that_see_them(kind):
    """Tokens that enter and leave the windows during the call."""
    b = Batch([4300], [4000], kind=kind, page=16, block=16, seed=26, hq=2, hkv=1, gate=False)
    toks = [240, 299, 1000, 1001, 2047, 2048, 4299]
    for t in toks:
        b.kv[b.table[0, t // 16], 0, t % 16, D + 5] = float("inf") if kind == "bf16" else 0xFF
        b.kv[b.table[0, t // 16], 0, t % 16, D + 9] = float("nan") if kind == "bf16" else 0x7F
    out = b.window(64, 0)
    assert Q.check_errors() == 0
    sees = np.zeros(4000, dtype=bool)
    for t in toks:
        sees |= (b.pos - 64 < t) & (t <= b.pos)
    clean = ~np.isin(np.arange(D), [5, 9])
    assert np.isnan(out[sees][:, :, 9]).all() and not np.isfinite(out[sees][:, :, 5]).any()
    assert np.isfinite(out[sees][:, :, clean]).all() and np.isfinite(out[~sees]).all()
    edge = [i for t in toks for p in (t - 1, t + 63, t + 64) for i in [p - 300] if 0 <= i < 4000]
    check_rows(b, out, [i for i in edge + some(4000) if not sees[i]], 64, 0)


@pytest.mark.parametrize("kind", ["e4m3", "block"])
@pytest.mark.parametrize("rows", [8, 1000])
def test_queries_with_one_loud_element(kind, rows):
    """Elements down to 2^-11 of their head's largest keep all their bits: keys
    that are blind to the loud one and weigh the others' last bits against each
    other get scores that are fp32 sums of exact products.  (Rounded to steps
    of 2^-19 of the largest, these elements would double the scores.)"""
    b = Batch([1300], [rows], kind=kind, page=64, block=32, seed=27, hq=2, hkv=1, gate=False)
    rng = np.random.default_rng(3)
    q = np.where(np.arange(D) % 2 == 0, 0.5 + 2.0 ** -8, 0.5 + 3 * 2.0 ** -8)
    q[17] = 1000.0
    b.q = (torch.from_numpy(q) * torch.from_numpy(rng.choice([-1.0, 1.0], (rows, 2, 1)))).bfloat16()
    key = np.where(np.arange(D) % 2 == 0, 1.0, -1.0)
    key[17] = 0.0
    c = rng.choice([-64.0, -32.0, 16.0, 48.0, 64.0], b.kv.shape[:3] + (1,))
    b.kv[..., :D] = torch.from_numpy(c * key).to(torch.float8_e4m3fn).view(torch.uint8)
    b.k_scale = 1.0
    if kind == "block":
        b.scales[..., 0] = 127
    out = b.window(600, 2)
    assert Q.check_errors() == 0
    check_rows(b, out, some(rows), 600, 2)


@pytest.mark.parametrize("kind", ["e4m3", "block"])
@pytest.mark.parametrize("rows", [8, 1000])
@pytest.mark.parametrize("ratio", [2.0 ** 14, 2.0 ** 18])
def test_queries_of_a_wide_range(kind, rows, ratio):
    """Smaller elements are off by at most 2^-21 of their head's largest, so a
    score by 2^-21 max|q| sum|k| / sqrt(D) beyond its bound: every weight moves
    by at most e^2d - 1 of itself, the output by that times sum w|v|."""
    b = Batch([1300], [rows], kind=kind, page=64, block=32, seed=28, hq=2, hkv=1, gate=False)
    b.q[:, :, 17] = ratio
    b.kv[..., 17] = 0
    if kind == "block":
        b.scales[..., 0] = 119
    out = b.window(600, 2)
    assert Q.check_errors() == 0
    for i in some(rows):
        q = f64(b.q[i])
        K, V = b.values(0, O.window_tokens(int(b.pos[i]), 600, 2))
        want, bound = attend_row(q, K, V)
        size = attend_row(q, K, np.abs(V))[0]  # sum w|v|
        d = (np.abs(K[:, 0]).sum(1) / np.sqrt(D)).max() * np.abs(q).max(1) * 2.0 ** -21
        more = np.expm1(2 * d)[:, None] * size * (1 + 2.0 ** -6)
        assert (np.abs(out[i] - want) <= bound * (1 + np.expm1(2 * d)[:, None]) + more).all(), i


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [60, 6000])
def test_odd_queries_that_see_nothing_are_zero(kind, rows):
    """A query that is not finite makes what it sees a NaN, and nothing of a
    window that lies on pages outside the cache."""
    b = Batch([rows + 240], [rows], kind=kind, page=16, block=16, seed=29, hq=2, hkv=1, gate=False)
    b.table[0, 16:18] = b.blocks, -1       # tokens 256 .. 287, the window of position 287
    i = 287 - 240
    b.q[i, 0, 3], b.q[i, 1, 100] = float("nan"), float("inf")
    b.q[i - 1, 0, 3], b.q[7, 1, 5] = float("nan"), float("-inf")
    out = b.window(32, 0)
    assert Q.check_errors() > 0
    assert (out[i] == 0).all()
    assert np.isnan(out[i - 1, 0]).all() and np.isnan(out[7, 1]).all()
    assert np.isfinite(out[i - 1, 1]).all() and np.isfinite(out[7, 0]).all()
    check_rows(b, out, [r for r in some(rows) if r not in (i, i - 1, 7)], 32, 0, lost=np.arange(256, 288))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [5, 1000])
@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 34, 2.0 ** 60])
def test_scores_beyond_fp32_steps_of_one(kind, rows, size):
    """Scores so large that neighbouring fp32 values are further apart than a
    weight's range pick the best token, not an infinity or a NaN."""
    b = Batch([1300], [rows], kind=kind, page=64, block=32, seed=30, hq=2, hkv=1, gate=False)
    b.q *= size / 2.0 ** 15
    if kind == "bf16":
        b.kv[..., :D] *= 2.0 ** 15
    elif kind == "e4m3":
        b.k_scale = 2.0 ** 10
    else:
        b.scales[..., 0] = 127 + 10
    out = b.window(300, 2)
    assert Q.check_errors() == 0 and np.isfinite(out).all()
    checked = 0
    for i in some(rows):
        K, V = b.values(0, O.window_tokens(int(b.pos[i]), 300, 2))
        for h in range(2):
            z = K[:, 0] @ f64(b.q[i])[h] / np.sqrt(D)
            top = np.argsort(z)[-2:]
            # a score's error is at most 2^-24 * 130 of sum |q k| / sqrt(D)
            off = 130 * 2.0 ** -24 * (np.abs(K[:, 0]) @ np.abs(f64(b.q[i])[h])).max() / np.sqrt(D)
            if z[top[1]] - z[top[0]] > 2 * off + 100:
                v = V[top[1], 0]
                assert (np.abs(out[i, h] - v) <= 2.0 ** -8 * np.abs(v) + 1e-30).all(), (i, h)
                checked += 1
    assert checked > len(some(rows))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv", [(8, 1), (8, 2)])
def test_workspace_of_the_largest_call_serves_smaller_ones(kind, hq, hkv):
    """Single rows with one split, joined in a cluster and joined by a second
    launch, tiles with and without splits, in one buffer."""
    b = Batch([4100], [256], hq=hq, hkv=hkv, kind=kind, page=64, block=32, seed=34)
    b.table = b.table.repeat(256, 0)  # (requests that share their pages)
    d = b.to_gpu()

    def args(rows, reqs, context):
        qsl = torch.arange(reqs + 1, dtype=torch.int32, device="cuda") * (rows // reqs)
        t2r = torch.arange(rows, dtype=torch.int32, device="cuda") // (rows // reqs)
        pos = context - rows // reqs + torch.arange(rows, dtype=torch.int32, device="cuda") % (rows // reqs)
        return Q.window_args(d["q"][:rows], d["kv"], d["table"], t2r, qsl, pos, torch.empty_like(d["q"][:rows]), 100000, 0,
                             context, gate=d["gate"][:rows], scales=b.sc)

    most = Q.window_workspace_bytes(b.gcfg(), args(256, 256, 4100))
    shared = torch.full((most,), 0xFF, dtype=torch.uint8, device="cuda")
    for rows, reqs in [(256, 256), (256, 1), (64, 64), (64, 2), (48, 1), (16, 16), (8, 8), (5, 5), (4, 1), (1, 1)]:
        for context in (4100, 1100, 300):
            a = args(rows, reqs, context)
            Q.window_gqa(b.gcfg(), a, shared)
            own = Q.window_workspace_bytes(b.gcfg(), a)
            assert own <= most
            out = a._tensors[7].clone()
            Q.window_gqa(b.gcfg(), a, torch.empty(own, dtype=torch.uint8, device="cuda") if own else None)
            assert torch.equal(out, a._tensors[7]) and not torch.isnan(out.float()).any()
    assert Q.check_errors() == 0


def test_selection_workspace_of_the_largest_call_serves_smaller_ones():
    b = Batch([4200], [256], hq=8, hkv=1, kind="block", page=64, block=32, seed=35)
    b.table, b.t2r = b.table.repeat(256, 0), np.arange(256, dtype=np.int32)
    d = b.to_gpu()
    cfg = Q.make_cfg(8, 4, 4096, Q.DTYPE_BF16, 4, 1)
    ws = torch.full((Q.workspace_bytes(cfg, b.gcfg(), 256, 256, 0),), 0xFF, dtype=torch.uint8, device="cuda")
    for width in (4100, 1028, 260):
        packed = torch.arange(width, dtype=torch.int32, device="cuda").repeat(256, 1)
        packed[:, -1] = width - 1
        for rows in (256, 100, 64, 16, 8, 5, 1):
            Q.sparse_gqa_scaled(b.gcfg(), b.sc, d["q"][:rows], d["kv"], d["table"], packed[:rows], d["t2r"][:rows],
                                d["gate"][:rows], d["out"][:rows], ws)
            for i in {0, rows - 1}:
                K, V = b.values(i, np.arange(width - 1))
                assert_row(f64(d["out"][i]), f64(b.q[i]), K, V, f64(b.gate[i]), f"row {i} of {rows}")
    assert Q.check_errors() == 0


@pytest.mark.parametrize("rows", [8, 1000])
def test_scale_bytes_at_and_past_their_ends(rows):
    """V scales over all of 2^-40 .. 2^40 and bytes outside, which are read as
    the nearest of them; K scales from the ordinary down."""
    b = Batch([1300], [rows], kind="block", page=64, block=16, seed=31, hq=8, hkv=2)
    rng = np.random.default_rng(2)
    b.scales[..., 0] = torch.from_numpy(rng.choice([0, 87, 100, 118, 122], b.scales.shape[:-1]).astype(np.uint8))
    b.scales[..., 1] = torch.from_numpy(rng.choice([0, 87, 100, 127, 140, 167, 255], b.scales.shape[:-1]).astype(np.uint8))
    out = b.window(600, 2)
    assert Q.check_errors() == 0
    check_rows(b, out, some(rows), 600, 2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("splits", [False, True])
def test_tiles_captured_and_replayed(kind, splits):
    """A chunk (of a short context: one split; of a long one: several) as a
    graph, replayed on new rows with another's leavings in the workspace."""
    contexts = [9000] if splits else [700, 650]
    rows = [200] if splits else [700, 500]
    make = lambda seed: Batch(contexts, rows, hq=8, hkv=2, kind=kind, page=64, block=32, seed=seed)  # noqa: E731
    b = make(32)
    b.window(20000, 0)
    d = b.d
    a = Q.window_args(d["q"], d["kv"], d["table"], d["t2r"], d["qsl"], d["pos"], d["out"], 20000, 0, max(contexts),
                      gate=d["gate"], scales=b.sc)
    n = Q.window_workspace_bytes(b.gcfg(), a)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.window_gqa(b.gcfg(), a, ws)
    c = make(33)
    c.to_gpu()
    for k in ("q", "kv", "table", "gate", "scales"):
        if d[k] is not None:
            d[k].copy_(c.d[k])
    ws.fill_(0xFF)
    d["out"].fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    check_rows(c, f64(d["out"]), some(c.n, 12), 20000, 0)
    assert Q.check_errors() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_a_prompt_that_sees_all_before_it(kind):
    """Plain causal attention: windows back to token 0, from a row of one token
    to one of thousands, and a second request that goes on from 900."""
    b = Batch([3500, 1600], [3500, 700], hq=8, hkv=2, kind=kind, page=64, block=32, seed=36)
    out = b.window(2 ** 31 - 1, 0)
    assert Q.check_errors() == 0
    check_rows(b, out, some(b.n, 20) + [1, 127, 128, 3499, 3500], 2 ** 31 - 1, 0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,context", [(1, 700), (1, 1300), (1, 6000), (3, 6000), (40, 6000), (600, 6000)])
def test_odd_values_of_negligible_weight_reach_who_sees_them(kind, rows, context):
    """Half of the tokens weigh less than 2^-126 of the other half's, with an
    odd value among them: single rows and tiles, joined over splits or not."""
    b = Batch([context], [rows], kind=kind, page=64, block=32, seed=37, hq=8, hkv=1, gate=False)
    sign = torch.from_numpy(np.random.default_rng(5).choice([-1.0, 1.0], D))
    b.q[:] = 2 * sign.bfloat16()
    half = (context - rows) // 2
    code = {"bf16": 4.0, "e4m3": 128.0, "block": 4.0}[kind]
    if kind == "block":
        b.scales[..., 0] = 127
    for t in range(context):
        row = (-code if t < half else code) * sign
        k = row.bfloat16() if kind == "bf16" else row.to(torch.float8_e4m3fn).view(torch.uint8)
        b.kv[b.table[0, t // 64], 0, t % 64, :D] = k
    tok = half // 3
    b.kv[b.table[0, tok // 64], 0, tok % 64, D + 9] = float("nan") if kind == "bf16" else 0x7F
    out = b.window(100000, 0)
    assert Q.check_errors() == 0
    assert np.isnan(out[:, :, 9]).all()
    assert np.isfinite(out[:, :, np.arange(D) != 9]).all()
