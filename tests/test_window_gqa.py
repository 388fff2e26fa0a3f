"""Attention over the cache with block scales (qsa_sparse_gqa_scaled) and
window attention (qsa_window_gqa) on GB300 against float64 rows."""

import numpy as np
import pytest
import torch

from learned_sparse_attention_gb300 import qsa as Q
from oracle import qsa_oracle as O
from tests.attention_bounds import assert_row, attend_row
from tests.oracle_io import f64

pytestmark = pytest.mark.gpu

D = 128
KINDS = {"bf16": Q.DTYPE_BF16, "e4m3": Q.DTYPE_E4M3, "block": Q.DTYPE_E4M3_BLOCK}


class Batch:
    """Requests of contexts[i] tokens whose last rows[i] are the call's rows."""

    def __init__(self, contexts, rows, hq=8, hkv=2, page=16, kind="block", block=16, seed=0, pad=0, gate=True, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.contexts, self.rows_per, self.hq, self.hkv, self.page = contexts, rows, hq, hkv, page
        self.kind, self.block = kind, block
        n = sum(rows)
        self.n, self.total = n, n + pad
        need = [max(1, -(-c // page)) for c in contexts]
        self.blocks = sum(need) + 1
        perm = rng.permutation(self.blocks)
        self.table = np.zeros((len(contexts), max(need)), dtype=np.int32)
        at = 0
        for i, b in enumerate(need):
            self.table[i, :b] = perm[at:at + b]
            at += b
        self.t2r = np.concatenate([np.repeat(np.arange(len(rows)), rows), np.full(pad, -1)]).astype(np.int32)
        self.qsl = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.pos = np.concatenate([np.arange(c - r, c) for c, r in zip(contexts, rows)] + [np.zeros(pad)]).astype(np.int32)
        self.q = torch.randn((self.total, hq, D), generator=g).bfloat16() * spread
        self.gate = torch.randn((self.total, hq, D), generator=g).bfloat16() if gate else None
        shape = (self.blocks, hkv, page, 2 * D)
        self.scales = None
        if kind == "bf16":
            self.kv = torch.randn(shape, generator=g).bfloat16()
        else:
            self.kv = (torch.randn(shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            if kind == "block":
                self.scales = torch.randint(118, 123, (self.blocks, hkv, page // block, 2), generator=g, dtype=torch.uint8)
        self.k_scale, self.v_scale = (0.03125, 0.0625) if kind == "e4m3" else (1.0, 1.0)

    def gcfg(self):
        return Q.make_gqa_cfg(self.hq, self.hkv, self.page, self.blocks, kv_dtype=KINDS[self.kind], k_scale=self.k_scale,
                              v_scale=self.v_scale)

    def to_gpu(self):
        self.d = {k: (torch.from_numpy(v) if isinstance(v, np.ndarray) else v).cuda()
                  for k, v in dict(q=self.q, kv=self.kv, table=self.table, t2r=self.t2r, qsl=self.qsl, pos=self.pos).items()}
        self.d["gate"] = self.gate.cuda() if self.gate is not None else None
        self.d["scales"] = self.scales.cuda() if self.scales is not None else None
        self.d["out"] = torch.full((self.total, self.hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.sc = Q.kv_scales(self.d["scales"], self.block) if self.scales is not None else None
        return self.d

    def values(self, req, tok):
        """K, V [n, Hkv, D] of tokens of a request."""
        tok = np.asarray(tok, dtype=np.int64)
        blk, off = self.table[req, tok // self.page], tok % self.page
        raw = self.kv[torch.from_numpy(blk.astype(np.int64)), :, torch.from_numpy(off)]
        x = f64(raw)
        if self.kind == "block":
            s = O.scale_value(self.scales.numpy()[blk, :, off // self.block])  # [n, Hkv, 2]
            x = x * np.repeat(s, D, axis=2)
        k, v = x[..., :D], x[..., D:]
        return k * self.k_scale, v * self.v_scale

    def window(self, window, sinks, ws=None, **kw):
        d = self.to_gpu() if not hasattr(self, "d") else self.d
        a = Q.window_args(d["q"], d["kv"], d["table"], d["t2r"], d["qsl"], d["pos"], d["out"], window, sinks,
                          kw.get("max_context", max(self.contexts)), gate=d["gate"], scales=self.sc)
        n = Q.window_workspace_bytes(self.gcfg(), a)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
        Q.window_gqa(self.gcfg(), a, ws)
        torch.cuda.synchronize()
        return f64(d["out"])

    def check_window(self, out, window, sinks, sample=None):
        rows = range(self.n) if sample is None else sample
        for i in rows:
            tok = O.window_tokens(int(self.pos[i]), window, sinks)
            K, V = self.values(self.t2r[i], tok)
            assert_row(out[i], f64(self.q[i]), K, V, None if self.gate is None else f64(self.gate[i]), f"row {i} p {self.pos[i]}")
        assert (out[self.n:] == 7.0).all()  # rows of no request


# (In these tests ~1000 rows and more of a request are many enough for the
# kernel of tiles, ~100 and fewer for that of single rows.)

def sample_of(n, k=24, seed=0):
    if n <= k:
        return None
    return sorted(set(np.random.default_rng(seed).choice(n, k, replace=False).tolist()) | {0, n - 1})


# ------------------------------------------------------------------ the packed selection

def packed_rows(b, width, seed, counts):
    rng = np.random.default_rng(seed)
    out = np.full((b.total, width), -1, dtype=np.int32)
    for i in range(b.total):
        p = int(b.pos[i])
        n = min(counts[i % len(counts)], width - 1, p + 1)
        out[i, :n] = rng.choice(p + 1, size=n, replace=False)
        out[i, -1] = n
    return out


def run_sparse(b, packed, ws_fill=0xFF):
    d = b.to_gpu()
    width = packed.shape[1]
    cfg = Q.make_cfg(8, 4, width - 4, Q.DTYPE_BF16, 4, 1)
    n = Q.workspace_bytes(cfg, b.gcfg(), b.total, len(b.contexts), 1)
    ws = torch.full((n,), ws_fill, dtype=torch.uint8, device="cuda")
    Q.sparse_gqa_scaled(b.gcfg(), b.sc, d["q"], d["kv"], d["table"], torch.from_numpy(packed).cuda(), d["t2r"], d["gate"],
                        d["out"], ws)
    torch.cuda.synchronize()
    return f64(d["out"])


def check_sparse(b, packed, out):
    for i in range(b.n):
        tok = packed[i, :packed[i, -1]]
        K, V = b.values(b.t2r[i], tok)
        assert_row(out[i], f64(b.q[i]), K, V, None if b.gate is None else f64(b.gate[i]), f"row {i}")


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (10, 2), (8, 1), (16, 1), (12, 2), (14, 2), (32, 2)])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 64), (96, 32)])
def test_sparse_groups_and_blocks(hq, hkv, page, block):
    b = Batch([37, 301, 5, 1], [1, 2, 1, 1], hq=hq, hkv=hkv, page=page, block=block, seed=hq)
    packed = packed_rows(b, 64 + 4, 1, [64, 33, 1, 0, 17])
    check_sparse(b, packed, run_sparse(b, packed))
    assert Q.check_errors() == 0


@pytest.mark.parametrize("rows,counts,width", [
    (1, [2051], 2052), (3, [4103, 2600, 0], 4104), (40, [2051, 1000, 17], 2052), (200, [515, 0, 64], 516), (700, [100], 132)])
def test_sparse_lengths_and_splits(rows, counts, width):
    b = Batch([6000] * rows if rows < 10 else [700] * rows, [1] * rows, hq=16, hkv=4 if rows < 100 else 8, page=64, block=32,
              seed=rows, gate=rows != 40)
    packed = packed_rows(b, width, rows, counts)
    out = run_sparse(b, packed)
    if rows > 40:
        b.n = 40
    check_sparse(b, packed, out)
    assert Q.check_errors() == 0


def test_sparse_odd_scales_queries_and_pages():
    """Scale bytes out of range, queries far from 1, a token on a page outside
    the cache, a request outside the table."""
    b = Batch([64, 64, 64, 64], [1, 1, 1, 1], hq=8, hkv=1, page=16, block=16, seed=4, gate=False)
    b.scales[:] = torch.from_numpy(np.random.default_rng(1).choice([0, 87, 100, 127, 140], b.scales.shape).astype(np.uint8))
    b.scales[..., 0] = 120
    b.q[0] *= 2.0 ** 30
    b.q[1] *= 2.0 ** -60
    b.table[2, 1] = b.blocks
    packed = packed_rows(b, 68, 2, [64])
    b.t2r[3] = 4
    out = run_sparse(b, packed)
    assert Q.check_errors() >= 2
    assert (out[3] == 0).all()
    packed[2, :48] = [t for t in packed[2, :64] if t // 16 != 1]
    packed[2, -1] = 48
    b.n = 3
    # (the 2^30 scores of row 0 pick one token each: fp32 scores of that size
    # are off by more than 1, so only the two others are held to the bound)
    for i in (1, 2):
        tok = packed[i, :packed[i, -1]]
        K, V = b.values(b.t2r[i], tok)
        assert_row(out[i], f64(b.q[i]), K, V, None, f"row {i}")
    assert np.isfinite(out[0]).all()


# ------------------------------------------------------------------ windows

@pytest.mark.parametrize("kind", ["bf16", "e4m3", "block"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 4), (128, 0), (100, 150), (1000000, 0), (0, 3), (0, 0), (2147483647, 2147483647)])
def test_window_decode(kind, window, sinks):
    b = Batch([37, 301, 5, 1, 128, 129, 517], [1] * 7, kind=kind, seed=window % 97 + sinks % 89, pad=3)
    b.check_window(b.window(window, sinks), window, sinks)
    assert Q.check_errors() == 0


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (10, 2), (12, 2), (14, 2), (16, 1), (40, 8)])
@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("rows", [60, 1060])
def test_window_groups(hq, hkv, kind, rows):
    b = Batch([200, rows + 5], [1, rows], hq=hq, hkv=hkv, kind=kind, page=48, seed=hq, pad=1)
    b.check_window(b.window(50, 7), 50, 7, None if rows == 60 else sample_of(b.n))
    assert Q.check_errors() == 0


@pytest.mark.parametrize("kind,page,block", [("bf16", 16, 16), ("bf16", 64, 64), ("e4m3", 48, 16), ("block", 16, 16),
                                              ("block", 96, 32), ("block", 128, 64), ("bf16", 80, 16), ("bf16", 256, 64)])
@pytest.mark.parametrize("contexts,rows,window,sinks", [
    ([700], [700], 128, 4),            # a whole prompt
    ([1500, 300, 40], [257, 300, 33], 200, 0),
    ([2000, 900], [64, 1], 700, 130),  # a chunk and a decode row
    ([333] * 9, [4] * 9, 100, 1),      # verify steps
    ([1100], [1030], 5000, 0),         # plain causal
    ([2000, 900], [640, 1], 700, 130),
    ([333] * 9, [120] * 9, 100, 1),
])
def test_window_prefill(kind, page, block, contexts, rows, window, sinks):
    b = Batch(contexts, rows, hq=8, hkv=2, kind=kind, page=page, block=block, seed=page + window, pad=5, gate=page != 64)
    b.check_window(b.window(window, sinks), window, sinks, sample_of(b.n))
    assert Q.check_errors() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "block"])
@pytest.mark.parametrize("contexts,rows,hq,hkv,window,sinks", [
    ([1500 - 7 * i for i in range(40)], [4] * 40, 8, 2, 1400, 5),   # verify steps, whole windows
    ([20000, 11003], [8, 5], 8, 1, 30000, 0),                       # the same, split
    ([900, 700, 801], [100, 128, 99], 2, 2, 790, 0),                # heads of their own
    ([3000] * 20, [16] * 20, 8, 2, 257, 40),                        # few key tiles, an odd number of them
])
def test_window_requests_of_one_row_tile(kind, contexts, rows, hq, hkv, window, sinks):
    b = Batch(contexts, rows, hq=hq, hkv=hkv, kind=kind, page=64, block=32, seed=len(rows), pad=2)
    b.check_window(b.window(window, sinks), window, sinks, sample_of(b.n))
    assert Q.check_errors() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "block"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 2), (8, 1), (32, 2)])
@pytest.mark.parametrize("n", [300, 700, 1000, 2000])
def test_window_single_rows_in_few_splits(kind, hq, hkv, n):
    """Two to eight splits; rows shorter than one of them, before the start and
    of no request among them."""
    b = Batch([n, n // 2, 3, n - 1], [1, 1, 1, 1], hq=hq, hkv=hkv, kind=kind, page=64, block=32, seed=n + hq, pad=2)
    b.pos[1] = -1
    out = b.window(100000, 0)
    assert (out[1] == 0).all()
    b.check_window(out, 100000, 0)
    assert Q.check_errors() == 0


@pytest.mark.parametrize("hq,hkv", [(3, 1), (16, 1), (8, 2)])
@pytest.mark.parametrize("n", [500, 1300, 2000])
def test_sparse_in_few_splits(hq, hkv, n):
    b = Batch([3000, 2500, 2200], [1, 1, 1], hq=hq, hkv=hkv, page=64, block=64, seed=n + hq)
    packed = packed_rows(b, n + 1, n, [n, 0, n // 3])
    check_sparse(b, packed, run_sparse(b, packed))
    assert Q.check_errors() == 0


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("contexts,rows", [([40, 30, 20, 10], [0, 20, 0, 10]), ([40, 900, 20, 700], [0, 800, 0, 700])])
def test_window_requests_without_rows(kind, contexts, rows):
    b = Batch(contexts, rows, kind=kind, seed=2)
    b.check_window(b.window(16, 2), 16, 2, sample_of(b.n, 48))
    assert Q.check_errors() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "block"])
@pytest.mark.parametrize("rows", [1, 3, 90, 900])
def test_window_unseen_pages_and_garbage(kind, rows):
    """Pages that slid out of every window are -1 in the table, tokens behind
    the last position and before the window hold NaN (bf16: infinities too)."""
    b = Batch([1000, 501] if rows < 500 else [1500, 1301], [rows, rows], kind=kind, page=32, block=32, seed=rows, hq=4, hkv=1)
    window, sinks = 150, 3
    bad = 0x7F if kind != "bf16" else float("nan")
    for r, c in enumerate(b.contexts):
        first = max(0, c - rows - window + 1)
        for pg in range(first // 32):
            if pg * 32 >= sinks:
                b.table[r, pg] = -1
        for t in list(range(sinks, 32)) + list(range(first - first % 32, first)) + list(range(c, -(-c // 32) * 32)):
            if first <= t < c:
                continue
            b.kv[b.table[r, t // 32], :, t % 32] = bad
    b.check_window(b.window(window, sinks), window, sinks, sample_of(b.n))
    assert Q.check_errors() == 0


@pytest.mark.parametrize("rows", [1, 70, 1000])
def test_window_poisoned_token_reaches_only_rows_that_see_it(rows):
    context = 400 if rows < 300 else 1400
    b = Batch([context], [rows], kind="bf16", page=16, seed=5, hq=2, hkv=1, gate=False)
    window = 40
    tok = context - rows - window + 10 if rows > 1 else context - window - 2   # leaves the window during the call, or just has
    blk, off = b.table[0, tok // 16], tok % 16
    b.kv[blk, 0, off, D + 5] = float("inf")
    b.kv[blk, 0, off, D + 9] = float("nan")
    out = b.window(window, 0)
    for i in range(b.n):
        p = int(b.pos[i])
        sees = p - window < tok <= p
        clean = np.ones(D, dtype=bool)
        if sees:
            assert not np.isfinite(out[i][:, 5]).any() and np.isnan(out[i][:, 9]).all()
            clean[[5, 9]] = False
        assert np.isfinite(out[i][:, clean]).all(), i
        K, V = b.values(0, O.window_tokens(p, window, 0))
        if not sees:
            assert_row(out[i], f64(b.q[i]), K, V, None, f"row {i}")


@pytest.mark.parametrize("rows", [1, 70, 1000])
def test_window_bad_page_is_left_out_and_counted(rows):
    b = Batch([300 if rows < 300 else 1200], [rows], kind="bf16", page=16, seed=6, hq=2, hkv=1, gate=False)
    b.table[0, 16] = b.blocks + 5    # tokens 256 .. 271
    out = b.window(64, 0)
    assert Q.check_errors() > 0
    for i in range(b.n):
        tok = O.window_tokens(int(b.pos[i]), 64, 0)
        tok = tok[(tok < 256) | (tok >= 272)]
        K, V = b.values(0, tok)
        assert_row(out[i], f64(b.q[i]), K, V, None, f"row {i}")


@pytest.mark.parametrize("rows", [40, 1000])
def test_window_rows_before_the_start(rows):
    """A negative position sees nothing."""
    b = Batch([20, rows // 2], [2, rows], kind="bf16", seed=7)
    b.pos[2:] = np.arange(-(rows // 2), rows // 2)
    out = b.window(8, 1)
    assert (out[2:2 + rows // 2] == 0).all()
    b.check_window(out, 8, 1, None if rows == 40 else sample_of(b.n, 100))


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("contexts,rows", [([5000], [1]), ([9000, 300], [40, 40])])
def test_window_long_rows_are_split(kind, contexts, rows):
    b = Batch(contexts, rows, kind=kind, page=64, block=32, seed=8, hq=8, hkv=1)
    b.check_window(b.window(100000, 0), 100000, 0, sample_of(b.n, 8))
    # a bound that is too small changes nothing but the split
    b2 = Batch(contexts, rows, kind=kind, page=64, block=32, seed=8, hq=8, hkv=1)
    b2.check_window(b2.window(100000, 0, max_context=10), 100000, 0, sample_of(b.n, 8))
    assert Q.check_errors() == 0


@pytest.mark.parametrize("rows", [100, 800])
def test_window_strong_scores(rows):
    """Scores that rise and fall along the row move the running maximum."""
    b = Batch([900], [rows], kind="bf16", page=64, seed=9, hq=8, hkv=1, spread=8.0)
    ramp = torch.linspace(0.1, 6.0, 64).bfloat16()
    b.kv[..., :D] *= ramp[:, None]
    b.check_window(b.window(600, 4), 600, 4, sample_of(rows, 48))


def test_window_captured_and_on_two_streams():
    """Two graphs that share one workspace, replayed in order, and a call on
    another stream."""
    b = Batch([3000, 2500], [1, 1], kind="block", page=64, block=32, seed=10, hq=8, hkv=1)
    c = Batch([1600], [1200], kind="block", page=64, block=32, seed=11, hq=8, hkv=1)
    out_b, out_c = b.window(2048, 4), c.window(256, 4)
    sizes, calls = [], []
    for x, w in ((b, 2048), (c, 256)):
        a = Q.window_args(x.d["q"], x.d["kv"], x.d["table"], x.d["t2r"], x.d["qsl"], x.d["pos"], x.d["out"], w, 4,
                          max(x.contexts), gate=x.d["gate"], scales=x.sc)
        calls.append((x.gcfg(), a))
        sizes.append(Q.window_workspace_bytes(x.gcfg(), a))
    ws = torch.empty(max(sizes + [1]), dtype=torch.uint8, device="cuda")
    graphs = []
    for g, a in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            Q.window_gqa(g, a, ws)
        graphs.append(graph)
    for x in (b, c):
        x.d["out"].fill_(3.0)
    for k in (0, 1, 0, 1):
        graphs[k].replay()
    torch.cuda.synchronize()
    assert np.array_equal(f64(b.d["out"]), out_b) and np.array_equal(f64(c.d["out"]), out_c)
    s = torch.cuda.Stream()
    b.d["out"].fill_(3.0)
    s.wait_stream(torch.cuda.current_stream())
    Q.window_gqa(*calls[0], ws, stream=s)
    s.synchronize()
    assert np.array_equal(f64(b.d["out"]), out_b)


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("rows", [1, 70, 1000])
def test_window_positions_past_the_table(kind, rows):
    """Only the table's tokens are looked at, however far a position is."""
    b = Batch([320], [rows], kind=kind, page=32, seed=13, hq=2, hkv=1, gate=False)
    b.pos[:] = 2 ** 31 - 1 - np.arange(rows)[::-1]
    out = b.window(2 ** 31 - 1, 2 ** 31 - 1)
    assert Q.check_errors() > 0
    some = sample_of(rows) or range(rows)
    for i in some:
        K, V = b.values(0, np.arange(320))
        assert_row(out[i], f64(b.q[i]), K, V, None, f"row {i}")
    assert (b.window(1000, 0) == 0).all()
    assert Q.check_errors() > 0
    out = b.window(0, 40)
    assert Q.check_errors() == 0
    for i in some:
        K, V = b.values(0, np.arange(40))
        assert_row(out[i], f64(b.q[i]), K, V, None, f"row {i}")


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("rows", [40, 140])
def test_window_odd_values_beside_rows_before_the_start(kind, rows):
    """Values that are not finite in many tiles reach every row that sees them
    and no row at a negative position."""
    b = Batch([6000], [rows], kind=kind, page=32, block=32, seed=14, hq=8, hkv=1, gate=False)
    b.pos[5:20] = -np.arange(1, 16)
    odd = np.arange(0, 6000, 130)
    b.kv[torch.from_numpy(b.table[0, odd // 32].astype(np.int64)), 0, torch.from_numpy(odd % 32), D + 5] = \
        0x7F if kind == "block" else float("nan")
    out = b.window(100000, 0)
    assert Q.check_errors() == 0
    assert (out[5:20] == 0).all()
    rest = np.r_[0:5, 20:rows]
    assert np.isnan(out[rest][:, :, 5]).all()
    clean = np.arange(D) != 5
    b.kv[torch.from_numpy(b.table[0, odd // 32].astype(np.int64)), 0, torch.from_numpy(odd % 32), D + 5] = 0
    for i in (0, 4, 20, rows - 1):
        K, V = b.values(0, O.window_tokens(int(b.pos[i]), 100000, 0))
        out[i][:, ~clean] = attend_row(f64(b.q[i]), K, V)[0][:, ~clean]
        assert_row(out[i], f64(b.q[i]), K, V, None, f"row {i}")


@pytest.mark.parametrize("kind", ["e4m3", "block"])
@pytest.mark.parametrize("page,rows", [(16, 70), (16, 1000), (64, 1000)])
def test_window_nan_codes_reach_only_rows_that_see_them(kind, page, rows):
    context = 400 if rows < 300 else 1400
    b = Batch([context], [rows], kind=kind, page=page, block=16, seed=15, hq=2, hkv=1, gate=False)
    toks = [context - 55, context - 29, context - 1]   # left by the window, ahead of some rows, the last one's own
    for tok in toks:
        b.kv[b.table[0, tok // page], 0, tok % page, D + 9] = 0xFF
    out = b.window(40, 0)
    for i in range(b.n):
        p = int(b.pos[i])
        assert np.isnan(out[i][:, 9]).all() == any(p - 40 < t <= p for t in toks), p
        assert np.isfinite(out[i][:, np.arange(D) != 9]).all(), p
    assert Q.check_errors() == 0


@pytest.mark.parametrize("kind", ["bf16", "block"])
@pytest.mark.parametrize("rows", [1, 1000])
def test_window_far_into_a_large_cache(kind, rows):
    """Pages whose bytes lie past 2^32."""
    b = Batch([1300], [rows], kind=kind, page=64, block=64, seed=16, hq=4, hkv=1)
    row_bytes = 512 if kind == "bf16" else 256
    ahead = 2 ** 32 // (64 * row_bytes) + 1
    out_near = b.window(120, 3)
    kv = torch.zeros((ahead + b.blocks,) + tuple(b.kv.shape[1:]), dtype=b.kv.dtype, device="cuda")
    kv[ahead:] = b.d["kv"]
    b.d["kv"], b.d["table"] = kv, b.d["table"] + ahead
    if kind == "block":
        b.d["scales"] = torch.cat([torch.zeros((ahead, 1, 1, 2), dtype=torch.uint8, device="cuda"), b.d["scales"]])
        b.sc = Q.kv_scales(b.d["scales"], 64)
    b.blocks += ahead
    b.d["out"].fill_(7.0)
    assert np.array_equal(b.window(120, 3), out_near)
    assert Q.check_errors() == 0


def test_calls_on_streams_side_by_side():
    """Calls on three streams at once, each with a workspace of its own."""
    batches = [Batch([4000, 2500], [1, 1], kind="block", page=64, block=32, seed=17, hq=8, hkv=2),
               Batch([900], [300], kind="bf16", page=64, seed=18, hq=8, hkv=2),
               Batch([2000] * 3, [1] * 3, kind="block", page=64, block=32, seed=19, hq=8, hkv=2)]
    packed = packed_rows(batches[2], 1028, 3, [1024])
    want = [batches[0].window(5000, 0), batches[1].window(400, 4), run_sparse(batches[2], packed)]
    cfg = Q.make_cfg(8, 4, 1024, Q.DTYPE_BF16, 4, 1)
    x = batches[2]
    ws = [torch.empty(1 << 24, dtype=torch.uint8, device="cuda") for _ in range(3)]
    assert Q.workspace_bytes(cfg, x.gcfg(), 3, 3, 1) <= 1 << 24
    args = []
    for b, w, s in ((batches[0], 5000, 0), (batches[1], 400, 4)):
        args.append(Q.window_args(b.d["q"], b.d["kv"], b.d["table"], b.d["t2r"], b.d["qsl"], b.d["pos"], b.d["out"], w, s,
                                  max(b.contexts), gate=b.d["gate"], scales=b.sc))
        assert Q.window_workspace_bytes(b.gcfg(), args[-1]) <= 1 << 24
    pk = torch.from_numpy(packed).cuda()
    for b in batches:
        b.d["out"].fill_(3.0)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for k in range(2):
            Q.window_gqa(batches[k].gcfg(), args[k], ws[k], stream=streams[k])
        Q.sparse_gqa_scaled(x.gcfg(), x.sc, x.d["q"], x.d["kv"], x.d["table"], pk, x.d["t2r"], x.d["gate"], x.d["out"], ws[2],
                            stream=streams[2])
    torch.cuda.synchronize()
    for b, w in zip(batches, want):
        assert np.array_equal(f64(b.d["out"]), w)


def test_sparse_captured_and_replayed():
    """Split rows as a graph, replayed on new selections."""
    b = Batch([5000] * 4, [1] * 4, hq=8, hkv=2, page=64, block=32, seed=20)
    packed = packed_rows(b, 2052, 1, [2048, 700])
    run_sparse(b, packed)
    d, pk = b.d, torch.from_numpy(packed).cuda()
    cfg = Q.make_cfg(8, 4, 2048, Q.DTYPE_BF16, 4, 1)
    ws = torch.empty(Q.workspace_bytes(cfg, b.gcfg(), 4, 4, 1), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.sparse_gqa_scaled(b.gcfg(), b.sc, d["q"], d["kv"], d["table"], pk, d["t2r"], d["gate"], d["out"], ws)
    packed = packed_rows(b, 2052, 2, [33, 0, 2048, 1])
    pk.copy_(torch.from_numpy(packed))
    ws.fill_(0xFF)
    graph.replay()
    torch.cuda.synchronize()
    check_sparse(b, packed, f64(d["out"]))
    assert Q.check_errors() == 0


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("rows", [[1, 1, 1], [5, 130, 1], [5, 400, 1]])
def test_append_then_both_attentions(rows):
    """A step as a model runs it: keys and values into the cache with block
    scales, then the sparse layer's and the window layer's attention of the
    same rows, which see the tokens just appended."""
    b = Batch([150, 400, 33], rows, hq=8, hkv=2, page=64, block=32, seed=12)
    d = b.to_gpu()
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn((b.n, (2 * b.hq + 2 * b.hkv) * D), generator=g).bfloat16().cuda()
    from learned_sparse_attention_gb300 import workloads as W
    cs = W.rope_cos_sin(512, 64).cuda()
    slots = b.table[b.t2r, b.pos // 64].astype(np.int64) * 64 + b.pos % 64
    t = dict(main_qkv=qkv, main_q_norm_w=torch.zeros(D, dtype=torch.bfloat16, device="cuda"),
             main_k_norm_w=torch.zeros(D, dtype=torch.bfloat16, device="cuda"), kv=d["kv"],
             slot_mapping=torch.from_numpy(slots).cuda(), main_q_out=d["q"], main_gate_out=d["gate"])
    cfg = Q.make_cfg(8, 4, 64, Q.DTYPE_BF16, 4, 512)
    pos = torch.from_numpy(np.repeat(b.pos.astype(np.int64)[:, None, None], 3, 2)).cuda()
    Q.kv_append(cfg, b.gcfg(), Q.main_prep(t), pos, cs, scales=b.sc)
    out = b.window(100, 4)
    b.q, b.gate, b.kv, b.scales = d["q"].cpu(), d["gate"].cpu(), d["kv"].cpu(), d["scales"].cpu()
    b.check_window(out, 100, 4, sample_of(b.n))
    packed = packed_rows(b, 68, 5, [64])
    packed[:, 0] = b.pos  # the row's own token among them
    for i in range(b.n):
        seen = list(dict.fromkeys(packed[i, :packed[i, -1]].tolist()))
        packed[i, :-1] = -1
        packed[i, :len(seen)] = seen
        packed[i, -1] = len(seen)
    ws = torch.empty(Q.workspace_bytes(cfg, b.gcfg(), b.n, 3, 1), dtype=torch.uint8, device="cuda")
    Q.sparse_gqa_scaled(b.gcfg(), b.sc, d["q"], d["kv"], d["table"], torch.from_numpy(packed).cuda(), d["t2r"], d["gate"],
                        d["out"], ws)
    torch.cuda.synchronize()
    check_sparse(b, packed, f64(d["out"]))
    assert Q.check_errors() == 0
