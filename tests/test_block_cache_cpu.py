"""Host-side checks of the cache with block scales and of window attention,
and the oracle's pins for them (CPU only; nothing is launched)."""

import ctypes

import numpy as np
import pytest
import torch

from learned_sparse_attention_gb300 import build as B
from learned_sparse_attention_gb300 import qsa as Q
from oracle import qsa_oracle as O
from tests.attention_bounds import assert_row, attend_row


@pytest.fixture(scope="module")
def lib():
    B.build_library()
    return Q.load(build_if_missing=False)


D256 = ctypes.c_void_p(256)


def _cfg():
    return Q.make_cfg(8, 4, 64, Q.DTYPE_BF16, 4, 100)


def _gcfg(dtype=Q.DTYPE_E4M3_BLOCK, page=64, **kw):
    return Q.make_gqa_cfg(8, 2, page, kw.pop("blocks", 10), kv_dtype=dtype, **kw)


def _scales(ptr=256, block=32):
    s = Q.QsaKvScales()
    s.scales, s.scale_block = ptr, block
    return s


def _main(**kw):
    m = Q.QsaMainPrep()
    f = dict(qkv=256, q_norm_w=256, k_norm_w=256, eps=1e-6, q_out=256, gate_out=256, kv=256, slot_mapping=256)
    f.update(kw)
    for k, v in f.items():
        setattr(m, k, v)
    return m


def _append(lib, m=None, g=None, s="default", rows=4, positions=D256, cos_sin=D256, cfg=None):
    s = _scales() if s == "default" else s
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return lib.qsa_kv_append(ref(cfg or _cfg()), ref(g or _gcfg()), ref(m or _main()), ref(s), positions, cos_sin, rows, None)


def test_append_refusals(lib):
    assert _append(lib, rows=0) == 0
    assert _append(lib, rows=-1) == 2
    assert _append(lib, s=None) == 1
    assert _append(lib, s=_scales(ptr=None)) == 1
    assert _append(lib, s=_scales(ptr=258)) == 1
    assert _append(lib, s=_scales(block=8)) == 4
    assert _append(lib, s=_scales(block=48)) == 4
    assert _append(lib, g=_gcfg(page=48)) == 2                       # 32 does not divide the page
    assert _append(lib, g=_gcfg(Q.DTYPE_BF16)) == 1                  # scales for a cache without them
    assert _append(lib, g=_gcfg(3)) == 3
    assert _append(lib, m=_main(q_out=None)) == 1                    # a gate without its q
    assert _append(lib, m=_main(gate_out=None)) == 1
    assert _append(lib, m=_main(q_norm_w=None)) == 1
    for missing in ("qkv", "k_norm_w", "kv", "slot_mapping"):
        assert _append(lib, m=_main(**{missing: None})) == 1
    for odd in ("qkv", "kv", "q_out"):
        assert _append(lib, m=_main(**{odd: 264})) == 1
    assert _append(lib, m=_main(slot_mapping=260)) == 1
    assert _append(lib, m=_main(eps=float("nan"))) == 1
    assert _append(lib, positions=None) == 1
    assert _append(lib, cos_sin=None) == 1
    assert _append(lib, cfg=Q.make_cfg(8, 4, 64, 0, 4, 100, head_dim=64)) == 4
    assert _append(lib, rows=(1 << 31) - 1) == 2
    assert lib.qsa_kv_append(None, None, None, None, None, None, 1, None) == 1


def test_other_entry_points_refuse_block_scales(lib):
    g = _gcfg()
    assert lib.qsa_sparse_gqa(ctypes.byref(g), D256, D256, D256, 1, D256, 68, D256, None, D256, 4, D256, 1 << 30, None) == 3
    assert lib.qsa_sparse_gqa_noalloc(ctypes.byref(g), D256, D256, D256, 1, D256, 68, D256, None, D256, 4, None) == 3
    m = _main()
    assert lib.qsa_main_prepare(ctypes.byref(_cfg()), ctypes.byref(g), ctypes.byref(m), D256, D256, 4, None) == 3
    a = Q.QsaStepArgs()
    a.rows, a.reqs, a.packed = 4, 1, 256
    assert lib.qsa_layer_step(ctypes.byref(_cfg()), ctypes.byref(g), ctypes.byref(a), 0, D256, 1 << 30, None) == 3
    # a statically scaled prepare still wants its q
    m = _main(q_out=None, gate_out=None)
    g1 = _gcfg(Q.DTYPE_BF16)
    assert lib.qsa_main_prepare(ctypes.byref(_cfg()), ctypes.byref(g1), ctypes.byref(m), D256, D256, 4, None) == 1


def _sparse(lib, g=None, s="default", q=D256, kv=D256, bt=D256, stride=1, packed=D256, width=68, t2r=D256, out=D256, rows=4,
            reqs=1, ws=D256, ws_bytes=1 << 30, gate=None):
    s = _scales() if s == "default" else s
    return lib.qsa_sparse_gqa_scaled(ctypes.byref(g or _gcfg()), None if s is None else ctypes.byref(s), q, kv, bt, stride,
                                     packed, width, t2r, gate, out, rows, reqs, ws, ws_bytes, None)


def test_sparse_refusals(lib):
    assert _sparse(lib, rows=0) == 0
    assert _sparse(lib, rows=-1) == 2
    assert _sparse(lib, g=_gcfg(Q.DTYPE_BF16), s=None) == 3
    assert _sparse(lib, g=_gcfg(Q.DTYPE_E4M3), s=None) == 3
    assert _sparse(lib, s=None) == 1
    for k in ("q", "kv", "bt", "packed", "t2r", "out"):
        assert _sparse(lib, **{k: None}) == 1
    for k in ("q", "kv", "out", "gate"):
        assert _sparse(lib, **{k: ctypes.c_void_p(264)}) == 1
    assert _sparse(lib, width=1) == 2
    assert _sparse(lib, stride=0) == 2
    assert _sparse(lib, reqs=0) == 2
    assert _sparse(lib, s=_scales(block=128)) == 4
    assert _sparse(lib, g=_gcfg(page=48)) == 2
    assert _sparse(lib, g=_gcfg(blocks=1 << 26)) == 2                # row ids past 32 bits
    assert _sparse(lib, g=Q.make_gqa_cfg(24, 2, 64, 10, kv_dtype=2)) == 4


def _window(lib, g=None, s="default", ws=D256, ws_bytes=1 << 40, **kw):
    a = Q.QsaWindowArgs()
    f = dict(rows=4, reqs=1, window=16, sinks=4, max_context=100, bt_stride=2, q=256, kv=256, block_table=256, token_to_req=256,
             query_start_loc=256, logical_positions=256, gate=None, out=256)
    f.update(kw)
    for k, v in f.items():
        setattr(a, k, v)
    s = _scales() if s == "default" else s
    a.scales = None if s is None else ctypes.addressof(s)
    return lib.qsa_window_gqa(ctypes.byref(g or _gcfg()), ctypes.byref(a), ws, ws_bytes, None)


def test_window_refusals(lib):
    assert _window(lib, rows=0) == 0
    assert _window(lib, rows=-1) == 2
    assert _window(lib, reqs=-1) == 2
    assert _window(lib, reqs=0) == 2
    assert _window(lib, max_context=-1) == 2
    assert _window(lib, window=-1) == 1
    assert _window(lib, sinks=-1) == 1
    assert _window(lib, bt_stride=0) == 2
    for k in ("q", "kv", "block_table", "token_to_req", "query_start_loc", "logical_positions", "out"):
        assert _window(lib, **{k: None}) == 1
    for k in ("q", "kv", "out", "gate"):
        assert _window(lib, **{k: 264}) == 1
    assert _window(lib, s=None) == 1
    assert _window(lib, g=_gcfg(Q.DTYPE_BF16)) == 1
    assert _window(lib, g=_gcfg(page=40)) == 2
    assert _window(lib, g=Q.make_gqa_cfg(26, 2, 64, 10), s=None) == 4
    assert _window(lib, g=_gcfg(blocks=1 << 26)) == 2
    assert lib.qsa_window_gqa(ctypes.byref(_gcfg()), None, None, 0, None) == 1
    assert lib.qsa_window_gqa(None, None, None, 0, None) == 1


def test_split_rows_want_their_workspace(lib):
    big = dict(rows=1, reqs=1, window=1 << 20, max_context=100000)
    a = Q.QsaWindowArgs()
    for k, v in big.items():
        setattr(a, k, v)
    need = lib.qsa_window_workspace_bytes(ctypes.byref(_gcfg()), ctypes.byref(a))
    assert need > 0
    for ws, n in ((None, need), (D256, need - 1), (ctypes.c_void_p(128), need)):
        assert _window(lib, ws=ws, ws_bytes=n, **big) == 5
    g = _gcfg()
    assert lib.qsa_gqa_splits(ctypes.byref(g), 1, 4100) > 1
    for ws, n in ((None, 1 << 30), (D256, 256), (ctypes.c_void_p(128), 1 << 30)):
        assert _sparse(lib, rows=1, width=4100, ws=ws, ws_bytes=n) == 5


def test_window_workspace_of_bad_sizes(lib):
    a = Q.QsaWindowArgs()
    a.rows = -1
    assert lib.qsa_window_workspace_bytes(ctypes.byref(_gcfg()), ctypes.byref(a)) == 0
    assert lib.qsa_window_workspace_bytes(None, ctypes.byref(a)) == 0
    assert lib.qsa_window_workspace_bytes(ctypes.byref(_gcfg()), None) == 0


def test_binding_refuses_host_tensors_and_small_scales(lib):
    with pytest.raises(ValueError):
        Q.kv_scales(torch.zeros(8, dtype=torch.uint8), 16)
    s = _scales(block=32)
    s._tensors = torch.zeros(39, dtype=torch.uint8)
    kv = torch.zeros((10, 2, 64, 256), dtype=torch.uint8)
    with pytest.raises(ValueError, match="scales"):
        Q._pointers(-1, Q._cache_specs(_gcfg(), s, kv))       # 10 blocks x 2 heads x 2 scale blocks x 2 = 80


def test_binding_refuses_tensors_that_are_too_small():
    """Each would be read or written past its end."""
    g = Q.make_gqa_cfg(2, 1, 16, 3, kv_dtype=Q.DTYPE_E4M3_BLOCK)
    cfg = Q.make_cfg(8, 4, 64, Q.DTYPE_BF16, 4, 10)
    sc = _scales(block=16)
    sc._tensors = torch.zeros(6, dtype=torch.uint8)
    kv = torch.zeros((3, 1, 16, 256), dtype=torch.uint8)
    bf = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32)    # noqa: E731

    def append(**kw):
        t = dict(main_qkv=bf(4, 6 * 128), main_q_out=bf(4, 2, 128), main_gate_out=bf(4, 2, 128), kv=kv,
                 slot_mapping=torch.zeros(4, dtype=torch.int64))
        pos, cs = kw.pop("positions", torch.zeros((4, 1, 3), dtype=torch.int64)), kw.pop("cos_sin", torch.zeros(10, 64))
        t.update(kw)
        m = Q.QsaMainPrep()
        m._tensors, m._entries = t, Q._main_entries(t)
        Q.kv_append(cfg, g, m, pos, cs, scales=sc)

    for name, small in dict(main_qkv=bf(3, 6 * 128), main_q_out=bf(3, 2, 128), main_gate_out=bf(4, 1, 128), kv=kv[:2],
                            slot_mapping=torch.zeros(3, dtype=torch.int64), positions=torch.zeros((4, 1), dtype=torch.int64),
                            cos_sin=torch.zeros(9, 64)).items():
        with pytest.raises(ValueError, match=name):
            append(**{name: small})
    with pytest.raises(ValueError, match="kv has dtype"):
        append(kv=kv.to(torch.bfloat16))

    def sparse(**kw):
        t = dict(q=bf(4, 2, 128), kv=kv, table=i32(1, 3), packed=i32(4, 9), t2r=i32(4), gate=None, out=bf(4, 2, 128))
        t.update(kw)
        Q.sparse_gqa_scaled(g, sc, t["q"], t["kv"], t["table"], t["packed"], t["t2r"], t["gate"], t["out"], None)

    for name, small in dict(q=bf(4, 1, 128), kv=kv[:2], packed=i32(3, 9), t2r=i32(3), gate=bf(3, 2, 128), out=bf(4, 127)).items():
        with pytest.raises(ValueError, match="token_to_req" if name == "t2r" else name):
            sparse(**{name: small})
    with pytest.raises(ValueError, match="CUDA"):
        sparse()


# ------------------------------------------------------------------ the oracle

def test_scale_exponent():
    assert O.scale_exponent(448.0) == 0 and O.scale_exponent(np.nextafter(448.0, 1e9)) == 1
    assert O.scale_exponent(224.0) == -1 and O.scale_exponent(0.0) == -40 and O.scale_exponent(1e38) == 40
    for e in range(-30, 30):
        peak = 300.0 * 2.0 ** e
        assert 224.0 < peak / 2.0 ** O.scale_exponent(peak) <= 448.0


def test_append_runs():
    assert O.append_runs([64, 65, 66], 32) == [(0, 3)]
    assert O.append_runs([94, 95, 96, 97], 32) == [(0, 2), (2, 2)]
    assert O.append_runs([3, -1, 4, 4, 5], 16) == [(0, 1)] and O.append_runs([3, -1, 20], 16) == [(0, 1), (2, 1)]
    assert O.append_runs([3] + [-1] * 31 + [4], 16) == [(0, 1)]
    assert O.append_runs([9, 8], 16) == [(0, 1)] and O.append_runs([9, 40, 8], 16) == [(0, 1), (1, 1), (2, 1)]
    assert O.append_runs([1, 3, 9], 16) == [(0, 3)]


def test_append_block_kv_by_hand():
    codes, scales = np.zeros((1, 1, 16, 8), dtype=np.uint8), np.full((1, 1, 1, 2), 127, dtype=np.uint8)
    k = np.array([[[1.0, -2.0, 0.5, 0.0]]])
    O.append_block_kv(codes, scales, [0], k, k * 448, 16, 16)
    # 448 * 2^-7 = 3.5 covers 2, 448 * 2^-8 = 1.75 does not; V peaks at 896
    assert scales.ravel().tolist() == [120, 128]
    x = O.dequantise_block_kv(codes, scales, 16)
    assert np.array_equal(x[0, 0, 0], np.concatenate([k[0, 0], k[0, 0] * 448]))
    O.append_block_kv(codes, scales, [1], k * 1024, k, 16, 16)       # K grows by 2^10, V does not
    assert scales.ravel().tolist() == [130, 128]
    x = O.dequantise_block_kv(codes, scales, 16)
    assert np.array_equal(x[0, 0, 1, :4], k[0, 0] * 1024)
    assert np.array_equal(x[0, 0, 0, :4], k[0, 0])                   # 2^-3 .. still a code: nothing is lost
    O.append_block_kv(codes, scales, [0], k / 64, k, 16, 16)         # the block begins anew
    assert scales.ravel().tolist() == [114, 120]


def test_window_tokens():
    assert O.window_tokens(9, 3, 2).tolist() == [0, 1, 7, 8, 9]
    assert O.window_tokens(1, 100, 7).tolist() == [0, 1]
    assert O.window_tokens(5, 0, 0).tolist() == [] and O.window_tokens(-1, 5, 5).tolist() == []
    assert O.window_tokens(5, 1 << 31, 0).tolist() == list(range(6))


def test_attention_bound_is_of_the_rounding_s_size():
    """The row agrees with torch in 64 bits; the bound lets bf16 roundings
    pass and catches a token too many."""
    rng = np.random.default_rng(0)
    q, K, V = rng.normal(size=(4, 128)), rng.normal(size=(50, 2, 128)), rng.normal(size=(50, 2, 128))
    out, bound = attend_row(q, K, V)
    t = lambda x: torch.from_numpy(x)  # noqa: E731
    want = torch.nn.functional.scaled_dot_product_attention(
        t(q)[:, None], t(K).transpose(0, 1).repeat_interleave(2, 0), t(V).transpose(0, 1).repeat_interleave(2, 0))
    assert np.abs(out - want[:, 0].numpy()).max() < 1e-12
    assert_row(O.round_bf16(out), q, K, V)
    less = attend_row(q, K[1:], V[1:])[0]
    assert (np.abs(less - out) > bound).any()
    gated, _ = attend_row(q, K, V, np.zeros((4, 128)))
    assert np.allclose(gated, out / 2)
