"""The operators of the 8-bit cache with block scales and of window attention, as they are measured.

Three operators over the paged KV cache [blocks, Hkv, page, 2 * 128] (K then V of a token and KV head):

* append: a step's projection rows become q, gate and the cache rows of their tokens (Gemma RMSNorm, RoPE, cache write),
  in bf16, in e4m3 with a static scale, or in e4m3 with a power-of-two scale for each block of tokens and KV head;
* sparse: grouped-query attention over the packed selection, reading the cache with block scales;
* window: grouped-query attention over the last `window` tokens and the first `sinks`, reading any of the three caches.

A case's lengths follow from the case alone; values, page tables and selections follow from the seed.
"""

import math
import random

import torch

own = False

D = 128          # head dim
ROT = 64         # rotated dims
EPS = 1e-6
STATIC = 1.0 / 16  # scale of the static e4m3 cache, K and V alike
SECTIONS = (8, 12, 12)  # interleaved MRoPE sections


def listed():
    big = dict(hq=32, hkv=4, page=64)
    return [
        # two requests of a small model: nothing but latency
        dict(name="append_two_rows", op="append", kv="block", reqs=2, rows=1, context=300, hq=8, hkv=1, page=16, block=16,
             mrope=False, q=True),
        # one decode step of a serving batch, each row somewhere inside a scale block
        dict(name="append_decode_64", op="append", kv="block", reqs=64, rows=1, context=32768, block=32, mrope=False, q=True, **big),
        # the verify step of a draft of four over image spans, the scale block as long as the page
        dict(name="append_verify_32x4", op="append", kv="block", reqs=32, rows=4, context=65536, block=64, mrope=True, q=True, **big),
        # a prefill chunk
        dict(name="append_prefill_16384", op="append", kv="block", reqs=1, rows=16384, context=49152, block=32, mrope=False, q=True,
             **big),
        # two requests of a small model
        dict(name="sparse_two_rows", op="sparse", kv="block", reqs=2, rows=1, context=300, hq=8, hkv=1, page=16, block=16, topk=64,
             ratio=4, gate=True),
        # the selection of one decode step of a serving batch
        dict(name="sparse_decode_64", op="sparse", kv="block", reqs=64, rows=1, context=32768, block=32, topk=2048, ratio=4,
             gate=True, **big),
        # eight long requests with twice the heads and twice the selection
        dict(name="sparse_long_8", op="sparse", kv="block", reqs=8, rows=1, context=131072, hq=64, hkv=8, page=64, block=64,
             topk=4096, ratio=8, gate=True),
        # one request alone, a short window
        dict(name="window_one_row", op="window", kv="bf16", reqs=1, rows=1, context=4000, hq=8, hkv=1, page=16, block=0,
             window=512, sinks=4, gate=False),
        # a decode step of a serving batch over the cache with block scales
        dict(name="window_decode_64", op="window", kv="block", reqs=64, rows=1, context=32768, block=32, window=4096, sinks=4,
             gate=True, **big),
        # the verify step of a draft of four
        dict(name="window_verify_32x4", op="window", kv="bf16", reqs=32, rows=4, context=65536, block=0, window=4096, sinks=16,
             gate=True, **big),
        # three ragged requests prefilled together over the cache with block scales
        dict(name="window_ragged_3", op="window", kv="block", reqs=3, rows=2011, context=9001, hq=24, hkv=4, page=48, block=16,
             window=1000, sinks=5, gate=True),
        # a prefill chunk
        dict(name="window_prefill_16384", op="window", kv="bf16", reqs=1, rows=16384, context=49152, block=0, window=4096, sinks=4,
             gate=True, **big),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "sparse", "window"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 6, 8, 16]) if hkv <= 4 else rng.choice([1, 2, 5, 8])
    page = rng.choice([16, 32, 48, 64, 128])
    block = rng.choice([b for b in (16, 32, 64) if page % b == 0])
    c = dict(op=op, hq=hkv * group, hkv=hkv, page=page, block=block)
    if op == "append":
        kind = rng.choice(["decode", "verify", "prefill"])
        c["reqs"] = _log_int(rng, 1, 96) if kind != "prefill" else rng.randint(1, 4)
        c["rows"] = 1 if kind == "decode" else rng.randint(2, 7) if kind == "verify" else _log_int(rng, 33, 8192 // c["reqs"])
        c["context"] = c["rows"] + _log_int(rng, 16, 32768)
        c["kv"] = rng.choice(["block", "block", "bf16", "e4m3"])
        c["mrope"] = rng.random() < 0.3
        c["q"] = rng.random() < 0.8
    elif op == "sparse":
        c["reqs"] = _log_int(rng, 1, 64)
        c["rows"] = rng.choice([1, 1, 2, 4]) if c["reqs"] > 2 else _log_int(rng, 1, 120)
        c["context"] = c["rows"] + _log_int(rng, 64, 32768)
        c["ratio"] = rng.choice([2, 4, 8])
        c["topk"] = c["ratio"] * _log_int(rng, 16, 2048 // c["ratio"])
        c["gate"] = rng.random() < 0.7
        c["kv"] = "block"
    else:
        kind = rng.choice(["decode", "verify", "prefill"])
        c["reqs"] = _log_int(rng, 1, 64) if kind != "prefill" else rng.randint(1, 4)
        c["rows"] = 1 if kind == "decode" else rng.randint(2, 9) if kind == "verify" else _log_int(rng, 33, 4096 // c["reqs"])
        c["context"] = c["rows"] + _log_int(rng, 16, 16384)
        c["window"] = _log_int(rng, 32, 4096)
        c["sinks"] = rng.choice([0, 1, 4, 16, 130])
        c["kv"] = rng.choice(["block", "bf16", "e4m3"])
        c["gate"] = rng.random() < 0.7
    return c


def _lengths(case):
    """Rows and final context length of each request: the first has the case's, the others up to half less."""
    r = random.Random(",".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name"))
    rows, ctx = [], []
    for i in range(case["reqs"]):
        n = case["rows"] if i == 0 or case["rows"] < 33 else r.randint(case["rows"] // 2, case["rows"])
        top = case["context"]
        rows.append(n)
        ctx.append(top if i == 0 else r.randint(max(n, top // 2), top))
    return rows, ctx


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _cache(case, g, blocks):
    """The cache as a serving process holds it: N(0, 1) keys and values in the case's type."""
    shape = (blocks, case["hkv"], case["page"], 2 * D)
    if case["kv"] == "bf16":
        return _randn(g, *shape).bfloat16(), None
    if case["kv"] == "e4m3":
        return (_randn(g, *shape) / STATIC).to(torch.float8_e4m3fn).view(torch.uint8), None
    # codes as 2^-6 or 2^-7 a step leaves them, and the scales' bytes
    kv = (_randn(g, *shape) * 96.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    n = (blocks, case["hkv"], case["page"] // case["block"], 2)
    return kv, torch.randint(119, 122, n, generator=g, device="cuda", dtype=torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, ctx = _lengths(case)
    n, reqs, page = sum(rows), case["reqs"], case["page"]
    need = [-(-c // page) for c in ctx]
    blocks, stride = sum(need), max(need)
    perm = torch.randperm(blocks, generator=g, device="cuda").int()
    table = torch.zeros((reqs, stride), dtype=torch.int32, device="cuda")
    at = 0
    for i, b in enumerate(need):
        table[i, :b] = perm[at:at + b]
        at += b
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    logical = torch.cat([torch.arange(c - r, c, dtype=torch.int32) for r, c in zip(rows, ctx)]).cuda()
    t2r = torch.repeat_interleave(torch.arange(reqs, dtype=torch.int32), torch.tensor(rows)).cuda()
    s = dict(case=case, rows=n, reqs=reqs, max_context=max(ctx), table=table, logical=logical, t2r=t2r,
             qsl=torch.tensor(starts, dtype=torch.int32).cuda())
    s["kv"], s["scales"] = _cache(case, g, blocks)
    if case["op"] == "append":
        s["qkv"] = _randn(g, n, (2 * case["hq"] + 2 * case["hkv"]) * D).bfloat16()
        # a few loud tokens, as keys of first tokens and separators are
        loud = torch.rand((n, 1), generator=g, device="cuda") < 0.02
        s["qkv"] = torch.where(loud, s["qkv"] * 6.0, s["qkv"]).contiguous()
        s["q_norm_w"], s["k_norm_w"] = (_randn(g, D) * 0.1).bfloat16(), (_randn(g, D) * 0.1).bfloat16()
        pos = logical.long()[:, None].repeat(1, 3)
        if case["mrope"]:  # an image of rows of 32 patches over all of it
            pos[:, 1] = pos[:, 0] // 32
            pos[:, 2] = pos[:, 0] % 32
        s["positions"] = pos.reshape(n, 1, 3).contiguous()
        freq = 10000.0 ** (-torch.arange(ROT // 2, dtype=torch.float64) * 2.0 / ROT)
        ang = torch.arange(max(ctx) + 1, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
        blk = table[t2r.long(), (logical // page).long()].long()
        s["slots"] = blk * page + (logical % page).long()
        s["q_out"] = torch.zeros((n, case["hq"], D), dtype=torch.bfloat16, device="cuda")
        s["gate_out"] = torch.zeros_like(s["q_out"])
        return s
    s["q"] = _randn(g, n, case["hq"], D).bfloat16()
    s["gate"] = _randn(g, n, case["hq"], D).bfloat16() if case["gate"] else None
    s["out"] = torch.zeros_like(s["q"])
    if case["op"] == "sparse":
        ratio, kb = case["ratio"], case["topk"] // case["ratio"]
        width = case["topk"] + ratio - 1
        vis = (logical.long() + 1) // ratio
        score = torch.rand((n, max(1, int(vis.max()), kb)), generator=g, device="cuda")
        score = torch.where(torch.arange(score.shape[1], device="cuda") < vis[:, None], score, -1.0)
        top = score.topk(kb, dim=1)
        sel = torch.where(top.values >= 0, top.indices, 1 << 40).sort(dim=1).values
        tok = (sel[:, :, None] * ratio + torch.arange(ratio, device="cuda")).reshape(n, -1)
        tail = vis[:, None] * ratio + torch.arange(ratio - 1, device="cuda")
        tok = torch.cat([tok, torch.where(tail <= logical[:, None], tail, 1 << 40)], 1).sort(dim=1).values
        ok = tok < (1 << 30)
        s["packed"] = torch.cat([torch.where(ok, tok, -1), ok.sum(1, keepdim=True)], 1).int().contiguous()
        assert s["packed"].shape[1] == width + 1
    else:
        # the rows in tiles of one request each, for the plain form
        t = max(1, min(128, max(rows)))
        s["tile"] = t
        tiles = [(i, starts[i] + a, min(t, r - a)) for i, r in enumerate(rows) for a in range(0, r, t)]
        s["tiles"] = torch.tensor(tiles, dtype=torch.int64).cuda()
    return s


# ------------------------------------------------------------------ the plain forms

def _values(kv, scales, case):
    """Cache rows [..., tokens, 256] in 32 bits."""
    if case["kv"] == "bf16":
        return kv.float()
    x = kv.view(torch.float8_e4m3fn).float()
    if case["kv"] == "e4m3":
        return x * STATIC
    return x.unflatten(-1, (2, D)).mul_(torch.exp2(scales.float() - 127.0)[..., None]).flatten(-2)


def _gather(s, req, tok):
    """K|V [n, Hkv, L, 256] of tokens tok [n, L] (in range) of requests req [n]."""
    case, page = s["case"], s["case"]["page"]
    blk = s["table"][req[:, None], tok // page].long()
    head = torch.arange(case["hkv"], device="cuda")[None, :, None]
    row = (blk[:, None] * case["hkv"] + head) * page + (tok % page)[:, None]
    kv = s["kv"].view(-1, 2 * D)[row]
    sc = None
    if s["scales"] is not None:
        sc = s["scales"].view(-1, 2)[row // case["block"]]
    return _values(kv, sc, case)


def _attend(q, kv, mask):
    """q [n, Hkv, M, D] over kv [n, Hkv, L, 2 D], mask [n, 1, M, L] of what is seen."""
    p = (q @ kv[..., :D].transpose(-1, -2)).mul_(D ** -0.5).masked_fill_(~mask, -math.inf)
    m = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    return (p @ kv[..., D:]) / p.sum(-1, keepdim=True).clamp_min(1e-30)


def _gated(s, a):
    a = a.bfloat16()
    return a if s["gate"] is None else (a.float() * torch.sigmoid(s["gate"].float())).bfloat16()


def _plain_sparse(s):
    case, n = s["case"], s["rows"]
    g = case["hq"] // case["hkv"]
    tok = s["packed"][:, :-1].long()
    seen = torch.arange(tok.shape[1], device="cuda") < s["packed"][:, -1:]
    kv = _gather(s, s["t2r"].long(), tok.clamp_min(0))
    q = s["q"].float().view(n, case["hkv"], g, D)
    return _gated(s, _attend(q, kv, seen[:, None, None]).reshape(n, case["hq"], D))


def _plain_window(s):
    case, t = s["case"], s["tile"]
    hkv, g, w = case["hkv"], case["hq"] // case["hkv"], case["window"]
    sinks = min(case["sinks"], s["max_context"])
    req, row0, count = s["tiles"].unbind(1)
    row = row0[:, None] + torch.arange(t, device="cuda")
    live = torch.arange(t, device="cuda") < count[:, None]
    row = torch.where(live, row, row0[:, None])
    pos = s["logical"].long()[row]                                   # [tiles, t]
    base = (pos[:, :1] - w + 1).clamp_min(0)
    length = min(w + t - 1, s["max_context"])
    tok = torch.cat([torch.arange(sinks, device="cuda").expand(len(req), -1), base + torch.arange(length, device="cuda")], 1)
    first = torch.arange(sinks + length, device="cuda") < sinks      # the sinks' own columns
    near = (tok[:, None] > pos[..., None] - w) & ((tok >= sinks) & ~first)[:, None]
    seen = (tok[:, None] <= pos[..., None]) & (near | first)
    kv = _gather(s, req, torch.minimum(tok, pos.amax(1, keepdim=True)))
    q = s["q"].float()[row].view(-1, t, hkv, g, D).transpose(1, 2).reshape(-1, hkv, t * g, D)
    o = _attend(q, kv, seen.repeat_interleave(g, 1)[:, None])
    o = o.view(-1, hkv, t, g, D).transpose(1, 2).reshape(-1, t, hkv * g, D)
    return _gated(s, o[live])


def _norm_rope(x, w, pos, cos_sin, mrope):
    """Gemma RMSNorm of x [n, heads, D], then rotation of the first ROT dims at pos [n, 3]."""
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (1.0 + w.float())
    i = torch.arange(ROT // 2, device="cuda")
    comp = torch.zeros_like(i)
    if mrope:
        comp = torch.where((i % 3 == 1) & (i < 3 * SECTIONS[1]), 1, torch.where((i % 3 == 2) & (i < 3 * SECTIONS[2]), 2, 0))
    at = pos[:, comp]
    c, sn = cos_sin[at, i][:, None], cos_sin[at, i + ROT // 2][:, None]
    a, b = x[..., :ROT // 2], x[..., ROT // 2:ROT]
    return torch.cat([a * c - b * sn, b * c + a * sn, x[..., ROT:]], -1)


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _plain_append(s):
    case, n = s["case"], s["rows"]
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    x = s["qkv"].view(n, 2 * hq + 2 * hkv, D)
    pos = s["positions"].view(n, 3)
    out = {}
    if case["q"]:
        s["q_out"].copy_(_norm_rope(x[:, 0:2 * hq:2], s["q_norm_w"], pos, s["cos_sin"], case["mrope"]))
        s["gate_out"].copy_(x[:, 1:2 * hq:2])
        out = {"q": s["q_out"], "gate": s["gate_out"]}
    k = _norm_rope(x[:, 2 * hq:2 * hq + hkv], s["k_norm_w"], pos, s["cos_sin"], case["mrope"])
    new = torch.cat([k, x[:, 2 * hq + hkv:].float()], -1)             # [n, Hkv, 2 D]
    blk, off = s["slots"] // page, s["slots"] % page
    if case["kv"] == "bf16":
        s["kv"][blk, :, off] = new.bfloat16()
        return {**out, "kv": s["kv"]}
    codes = s["kv"].view(torch.float8_e4m3fn)
    if case["kv"] == "e4m3":
        s["kv"][blk, :, off] = _e4m3(new / STATIC).view(torch.uint8)
        return {**out, "kv": codes}
    # runs: consecutive rows whose slots lie in one scale block
    b = case["block"]
    group = s["slots"] // b
    start = torch.ones(n, dtype=torch.bool, device="cuda")
    start[1:] = group[1:] != group[:-1]
    run = start.long().cumsum(0) - 1                                  # [n]
    peak = torch.zeros((n, hkv, 2), device="cuda")                    # at most n runs
    peak.scatter_reduce_(0, run[:, None, None].expand(-1, hkv, 2), new.view(n, hkv, 2, D).abs().amax(-1), "amax")
    m, e = torch.frexp(peak)
    e = torch.where(peak == 0, -40, torch.where(m <= 0.875, e - 9, e - 8)).clamp(-40, 40)
    # each run's place; unused runs repeat the last row's
    lead = torch.full((n,), n - 1, dtype=torch.long, device="cuda")
    lead.scatter_reduce_(0, run, torch.arange(n, device="cuda"), "amin")
    rb, rsub, f = blk[lead], off[lead] // b, off[lead] % b
    spare = torch.arange(n, device="cuda") > run[-1]
    e = torch.where(spare[:, None, None], e[run[-1]], e)
    rb, rsub, f = (torch.where(spare, v[run[-1]], v) for v in (rb, rsub, f))
    old = s["scales"][rb, :, rsub].int() - 127
    e = torch.where((f == 0)[:, None, None], e, torch.maximum(e, old))
    view = s["kv"].view(-1, hkv, page // b, b, 2, D)
    before = view[rb, :, rsub]                                        # [n, Hkv, b, 2, D]
    again = _e4m3(before.view(torch.float8_e4m3fn).float() * torch.exp2((old - e).float())[:, :, None, :, None]).view(torch.uint8)
    keep = torch.arange(b, device="cuda") < f[:, None]
    view[rb, :, rsub] = torch.where(keep[:, None, :, None, None], again, before)
    s["scales"][rb, :, rsub] = (e + 127).to(torch.uint8)
    scaled = new.view(n, hkv, 2, D) * torch.exp2(-e[run].float())[..., None]
    s["kv"][blk, :, off] = _e4m3(scaled.view(n, hkv, 2 * D)).view(torch.uint8)
    return {**out, "kv": codes, "scales": s["scales"].view(torch.float8_e8m0fnu)}


# ------------------------------------------------------------------ the framework's calls

def _handle(s):
    """What a user's program keeps between calls: configurations, argument structs, the workspace."""
    from learned_sparse_attention_gb300 import qsa as Q

    case = s["case"]
    dtype = {"bf16": Q.DTYPE_BF16, "e4m3": Q.DTYPE_E4M3, "block": Q.DTYPE_E4M3_BLOCK}[case["kv"]]
    gcfg = Q.make_gqa_cfg(case["hq"], case["hkv"], case["page"], s["kv"].shape[0], kv_dtype=dtype, k_scale=STATIC, v_scale=STATIC)
    scales = Q.kv_scales(s["scales"], case["block"]) if s["scales"] is not None else None
    h = dict(Q=Q, gcfg=gcfg, scales=scales)
    if case["op"] == "append":
        h["cfg"] = Q.make_cfg(8, 4, 64, Q.DTYPE_BF16, 4, s["cos_sin"].shape[0],
                              mrope_section=SECTIONS if case["mrope"] else (0, 0, 0), eps=EPS)
        t = dict(main_qkv=s["qkv"], main_q_norm_w=s["q_norm_w"], main_k_norm_w=s["k_norm_w"], kv=s["kv"], slot_mapping=s["slots"])
        if case["q"]:
            t.update(main_q_out=s["q_out"], main_gate_out=s["gate_out"])
        h["main"] = Q.main_prep(t, EPS)
    elif case["op"] == "sparse":
        cfg = Q.make_cfg(8, case["ratio"], case["topk"], Q.DTYPE_BF16, 4, 1)
        h["ws"] = torch.empty(Q.workspace_bytes(cfg, gcfg, s["rows"], s["reqs"], 1), dtype=torch.uint8, device="cuda")
    else:
        h["args"] = Q.window_args(s["q"], s["kv"], s["table"], s["t2r"], s["qsl"], s["logical"], s["out"], case["window"],
                                  case["sinks"], s["max_context"], gate=s["gate"], scales=scales)
        h["ws"] = torch.empty(Q.window_workspace_bytes(gcfg, h["args"]), dtype=torch.uint8, device="cuda")
    return h


def _own(s):
    if "handle" not in s:
        s["handle"] = _handle(s)
    h, case = s["handle"], s["case"]
    Q = h["Q"]
    if case["op"] == "append":
        Q.kv_append(h["cfg"], h["gcfg"], h["main"], s["positions"], s["cos_sin"], scales=h["scales"])
        out = {"q": s["q_out"], "gate": s["gate_out"]} if case["q"] else {}
        out["kv"] = s["kv"] if case["kv"] == "bf16" else s["kv"].view(torch.float8_e4m3fn)
        if case["kv"] == "block":
            out["scales"] = s["scales"].view(torch.float8_e8m0fnu)
        return out
    if case["op"] == "sparse":
        Q.sparse_gqa_scaled(h["gcfg"], h["scales"], s["q"], s["kv"], s["table"], s["packed"], s["t2r"], s["gate"], s["out"], h["ws"])
    else:
        Q.window_gqa(h["gcfg"], h["args"], h["ws"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "sparse": _plain_sparse, "window": _plain_window}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    rows, ctx = _lengths(case)
    n, hq, hkv = sum(rows), case["hq"], case["hkv"]
    item = 4 * D if case["kv"] == "bf16" else 2 * D                   # K and V of a token and KV head
    scale = 2.0 / case["block"] if case["kv"] == "block" else 0.0
    if case["op"] == "append":
        read = n * (2 * hkv + (2 * hq if case["q"] else 0)) * D * 2 + n * (8 + 24)
        write = n * hkv * (item + scale) + (n * 2 * hq * D * 2 if case["q"] else 0)
        return {"bytes": read + write, "flops": n * (hkv + (hq if case["q"] else 0)) * D * 8}
    io = n * hq * D * 2 * (3 if case["gate"] else 2)
    if case["op"] == "sparse":
        seen = 0
        for r, c in zip(rows, ctx):
            for p in range(c - r, c):
                v, kb = (p + 1) // case["ratio"], case["topk"] // case["ratio"]
                seen += min(v, kb) * case["ratio"] + (p + 1) % case["ratio"]
        # rows of one request may share what they select: at the least one row's is read
        once = sum(min(c, case["topk"] + case["ratio"] - 1) for c in ctx)
        return {"bytes": io + once * hkv * (item + scale) + n * (case["topk"] + case["ratio"]) * 4, "flops": 4 * D * hq * seen}
    w, sinks = case["window"], case["sinks"]
    seen = once = 0
    for r, c in zip(rows, ctx):
        for p in range(c - r, c):
            lo = max(0, p - w + 1)
            seen += p + 1 - lo + min(sinks, lo)
        lo = max(0, c - r - w + 1)
        once += c - lo + min(sinks, lo)
    return {"bytes": io + once * hkv * (item + scale), "flops": 4 * D * hq * seen}


# ------------------------------------------------------------------ the definitions in 64 bits

def _x_dense(s, req, lo, hi):
    """K, V of tokens lo..hi-1 of a request, [Hkv, n, D] each, page by page from the table."""
    case, page = s["case"], s["case"]["page"]
    pages = s["table"][req, lo // page:(hi - 1) // page + 1].long()
    kv = s["kv"].index_select(0, pages)
    if case["kv"] == "bf16":
        x = kv.double()
    else:
        x = kv.view(torch.float8_e4m3fn).double()
        if case["kv"] == "e4m3":
            x = x * STATIC
        else:
            e = s["scales"].index_select(0, pages).double() - 127.0       # [pages, Hkv, page / block, 2]
            e = e.repeat_interleave(case["block"], 2).repeat_interleave(D, 3)
            x = x * 2.0 ** e
    x = x.transpose(0, 1).flatten(1, 2)[:, lo % page:lo % page + hi - lo]
    return x[..., :D], x[..., D:]


def _x_softmax(q, k, v, seen):
    """q [Hkv, R, G, D], k and v [Hkv, n, D], seen [R, n]."""
    z = torch.einsum("hrgd,hnd->hrgn", q, k) / math.sqrt(D)
    z = torch.where(seen[None, :, None], z, -math.inf)
    top = torch.amax(z, -1, keepdim=True)
    e = torch.exp(z - torch.where(torch.isfinite(top), top, 0.0))
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("hrgn,hnd->hrgd", e, v)
    return torch.where(total > 0, o / total, 0.0)


def _x_attention(s):
    case = s["case"]
    hkv, g = case["hkv"], case["hq"] // case["hkv"]
    rows, ctx = _lengths(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for req, (r, c) in enumerate(zip(rows, ctx)):
        step = 256 if case["op"] == "window" else 16
        for a in range(0, r, step):
            b = min(r, a + step)
            p = torch.arange(c - r + a, c - r + b, device="cuda")
            q = s["q"][at + a:at + b].double().view(b - a, hkv, g, D).transpose(0, 1)
            if case["op"] == "window":
                lo = max(0, c - r + a - case["window"] + 1)
                hi = c - r + b
                head = min(case["sinks"], lo)
                k, v = _x_dense(s, req, lo, hi)
                t = torch.arange(lo, hi, device="cuda")
                if head:
                    k0, v0 = _x_dense(s, req, 0, head)
                    k, v = torch.cat([k0, k], 1), torch.cat([v0, v], 1)
                    t = torch.cat([torch.arange(head, device="cuda"), t])
                seen = (t <= p[:, None]) & ((p[:, None] - t < case["window"]) | (t < case["sinks"]))
            else:
                k, v = _x_dense(s, req, 0, c)
                seen = torch.zeros((b - a, c), dtype=torch.bool, device="cuda")
                for i in range(a, b):
                    row = s["packed"][at + i]
                    seen[i - a, row[:int(row[-1])].long()] = True
            out[at + a:at + b] = _x_softmax(q, k, v, seen).transpose(0, 1).reshape(b - a, case["hq"], D)
        at += r
    if s["gate"] is not None:
        out = out / (1.0 + torch.exp(-s["gate"].double()))
    return out


def _x_round(x):
    """The nearest e4m3 value, ties to even, at most 448 (64 bits)."""
    a = x.abs().clamp_max(448.0)
    step = torch.exp2(torch.clamp_min(torch.floor(torch.log2(a.clamp_min(1e-300))), -6.0) - 3.0)
    return torch.sign(x) * torch.clamp_max(torch.round(a / step) * step, 448.0)


def _x_rotate(x, w, s):
    """Norm and rotation as a product of complex numbers."""
    x = x.double()
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * (w.double() + 1.0)
    pos = s["positions"].view(-1, 3)
    turn = []
    for i in range(ROT // 2):
        axis = 0
        if s["case"]["mrope"]:
            axis = 1 if i % 3 == 1 and i < 3 * SECTIONS[1] else 2 if i % 3 == 2 and i < 3 * SECTIONS[2] else 0
        row = s["cos_sin"].double()[pos[:, axis]]
        turn.append(torch.complex(row[:, i], row[:, ROT // 2 + i]))
    z = torch.complex(x[..., :ROT // 2], x[..., ROT // 2:ROT]) * torch.stack(turn, 1)[:, None]
    return torch.cat([z.real, z.imag, x[..., ROT:]], -1)


def _x_append(s):
    case = s["case"]
    n, hq, hkv, page, b = s["rows"], case["hq"], case["hkv"], case["page"], case["block"]
    x = s["qkv"].view(n, -1, D)
    out = {}
    if case["q"]:
        out["q"] = _x_rotate(x[:, :2 * hq].unflatten(1, (hq, 2))[:, :, 0], s["q_norm_w"], s)
        out["gate"] = x[:, :2 * hq].unflatten(1, (hq, 2))[:, :, 1].double()
    new = torch.stack([_x_rotate(x[:, 2 * hq:2 * hq + hkv], s["k_norm_w"], s), x[:, 2 * hq + hkv:].double()], 2)
    slots = s["slots"].tolist()
    flat = new.flatten(2)
    if case["kv"] != "block":
        kv = s["kv"].double() if case["kv"] == "bf16" else s["kv"].view(torch.float8_e4m3fn).double()
        at = torch.tensor(slots, device="cuda")
        kv[at // page, :, at % page] = flat if case["kv"] == "bf16" else _x_round(flat / STATIC)
        return {**out, "kv": kv}
    kv = s["kv"].view(torch.float8_e4m3fn).double()
    e = s["scales"].double() - 127.0
    i = 0
    while i < n:
        j = i + 1
        while j < n and slots[j] // b == slots[i] // b:
            j += 1
        blk, first = slots[i] // page, slots[i] % page
        sub, f = first // b, first % b
        top = new[i:j].abs().amax((0, 3))                             # [Hkv, 2]
        want = torch.where(top > 0, torch.ceil(torch.log2(top.clamp_min(1e-300) / 448.0)), -40.0).clamp(-40.0, 40.0)
        if f:
            now = torch.maximum(want, e[blk, :, sub])
            past = kv[blk, :, first - f:first].unflatten(-1, (2, D))
            kv[blk, :, first - f:first] = _x_round(past * 2.0 ** (e[blk, :, sub] - now)[:, None, :, None]).flatten(-2)
            want = now
        e[blk, :, sub] = want
        kv[blk, :, first:first + j - i] = _x_round(new[i:j] / 2.0 ** want[..., None]).flatten(2).transpose(0, 1)
        i = j
    return {**out, "kv": kv, "scales": 2.0 ** e}


def exact(case, seed):
    s = prepare(case, seed)
    return _x_append(s) if case["op"] == "append" else _x_attention(s)
