"""Timing cases of the serving-step operators.

A step of a paged serving engine: the step's block tables and slot maps are
built from the request lengths (``pa_step_maps``), the queries and keys are
normalised per head, rotated to their positions and the keys and values
written to the paged pools (``pa_qk_rope``, ``pa_qk_rope_append``), and the
queries attend over a sliding window and the first tokens of their sequence
(``pa_decode_window`` for one new token, ``pa_prefill_window`` for several).

``run`` computes a case's operator in plain torch operations in 32 bits, or,
where ``own`` is true, with the library's entry points. ``exact`` computes it
in 64 bits from the definition.
"""

import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One step of 64 decoding requests: a single new token each.
        dict(name="step maps, 64 decoding", op="step", B=64, new_lo=1, new_hi=1, ctx_lo=512, ctx_hi=32767, bs=16,
             pad=0, mix=1),
        # A large mixed step: 1024 requests, from one new token to long
        # prompt chunks, rows padded to a multiple of 1024 for a graph.
        dict(name="step maps, 1024 mixed chunks", op="step", B=1024, new_lo=1, new_hi=2048, ctx_lo=1, ctx_hi=16384,
             bs=16, pad=1024, mix=2),
        # The rotation of one decode step's rows, q and k views of a fused
        # projection.
        dict(name="rope, 64 rows", op="rope", T=64, Hq=32, Hkv=8, D=128, rot=128, layout="half",
             dtype="bf16", scaling="none", far=131072, fused=True),
        # A long prompt's rows: interleaved pairs on half of the head, long
        # context scaling.
        dict(name="rope, 16421 rows", op="rope", T=16421, Hq=32, Hkv=8, D=128, rot=64,
             layout="interleaved", dtype="bf16", scaling="yarn", far=131072, fused=True),
        # Norm, rotation and cache write of one decode step of 64 requests.
        dict(name="norm rope append, 64 rows", op="append", T=64, Hq=32, Hkv=8, D=128, rot=128,
             layout="half", dtype="bf16", scaling="parts", far=131072, fused=True, norm=True, bs=16),
        # The same for 32k rows of prompt chunks.
        dict(name="norm rope append, 32768 rows", op="append", T=32768, Hq=32, Hkv=8, D=128, rot=128,
             layout="half", dtype="bf16", scaling="parts", far=131072, fused=True, norm=True, bs=16),
        # A decode step with a short window over contexts of any length.
        dict(name="window decode, 64 x 1024", op="decode", B=64, Hq=32, Hkv=8, D=128, bs=16,
             window=1024, sinks=4, ctx_lo=512, ctx_hi=32768, mix=3),
        # One request far into a long context: latency.
        dict(name="window decode, 1 x 8191", op="decode", B=1, Hq=64, Hkv=8, D=128, bs=32,
             window=8191, sinks=64, ctx_lo=131072, ctx_hi=131072, mix=4),
        # A large batch without head grouping: the most bytes.
        dict(name="window decode, 128 x 4096 MHA", op="decode", B=128, Hq=32, Hkv=32, D=128, bs=16,
             window=4096, sinks=4, ctx_lo=4096, ctx_hi=32768, mix=5),
        # Verification of a few drafted tokens per request.
        dict(name="window prefill, 64 x 6 rows", op="prefill", B=64, Hq=32, Hkv=8, D=128, bs=16,
             window=4096, sinks=4, new_lo=6, new_hi=6, ctx_lo=512, ctx_hi=32768, mix=6),
        # Prompt chunks of a mixed batch.
        dict(name="window prefill, 16 x 256 rows", op="prefill", B=16, Hq=32, Hkv=8, D=128, bs=16,
             window=2048, sinks=4, new_lo=256, new_hi=256, ctx_lo=1024, ctx_hi=16384, mix=7),
        # A whole long prompt at once.
        dict(name="window prefill, 16384 rows", op="prefill", B=1, Hq=32, Hkv=8, D=128, bs=16,
             window=4096, sinks=64, new_lo=16384, new_hi=16384, ctx_lo=16384, ctx_hi=16384, mix=8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _heads(rng, most_group=16):
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([g for g in (1, 2, 4, 8, 16) if g <= most_group])
    return Hkv * g, Hkv


def draw(rng):
    most = {c["op"]: 0.0 for c in listed()}
    for c in listed():
        most[c["op"]] = max(most[c["op"]], _cost(c))
    op = rng.choice(["step", "rope", "append", "decode", "prefill"])
    while True:
        mix = rng.randrange(1 << 20)
        if op == "step":
            lo = rng.choice([0, 1])
            c = dict(op=op, B=_log(rng, 1, 4096), new_lo=lo, new_hi=_log(rng, 1, 4096), ctx_lo=0,
                     ctx_hi=_log(rng, 1, 65536),
                     bs=rng.choice([16, 32]), pad=rng.choice([0, 64, 1024]), mix=mix)
        elif op in ("rope", "append"):
            Hq, Hkv = _heads(rng)
            D = rng.choice([64, 128])
            c = dict(op=op, T=_log(rng, 1, 65536), Hq=Hq, Hkv=Hkv, D=D,
                     rot=rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= D]),
                     layout=rng.choice(["half", "interleaved"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                     scaling=rng.choice(["none", "linear", "parts", "yarn"]),
                     far=_log(rng, 1024, 1 << 20), fused=rng.random() < 0.5)
            if op == "append":
                c.update(norm=rng.random() < 0.7, bs=rng.choice([16, 32]))
        elif op == "decode":
            Hq, Hkv = _heads(rng)
            lo = _log(rng, 1, 32768)
            c = dict(op=op, B=_log(rng, 1, 256), Hq=Hq, Hkv=Hkv, D=rng.choice([64, 128]),
                     bs=rng.choice([16, 32]), window=_log(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 17, 64]),
                     ctx_lo=lo, ctx_hi=max(lo, _log(rng, 64, 131072)), mix=mix)
        else:
            Hq, Hkv = _heads(rng)
            n = _log(rng, 1, 8192)
            c = dict(op=op, B=_log(rng, 1, 64), Hq=Hq, Hkv=Hkv, D=128, bs=rng.choice([16, 32]),
                     window=_log(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 17, 64]),
                     new_lo=max(1, n // rng.choice([1, 2, 8])), new_hi=n, ctx_lo=n,
                     ctx_hi=max(n, _log(rng, 64, 32768)), mix=mix)
        if _cost(c) <= most[op]:
            return c


# ------------------------------------------------------------------ shapes


def _lens(c):
    """(tokens cached before the step, new tokens) of every request, from the case alone."""
    r = random.Random(c["mix"])
    lo, hi = c["ctx_lo"], c["ctx_hi"]
    total = [_log(r, max(lo, 1), max(hi, 1)) if hi else 0 for _ in range(c["B"])]
    if c["op"] == "decode":
        return [x - 1 for x in total], [1] * c["B"]
    new = [0 if c["new_lo"] == 0 and r.random() < 0.1 else _log(r, max(1, c["new_lo"]), c["new_hi"])
           for _ in range(c["B"])]
    if c["op"] == "step":
        return total, new
    return [max(0, x - n) for x, n in zip(total, new)], new


def _rows(c):
    rows = sum(_lens(c)[1])
    pad = c["pad"]
    return max(1, -(-rows // pad) * pad if pad else rows)


def _pairs(c):
    """(visible tokens over all requests, visible (query, token) pairs)."""
    W, S = c["window"], c["sinks"]

    def seen(p):                        # tokens that the query at position p sees
        return min(p + 1, W) + min(S, max(0, p + 1 - W))

    tokens = pairs = 0
    for cached, n in zip(*_lens(c)):
        first, last = cached, cached + n - 1
        tokens += min(last + 1, (last + 1 - max(0, first + 1 - W)) + min(S, max(0, first + 1 - W)))
        # Positions below W see everything before them, the others W and the sinks.
        split = min(max(first, W), last + 1)
        pairs += (split * (split + 1) - first * (first + 1)) // 2
        mid = min(max(split, W + S), last + 1)
        pairs += sum(seen(p) for p in range(split, mid)) + (last + 1 - mid) * (W + S)
    return tokens, pairs


def work(case):
    c = case
    if c["op"] == "step":
        cached, new = _lens(c)
        bs = c["bs"]
        T = _rows(c)
        blocks = sum(-(-(x + n) // bs) + (-x // bs) for x, n in zip(cached, new))
        return {"bytes": 8 * c["B"] + 4 + 4 * blocks + 12 * T + 8 * c["B"] + 8 + 4 * blocks, "flops": T}
    e = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "rope":
        n = c["T"] * (c["Hq"] + c["Hkv"]) * c["D"]
        return {"bytes": 2 * n * e + 4 * c["T"], "flops": 3 * c["T"] * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["op"] == "append":
        n = c["T"] * (c["Hq"] + 2 * c["Hkv"]) * c["D"]
        return {"bytes": 2 * n * e + 12 * c["T"], "flops": 7 * c["T"] * (c["Hq"] + c["Hkv"]) * c["D"]}
    tokens, pairs = _pairs(c)
    rows = sum(_lens(c)[1])
    return {"bytes": 4 * c["Hkv"] * c["D"] * tokens + 4 * rows * c["Hq"] * c["D"]
            + 4 * (tokens // c["bs"] + 2 * c["B"]), "flops": 4 * c["D"] * c["Hq"] * pairs}


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


# ------------------------------------------------------------------ inputs


def _normal(shape, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype) \
        if math.prod(shape) < 1 << 28 else torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _perm(n, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randperm(n, generator=g, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _frequencies(c):
    """(radians a position of every rotated pair, factor on the rotated elements), 64 bits."""
    rot, base, factor, orig = c["rot"], 10000.0, 8.0, 8192.0
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if c["scaling"] == "none":
        return f, 1.0
    if c["scaling"] == "linear":
        return [x / factor for x in f], 1.0
    if c["scaling"] == "parts":          # between 1 and 4 turns over the trained length
        keep = [min(1.0, max(0.0, (orig * x / (2 * math.pi) - 1.0) / 3.0)) for x in f]
        return [k * x + (1 - k) * x / factor for k, x in zip(keep, f)], 1.0
    def at(turns):
        return rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
    low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
    high = high + 0.001 if low == high else high
    keep = [1 - min(1.0, max(0.0, (i - low) / (high - low))) for i in range(rot // 2)]
    return [k * x + (1 - k) * x / factor for k, x in zip(keep, f)], 0.1 * math.log(factor) + 1.0


def _rope(c):
    import paged_kv_cache_202_gb300 as pa
    kind = {"none": pa.PA_ROPE_NONE, "linear": pa.PA_ROPE_LINEAR, "parts": pa.PA_ROPE_PARTS,
            "yarn": pa.PA_ROPE_YARN}[c["scaling"]]
    lo, hi = (1.0, 4.0) if c["scaling"] == "parts" else (1.0, 32.0)
    return pa.Rope(c["rot"], layout=pa.PA_ROPE_HALF if c["layout"] == "half" else pa.PA_ROPE_INTERLEAVED,
                   base=10000.0, scaling=kind, factor=8.0, orig_len=8192, low_turns=lo, high_turns=hi)


def _prepare_step(c, seed):
    cached, new = _lens(c)
    B, bs = c["B"], c["bs"]
    had = [-(-x // bs) for x in cached]
    has = [-(-(x + n) // bs) for x, n in zip(cached, new)]
    NB = sum(has) + B
    MB = max(max(has), 1) + 3
    ids = _perm(NB, seed).to(torch.int32)
    col = torch.arange(MB, device="cuda")
    start = _i32([0] + had).cumsum(0)[:-1]
    at = start[:, None] + col[None, :]
    table = torch.where(col[None, :] < _i32(had)[:, None], ids[at.clamp(max=NB - 1)],
                        torch.full((), -1, dtype=torch.int32, device="cuda"))
    free = ids[sum(had):].contiguous()
    T = _rows(c)
    s = dict(case=c, T=T, MB=MB, NB=NB, cached=_i32(cached), new=_i32(new), table=table.contiguous(),
             free=free, count=_i32([free.numel()]), max_len=MB * bs)
    for name, n, dt in (("seq", B, torch.int32), ("start", B + 1, torch.int32), ("pos", T, torch.int32),
                        ("slots", T, torch.int64), ("left", 1, torch.int32)):
        s[name] = torch.zeros(n, dtype=dt, device="cuda")
    return s


def _prepare_rows(c, seed):
    T, Hq, Hkv, D, dt = c["T"], c["Hq"], c["Hkv"], c["D"], _DT[c["dtype"]]
    if c["fused"]:
        qkv = _normal((T, Hq + 2 * Hkv, D), dt, seed)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = (_normal((T, h, D), dt, seed + 7 * i) for i, h in enumerate((Hq, Hkv, Hkv)))
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    pos = torch.randint(0, c["far"], (T,), generator=g, device="cuda").to(torch.int32)
    s = dict(case=c, q=q, k=k, v=v, pos=pos, q_out=torch.zeros(T, Hq, D, dtype=dt, device="cuda"))
    f, s["amp"] = _frequencies(c)
    s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    s["rope"] = _rope(c) if own else None
    if c["op"] == "rope":
        s["k_out"] = torch.zeros(T, Hkv, D, dtype=dt, device="cuda")
        return s
    bs = c["bs"]
    NB = -(-T // bs) + 5
    s["slots"] = _perm(NB, seed + 2).repeat_interleave(bs)[:T] * bs + torch.arange(T, device="cuda") % bs
    s["k_pool"] = _normal((NB, Hkv, bs, D), dt, seed + 3)
    s["v_pool"] = _normal((NB, Hkv, bs, D), dt, seed + 4)
    s["qw"] = (1 + 0.2 * _normal((D,), torch.float32, seed + 5)).to(dt) if c["norm"] else None
    s["kw"] = (1 + 0.2 * _normal((D,), torch.float32, seed + 6)).to(dt) if c["norm"] else None
    return s


def _prepare_window(c, seed):
    cached, new = _lens(c)
    B, bs, W, S = c["B"], c["bs"], c["window"], c["sinks"]
    L = [x + n for x, n in zip(cached, new)]
    MB = max(-(-x // bs) for x in L) + 1
    # Blocks wholly behind every query's window have been given back.
    held = [sorted(set(range(min(-(-S // bs), -(-x // bs)))) | set(range(max(0, x - n + 1 - W) // bs, -(-x // bs))))
            for x, n in zip(L, new)]
    NB = sum(map(len, held)) + 3
    ids = _perm(NB, seed).to(torch.int32).cpu().numpy()
    table = np.full((B, MB), -1, dtype=np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, h] = ids[at:at + len(h)]
        at += len(h)
    T = sum(new)
    s = dict(case=c, L=L, new=new, q=_normal((T, c["Hq"], c["D"]), torch.bfloat16, seed + 1),
             k_pool=_normal((NB, c["Hkv"], bs, c["D"]), torch.bfloat16, seed + 2),
             v_pool=_normal((NB, c["Hkv"], bs, c["D"]), torch.bfloat16, seed + 3),
             table=torch.from_numpy(table).cuda(), lens=_i32(L), scale=c["D"] ** -0.5, max_len=max(L),
             max_q=max(new), out=torch.zeros(T, c["Hq"], c["D"], dtype=torch.bfloat16, device="cuda"))
    s["start"] = _i32(np.concatenate([[0], np.cumsum(new)]).tolist())
    if own:
        import paged_kv_cache_202_gb300 as pa
        s["plan"] = pa.Plan()
    return s


def prepare(case, seed):
    if case["op"] == "step":
        return _prepare_step(case, seed)
    if case["op"] in ("rope", "append"):
        return _prepare_rows(case, seed)
    return _prepare_window(case, seed)


# ------------------------------------------------------------------ the library's calls


def _own(s):
    import paged_kv_cache_202_gb300 as pa
    c = s["case"]
    if c["op"] == "step":
        pa.pa_step_maps(s["cached"], s["new"], s["free"], s["count"], s["table"], c["bs"], s["NB"],
                        s["max_len"], s["seq"], s["start"], s["pos"], s["slots"], s["left"])
        return [s["seq"], s["start"], s["pos"], s["slots"], s["table"], s["left"]]
    if c["op"] == "rope":
        pa.pa_qk_rope(s["q"], s["k"], s["pos"], s["rope"], s["q_out"], s["k_out"])
        return [s["q_out"], s["k_out"]]
    if c["op"] == "append":
        pa.pa_qk_rope_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["rope"], s["k_pool"],
                             s["v_pool"], s["q_out"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6)
        return [s["q_out"], s["k_pool"], s["v_pool"]]
    if c["op"] == "decode":
        return [pa.pa_decode_window(s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["scale"],
                                    c["window"], c["sinks"], s["out"], s["max_len"], s["plan"])]
    return [pa.pa_prefill_window(s["q"], s["start"], s["k_pool"], s["v_pool"], s["table"], s["lens"],
                                 s["scale"], c["window"], c["sinks"], s["out"], s["max_q"], s["max_len"],
                                 s["plan"])]


# ------------------------------------------------------------------ plain forms


def _plain_step(s):
    c, bs = s["case"], s["case"]["bs"]
    cached, new = s["cached"].long(), s["new"].long()
    seq = cached + new
    had, has = (cached + bs - 1) // bs, (seq + bs - 1) // bs
    need = has - had
    before = need.cumsum(0) - need
    col = torch.arange(s["MB"], device="cuda")[None, :]
    take = s["count"].long() - 1 - before[:, None] - (col - had[:, None])
    fresh = (col >= had[:, None]) & (col < has[:, None])
    table = torch.where(fresh, s["free"][take.clamp(0, s["free"].numel() - 1)], s["table"])
    start = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), new.cumsum(0)])
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=c["B"] - 1)
    real = t < start[-1]
    pos = torch.where(real, cached[b] + t - start[b], torch.zeros_like(t))
    slots = torch.where(real, table[b, (pos // bs).clamp(max=s["MB"] - 1)].long() * bs + pos % bs,
                        torch.full_like(t, -1))
    left = s["count"] - need.sum().int()
    return [seq.int(), start.int(), pos.int(), slots, table, left]


def _turned(x, pos, freq, amp, rot, layout):
    """The rotation, 32 bits; the angles and their sines in 64."""
    a = pos.double()[:, None, None] * freq
    cos, sin = (a.cos() * amp).float(), (a.sin() * amp).float()
    r = x[..., :rot]
    if layout == "half":
        x1, x2 = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
    else:
        x1, x2 = r[..., 0::2], r[..., 1::2]
        r = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_rows(s):
    c = s["case"]
    outs = []
    for x, w in ((s["q"], s.get("qw")), (s["k"], s.get("kw"))):
        y = x.float()
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        outs.append(_turned(y, s["pos"], s["freq"], s["amp"], c["rot"], c["layout"]).to(x.dtype))
    if c["op"] == "rope":
        return outs
    blk, off = s["slots"] // c["bs"], s["slots"] % c["bs"]
    s["k_pool"][blk, :, off] = outs[1]
    s["v_pool"][blk, :, off] = s["v"]
    return [outs[0], s["k_pool"], s["v_pool"]]


def _plain_decode(s):
    c = s["case"]
    W, S, bs, Hkv, D = c["window"], c["sinks"], c["bs"], c["Hkv"], c["D"]
    L = s["lens"].long()[:, None]
    W = min(W, s["max_len"])
    sink = torch.arange(S, device="cuda")[None, :].expand(c["B"], S)
    near = L - W + torch.arange(W, device="cuda")[None, :]
    tok = torch.cat([sink, near], 1)
    ok = torch.cat([sink < L, (near >= S) & (near >= 0)], 1)
    tok = torch.where(ok, tok, (L - 1).expand_as(tok))
    blk, off = s["table"].long().gather(1, tok // bs), tok % bs
    k, v = (p[blk, :, off].permute(0, 2, 1, 3).float() for p in (s["k_pool"], s["v_pool"]))
    q = s["q"].float().view(c["B"], Hkv, c["Hq"] // Hkv, D) * s["scale"]
    x = q @ k.transpose(2, 3)
    x = torch.where(ok[:, None, None, :], x, torch.full_like(x, -math.inf))
    x = torch.exp(x - x.amax(-1, keepdim=True))
    o = (x @ v) / x.sum(-1, keepdim=True)
    return [o.reshape(c["B"], c["Hq"], D).to(torch.bfloat16)]


def _plain_prefill(s):
    c = s["case"]
    W, S, bs, Hkv, D, g = c["window"], c["sinks"], c["bs"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    out = torch.empty_like(s["q"])
    row = 0
    for b, (L, n) in enumerate(zip(s["L"], s["new"])):
        for i in range(0, n, 1024):
            m = min(1024, n - i)
            first, last = L - n + i, L - n + i + m - 1
            lo = max(0, first + 1 - W)
            tok = torch.cat([torch.arange(min(S, lo), device="cuda"), torch.arange(lo, last + 1, device="cuda")])
            blk, off = s["table"][b, tok // bs].long(), tok % bs
            k, v = (p[blk, :, off].transpose(0, 1).float() for p in (s["k_pool"], s["v_pool"]))
            q = s["q"][row:row + m].float().view(m, Hkv, g, D).permute(1, 2, 0, 3).reshape(Hkv, g * m, D)
            p = torch.arange(first, last + 1, device="cuda")[:, None]
            ok = (tok <= p) & ((p - tok < W) | (tok < S))
            x = (q * s["scale"] @ k.transpose(1, 2)).view(Hkv, g, m, -1)
            x = torch.where(ok, x, torch.full((), -math.inf, device="cuda"))
            x = torch.exp(x - x.amax(-1, keepdim=True))
            o = (x.view(Hkv, g * m, -1) @ v).view(Hkv, g, m, D) / x.sum(-1, keepdim=True)
            out[row:row + m] = o.permute(2, 0, 1, 3).reshape(m, c["Hq"], D).to(torch.bfloat16)
            row += m
    return [out]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "step":
        return _plain_step(state)
    if op in ("rope", "append"):
        return _plain_rows(state)
    return _plain_decode(state) if op == "decode" else _plain_prefill(state)


# ------------------------------------------------------------------ 64 bits, from the definitions


def _exact_step(s):
    c, bs = s["case"], s["case"]["bs"]
    cached, new = s["cached"].tolist(), s["new"].tolist()
    table, free = s["table"].cpu().numpy().copy(), s["free"].tolist()
    pos, slots = np.zeros(s["T"], dtype=np.int32), np.full(s["T"], -1, dtype=np.int64)
    start, t = [0], 0
    for b in range(c["B"]):
        for p in range(cached[b], cached[b] + new[b]):
            if p % bs == 0:
                table[b, p // bs] = free.pop()
            pos[t], slots[t] = p, int(table[b, p // bs]) * bs + p % bs
            t += 1
        start.append(t)
    i = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return [i([x + n for x, n in zip(cached, new)]), i(start), torch.from_numpy(pos),
            torch.from_numpy(slots), torch.from_numpy(table), i([len(free)])]


def _exact_rows(s):
    c = s["case"]
    D, rot = c["D"], c["rot"]
    # Complex numbers: pair i of the rotated part times A e^(i pos f_i).
    f = s["freq"]
    a = s["pos"].double()[:, None] * f[None, :]
    z = torch.polar(torch.full_like(a, s["amp"]), a)[:, None, :]
    outs = []
    for x, w in ((s["q"], s.get("qw")), (s["k"], s.get("kw"))):
        y = x.double().clone()
        if w is not None:
            y *= torch.rsqrt(y.square().sum(-1, keepdim=True) / D + 1e-6)
            y *= w.double()
        i = torch.arange(rot // 2, device="cuda")
        re, im = (i, i + rot // 2) if c["layout"] == "half" else (2 * i, 2 * i + 1)
        r = torch.complex(y[..., re], y[..., im]) * z
        y[..., re], y[..., im] = r.real, r.imag
        outs.append(y)
    if c["op"] == "rope":
        return outs
    pools = []
    for p, rows in ((s["k_pool"], outs[1]), (s["v_pool"], s["v"].double())):
        flat = p.double().transpose(1, 2).reshape(-1, c["Hkv"], D)   # [slot, head, D]
        flat.index_copy_(0, s["slots"], rows)
        pools.append(flat.view(-1, c["bs"], c["Hkv"], D).transpose(1, 2).contiguous())
    return [outs[0]] + pools


def _exact_attention(s):
    """Request by request, kv head by kv head, over the pages that some query sees."""
    c = s["case"]
    W, S, bs, Hkv, g, D = c["window"], c["sinks"], c["bs"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (L, n) in enumerate(zip(s["L"], s["new"])):
        for i in range(0, n, 512):
            m = min(512, n - i)
            p = L - n + i + torch.arange(m, device="cuda")
            end = -(-(L - n + i + m) // bs)
            far = max(0, L - n + i + 1 - W) // bs
            page = sorted(set(range(min(-(-S // bs), end))) | set(range(far, end)))
            page = torch.tensor(page, device="cuda")
            tok = (page[:, None] * bs + torch.arange(bs, device="cuda")).flatten()
            gap = p[:, None] - tok
            hidden = (gap < 0) | ((gap >= W) & (tok >= S))
            phys = s["table"][b].long()[page]
            for h in range(Hkv):
                k, v = (x[phys, h].reshape(-1, D).double() for x in (s["k_pool"], s["v_pool"]))
                q = s["q"][row:row + m, h * g:(h + 1) * g].double()
                x = torch.einsum("mgd,td->gmt", q, k) * s["scale"]
                x.masked_fill_(hidden, -math.inf)
                x -= torch.logsumexp(x, -1, keepdim=True)
                out[row:row + m, h * g:(h + 1) * g] = torch.einsum("gmt,td->mgd", x.exp_(), v)
            row += m
    return [out]


def exact(case, seed):
    c = dict(case)
    if c["op"] in ("decode", "prefill") and work(c)["flops"] > 6e12:
        return None
    s = prepare(c, seed)
    if c["op"] == "step":
        return _exact_step(s)
    return _exact_rows(s) if c["op"] in ("rope", "append") else _exact_attention(s)
