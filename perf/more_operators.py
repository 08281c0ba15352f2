"""What the operators of a layer's dense branch cost: appending keys and values to a paged
cache, causal attention of new tokens over it (all of it, or a sliding window and the first
tokens), joining the attention over disjoint keys, and the norm in front of the projections.

Each case is one pass through one operator as a serving loop calls it.  `own` picks the side:
elementary torch operations in 32 bits (False), or the framework's entry points (True).
`exact` computes the same outputs in 64 bits, straight from the definitions.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3_MAX = 448.0
SMALLEST = 2.0 ** -126          # smallest scale of a quantised vector
EPS = 1e-6


def listed():
    return [
        # a decode step: one token of each of 64 requests; latency counts
        dict(name="append step 64", op="append", requests=64, rows=1, keys=2048, heads=8, D=128,
             rot=64, layout="interleaved", dtype="bf16", kv="same", page=64),
        # a long-context chunk's keys and values into e4m3 caches
        dict(name="append chunk 16384", op="append", requests=1, rows=16384, keys=65536, heads=4,
             D=128, rot=128, layout="half", dtype="bf16", kv="fp8", page=64),
        # the smallest: the last 16 tokens of a short prompt, one shared key/value head
        dict(name="attend tiny", op="attend", requests=1, rows=16, keys=77, ragged=False, Hq=4,
             Hkv=1, D=64, window=0, sinks=0, dtype="fp16", kv="same", page=0),
        # a decode step of a dense layer: one token of each of 64 requests over 16,384 keys
        dict(name="attend step 64", op="attend", requests=64, rows=1, keys=16384, ragged=False,
             Hq=32, Hkv=4, D=128, window=0, sinks=0, dtype="bf16", kv="same", page=64),
        # a decode step of a window layer over e4m3 caches, small pages
        dict(name="attend step window", op="attend", requests=64, rows=1, keys=32768, ragged=False,
             Hq=64, Hkv=8, D=64, window=1024, sinks=4, dtype="bf16", kv="fp8", page=16),
        # a chunk of 2048 new tokens behind a cached prefix
        dict(name="attend chunk 2048", op="attend", requests=1, rows=2048, keys=31999,
             ragged=False, Hq=32, Hkv=4, D=128, window=0, sinks=0, dtype="bf16", kv="same",
             page=64),
        # three cold prompts of different lengths, packed keys, small heads
        dict(name="attend cold ragged", op="attend", requests=3, rows=7167, keys=7167, ragged=True,
             Hq=32, Hkv=8, D=64, window=0, sinks=0, dtype="fp16", kv="same", page=0),
        # a long-context chunk of a window layer, e4m3 caches
        dict(name="attend window 16384", op="attend", requests=1, rows=16384, keys=65536,
             ragged=False, Hq=64, Hkv=8, D=128, window=1024, sinks=4, dtype="bf16", kv="fp8",
             page=64),
        # a decode step's selected branch and window branch become one, with a learned logit
        # of attending to nothing
        dict(name="join step 64", op="join", rows=64, heads=32, D=128, parts=2, dtype="bf16",
             sink=True),
        # the same for a long-context chunk and three branches
        dict(name="join chunk 16384", op="join", rows=16384, heads=64, D=128, parts=3,
             dtype="bf16", sink=False),
        # the hidden states of a decode step: residual, norm and the projections' e4m3 operand
        dict(name="norm step 64", op="norm", rows=64, n=7168, dtype="bf16", residual=True,
             group=128),
        # the same for a long-context chunk
        dict(name="norm chunk 16384", op="norm", rows=16384, n=7168, dtype="bf16", residual=True,
             group=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "join", "norm"])
    if op == "append":
        D = rng.choice([64, 96, 128, 128])
        R = rng.choice([1, 1, 3, 64])
        keys = _log(rng, 64, 131072 // R)
        return dict(op=op, requests=R, rows=_log(rng, 1, min(keys, 16384 // R)), keys=keys,
                    heads=rng.choice([1, 2, 4, 8]), D=D, rot=rng.choice([D, D // 2]),
                    layout=rng.choice(["half", "interleaved"]),
                    dtype=rng.choice(["bf16", "bf16", "fp16"]), kv=rng.choice(["same", "fp8"]),
                    page=rng.choice([0, 1, 16, 48, 64]))
    if op == "join":
        rows, heads = _log(rng, 1, 16384), rng.choice([1, 4, 5, 32, 64])
        return dict(op=op, rows=rows, heads=heads, D=rng.choice([64, 128]),
                    parts=rng.choice([2, 2, 3]), dtype=rng.choice(["bf16", "bf16", "fp16"]),
                    sink=rng.random() < 0.5)
    if op == "norm":
        n = _log(rng, 64, 16384)
        group = rng.choice([0, 32, 128, 128])
        if group:
            n = max(1, n // group) * group
        return dict(op=op, rows=_log(rng, 1, 16384 * 7168 // max(n, 7168)), n=n,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    residual=rng.random() < 0.7, group=group)
    D, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 4, 5, 8, 16])
    R = rng.choice([1, 1, 2, 5, 32])
    keys = _log(rng, 16, 131072 // R)
    window = rng.choice([0, 0, 128, 1000, 4096])
    seen = min(keys, window + 8) if window else keys
    most = 2.5e11 / (4.0 * seen * Hq * D * R)              # rows a request may have
    rows = 1 if rng.random() < 0.35 else _log(rng, 1, max(1, min(keys, 16384 // R, int(most))))
    return dict(op=op, requests=R, rows=rows, keys=keys, ragged=rng.random() < 0.5, Hq=Hq, Hkv=Hkv,
                D=D, window=window, sinks=rng.choice([0, 4, 130]) if window else 0,
                dtype=rng.choice(["bf16", "bf16", "fp16"]), kv=rng.choice(["same", "fp8"]),
                page=rng.choice([0, 1, 16, 48, 64]))


# ------------------------------------------------------------------------------ inputs


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _lengths(c):
    """(new tokens, keys with them) of every request."""
    R = c["requests"]
    if not c.get("ragged"):
        return [(c["rows"], c["keys"])] * R
    keys = [max(1, c["keys"] * (i + 1) // R) for i in range(R)]
    return [(max(1, min(c["rows"] * (i + 1) // R, k)), k) for i, k in enumerate(keys)]


def _batch(c, g):
    """What a serving loop has of a batch: positions and causal lengths of its rows, its page
    table, its offsets on the host."""
    lens = _lengths(c)
    pos = torch.cat([torch.arange(k - n, k, dtype=torch.int32) for n, k in lens])
    cu_q = torch.tensor([0] + [n for n, _ in lens]).cumsum(0).int()
    cu_k = torch.tensor([0] + [k for _, k in lens]).cumsum(0).int()
    s = dict(case=c, pos=pos.to(DEV), lens=(pos + 1).to(DEV), host_lens=pos + 1, cu_q=cu_q,
             cu_k=cu_k, table=None, slots=int(cu_k[-1]))
    if c["page"] > 0:
        per = -(-c["keys"] // c["page"])
        R = c["requests"]
        s["table"] = torch.randperm(R * per, generator=g, device=DEV).to(torch.int32).reshape(R, per)
        s["slots"] = R * per * c["page"]
    if own:
        import sparse_attention_prefill_tcgen05_gb300 as K
        s["plan"] = K.indexer_plan(cu_q, cu_k, pos + 1, 32, 128, 64)
    return s


def _e4m3(x):
    """Codes and scales of vectors in 32 bits: scale = largest magnitude / 448."""
    amax = x.abs().amax(dim=-1, keepdim=True)
    s = torch.where(amax > 0, (amax / E4M3_MAX).clamp(min=SMALLEST), torch.ones_like(amax))
    return (x / s).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s.squeeze(-1)


def prepare(case, seed):
    c = dict(case)
    g = _generator(seed)
    return _PREPARE[c["op"]](c, g)


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _prepare_append(c, g):
    s = _batch(c, g)
    T, dt = s["pos"].shape[0], DT[c["dtype"]]
    s["k"], s["v"] = (_rand(g, T, c["heads"], c["D"]).to(dt) for _ in range(2))
    for name in ("kc", "vc"):                               # an occupied cache
        shape = (s["slots"], c["heads"], c["D"])
        if c["kv"] == "fp8":
            s[name] = torch.randint(0, 127, shape, generator=g, device=DEV, dtype=torch.uint8)
            s[name + "_scale"] = 0.005 + 0.01 * torch.rand(shape[:2], generator=g, device=DEV)
        else:
            s[name], s[name + "_scale"] = _rand(g, *shape).to(dt), None
    s["freq"] = _frequencies(c).to(DEV)
    if own:
        import sparse_attention_prefill_tcgen05_gb300 as K
        s["rope"] = K.indexer_rope_create(
            c["D"], c["rot"], layout=K.IDX_ROPE_HALF if c["layout"] == "half"
            else K.IDX_ROPE_INTERLEAVED, base=10000.0)
    return s


def _frequencies(c):
    return 10000.0 ** (-2.0 * torch.arange(c["rot"] // 2, dtype=torch.float64) / c["rot"])


def _prepare_attend(c, g):
    s = _batch(c, g)
    T, D, dt = s["pos"].shape[0], c["D"], DT[c["dtype"]]
    s["q"] = _rand(g, T, c["Hq"], D).to(dt)
    for name in ("k", "v"):
        x = _rand(g, s["slots"], c["Hkv"], D)
        if c["kv"] == "fp8":
            y, sc = _e4m3(x)
            s[name], s[name + "_scale"] = y.view(torch.uint8), sc.contiguous()
        else:
            s[name], s[name + "_scale"] = x.to(dt), None
        del x
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((T, c["Hq"]), dtype=torch.float32, device=DEV)
    if own:
        import sparse_attention_prefill_tcgen05_gb300 as K
        s["attn"] = K.indexer_causal_attention_create(
            s["plan"], c["Hq"], c["Hkv"], D, window=c["window"], sinks=c["sinks"],
            dtype=K.IDX_BF16 if c["dtype"] == "bf16" else K.IDX_FP16,
            kv_format=K.IDX_KV_FP8_E4M3 if c["kv"] == "fp8" else K.IDX_KV_DENSE,
            num_slots=s["slots"], page_size=c["page"])
        s["ws"] = torch.empty(max(256, s["attn"].workspace_bytes), dtype=torch.uint8, device=DEV)
    return s


def _prepare_join(c, g):
    shape, dt = (c["rows"], c["heads"], c["D"]), DT[c["dtype"]]
    s = dict(case=c, outs=[_rand(g, *shape).to(dt) for _ in range(c["parts"])])
    s["lses"] = [4.0 + 2.0 * _rand(g, *shape[:2]) for _ in range(c["parts"])]
    # a branch that has no key for a row
    for lse, o in zip(s["lses"][1:], s["outs"][1:]):
        none = torch.rand(shape[:2], generator=g, device=DEV) < 0.1
        lse.masked_fill_(none, -math.inf)
        o.masked_fill_(none[..., None], 0.0)
    s["sink"] = 2.0 + _rand(g, c["heads"]) if c["sink"] else None
    s["out"] = torch.empty(shape, dtype=dt, device=DEV)
    s["lse"] = torch.empty(shape[:2], dtype=torch.float32, device=DEV)
    return s


def _prepare_norm(c, g):
    shape, dt = (c["rows"], c["n"]), DT[c["dtype"]]
    s = dict(case=c, x=_rand(g, *shape).to(dt), weight=(1.0 + 0.2 * _rand(g, c["n"])).to(dt))
    # a few channels of a hidden state are far larger than the others
    s["residual"] = (_rand(g, *shape) * torch.exp2(2.0 * _rand(g, c["n"]))).to(dt) \
        if c["residual"] else None
    s["sum"] = torch.empty_like(s["x"]) if c["residual"] else None
    s["out"] = torch.empty_like(s["x"])
    s["codes"] = s["scales"] = None
    if c["group"]:
        s["codes"] = torch.empty(shape, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty((c["rows"], c["n"] // c["group"]), device=DEV)
    return s


_PREPARE = {"append": _prepare_append, "attend": _prepare_attend, "join": _prepare_join,
            "norm": _prepare_norm}


# ---------------------------------------------------------------------------- the passes


def run(state):
    return _RUN[state["case"]["op"]](state)


def _slots_of(s, r, j):
    """Cache slots of keys j (int64) of requests r (an int64 tensor, or one request)."""
    page = s["case"]["page"]
    if s["table"] is not None:
        return s["table"][r, j // page].long() * page + j % page
    return s["cu_k"].to(DEV).long()[r] + j


def _row_requests(s):
    n = (s["cu_q"][1:] - s["cu_q"][:-1]).to(DEV).long()
    return torch.repeat_interleave(torch.arange(n.shape[0], device=DEV), n,
                                   output_size=s["pos"].shape[0])


def _rotate(x, positions, freq, c):
    """Rotated vectors in 32 bits, the angles reduced in 64."""
    a = (positions.to(torch.float64)[:, None] * freq[None, :]) % (2 * math.pi)
    a = a.to(torch.float32)[:, None, :]
    cos, sin = torch.cos(a), torch.sin(a)
    r = c["rot"]
    y = x.clone()
    t = x[..., :r]
    if c["layout"] == "half":
        a, b = t[..., : r // 2], t[..., r // 2:]
        y[..., :r] = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    else:
        a, b = t[..., 0::2], t[..., 1::2]
        y[..., :r] = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    return y


def _append_outputs(s):
    if s["case"]["kv"] == "fp8":
        return (s["kc"].view(torch.float8_e4m3fn), s["kc_scale"],
                s["vc"].view(torch.float8_e4m3fn), s["vc_scale"])
    return s["kc"], s["vc"]


def _run_append(s):
    c = s["case"]
    if own:
        import sparse_attention_prefill_tcgen05_gb300 as K
        K.indexer_cache_append(s["plan"], s["k"], s["v"], s["kc"], s["vc"], s["pos"],
                               rope=s["rope"], page_table=s["table"], page_size=c["page"],
                               k_scale=s["kc_scale"], v_scale=s["vc_scale"])
        return _append_outputs(s)
    at = _slots_of(s, _row_requests(s), s["pos"].long())
    k, v = _rotate(s["k"].float(), s["pos"], s["freq"], c), s["v"].float()
    for name, x in (("kc", k), ("vc", v)):
        if c["kv"] == "fp8":
            y, sc = _e4m3(x)
            s[name][at] = y.view(torch.uint8)
            s[name + "_scale"][at] = sc
        else:
            s[name][at] = x.to(s[name].dtype)
    return _append_outputs(s)


def _pieces(s, most):
    """Rows [t0, t1) of requests r and the keys [0, s), [lo, hi) they see together."""
    c = s["case"]
    for r, (n, L) in enumerate(_lengths(c)):
        q0 = int(s["cu_q"][r])
        step = max(1, int(most / (c["Hq"] * min(L, c["window"] + c["sinks"] + 512 if c["window"]
                                                else L))))
        for i in range(0, n, step):
            m = min(step, n - i)
            first = L - n + i + 1                           # keys of the first row
            lo = max(0, first - c["window"]) if c["window"] else 0
            sinks = min(c["sinks"], lo)
            yield r, q0 + i, q0 + i + m, sinks, lo, first + m - 1


def _values(s, name, at, dtype):
    x = s[name][at]
    if s["case"]["kv"] == "fp8":
        return x.view(torch.float8_e4m3fn).to(dtype) * s[name + "_scale"][at].to(dtype)[..., None]
    return x.to(dtype)


def _visible(s, t0, t1, j):
    c = s["case"]
    n = s["lens"][t0:t1].long()[:, None]
    ok = j[None, :] < n
    if c["window"]:
        ok = ok & ((j[None, :] >= n - c["window"]) | (j[None, :] < c["sinks"]))
    return ok


def _run_attend(s):
    c = s["case"]
    if own:
        import sparse_attention_prefill_tcgen05_gb300 as K
        K.indexer_causal_attention(s["attn"], s["q"], s["k"], s["v"], s["lens"], s["out"], s["ws"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"],
                                   page_table=s["table"], lse=s["lse"])
        return s["out"], s["lse"]
    Hkv, D = c["Hkv"], c["D"]
    G = c["Hq"] // Hkv
    if c["rows"] == 1 and not c["ragged"]:
        pieces = _steps(s)
    else:
        pieces = (([r], t0, t1, sinks, lo, hi) for r, t0, t1, sinks, lo, hi in _pieces(s, 3e8))
    for rs, t0, t1, sinks, lo, hi in pieces:
        j = torch.cat([torch.arange(sinks, device=DEV), torch.arange(lo, hi, device=DEV)])
        B = len(rs)
        at = _slots_of(s, torch.tensor(rs, device=DEV)[:, None], j[None, :])          # [B, L]
        k = _values(s, "k", at, torch.float32).transpose(1, 2)                        # [B, Hkv, L, D]
        v = _values(s, "v", at, torch.float32).transpose(1, 2)
        n = (t1 - t0) // B
        q = s["q"][t0:t1].float().reshape(B, n, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, n * G, D)
        a = torch.matmul(q, k.transpose(2, 3)) * D ** -0.5
        ok = _visible(s, t0, t1, j).reshape(B, 1, n, 1, -1)
        a = a.reshape(B, Hkv, n, G, -1).masked_fill_(~ok, -math.inf)
        m = a.amax(dim=-1, keepdim=True)
        p = torch.exp(a - m.clamp(min=-3.0e38))
        z = p.sum(dim=-1, keepdim=True)
        o = torch.matmul(p.reshape(B, Hkv, n * G, -1), v).reshape(B, Hkv, n, G, D) / z.clamp(min=1e-30)
        s["out"][t0:t1] = o.transpose(1, 2).reshape(t1 - t0, c["Hq"], D).to(s["out"].dtype)
        s["lse"][t0:t1] = (m + torch.log(z)).transpose(1, 2).reshape(t1 - t0, c["Hq"])
    return s["out"], s["lse"]


def _steps(s):
    """Requests of one token each over as many keys, some at a time."""
    c = s["case"]
    lo = max(0, c["keys"] - c["window"]) if c["window"] else 0
    sinks = min(c["sinks"], lo)
    step = max(1, int(2e8 / ((c["keys"] - lo + sinks) * c["Hkv"] * c["D"])))
    for r in range(0, c["requests"], step):
        e = min(c["requests"], r + step)
        yield list(range(r, e)), r, e, sinks, lo, c["keys"]


def _run_join(s):
    if own:
        import sparse_attention_prefill_tcgen05_gb300 as K
        K.indexer_attention_join(s["outs"], s["lses"], s["out"], lse=s["lse"], sink=s["sink"])
        return s["out"], s["lse"]
    l = torch.stack(s["lses"])
    if s["sink"] is not None:
        l = torch.cat([l, s["sink"].expand_as(l[:1])])
    m = l.amax(dim=0)
    w = torch.exp(l - m.clamp(min=-3.0e38))
    z = w.sum(dim=0)
    o = sum(w[i][..., None] * s["outs"][i].float() for i in range(len(s["outs"])))
    o = o / z.clamp(min=1e-30)[..., None]
    return o.to(s["out"].dtype), m + torch.log(z)


def _norm_outputs(s, out, total, codes, scales):
    r = [out]
    if s["case"]["residual"]:
        r.append(total)
    if s["case"]["group"]:
        r += [codes, scales]
    return tuple(r)


def _run_norm(s):
    c = s["case"]
    if own:
        import sparse_attention_prefill_tcgen05_gb300 as K
        K.indexer_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], total=s["sum"],
                           out=s["out"], codes=s["codes"], scales=s["scales"])
        return _norm_outputs(s, s["out"], s["sum"],
                             s["codes"].view(torch.float8_e4m3fn) if c["group"] else None,
                             s["scales"])
    h = s["x"].float()
    if c["residual"]:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(dim=-1, keepdim=True) + EPS) * s["weight"].float()
    codes = scales = None
    if c["group"]:
        codes, scales = _e4m3(y.reshape(c["rows"], -1, c["group"]))
        codes = codes.reshape(y.shape)
    return _norm_outputs(s, y.to(s["x"].dtype), h.to(s["x"].dtype), codes, scales)


_RUN = {"append": _run_append, "attend": _run_attend, "join": _run_join, "norm": _run_norm}


# ------------------------------------------------------------------------- what it takes


def work(case):
    c = case
    eb = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "join":
        n = c["rows"] * c["heads"]
        return {"bytes": (c["parts"] + 1) * n * (2.0 * c["D"] + 4) + 4 * c["heads"] * c["sink"],
                "flops": 2.0 * n * c["D"] * c["parts"]}
    if c["op"] == "norm":
        n = c["rows"] * c["n"]
        per = eb * (4 if c["residual"] else 2) + (1 + 4.0 / c["group"] if c["group"] else 0)
        return {"bytes": n * per + eb * c["n"], "flops": 6.0 * n}
    if c["op"] == "append":
        T = c["requests"] * c["rows"]
        n = 2.0 * T * c["heads"]
        out = n * (c["D"] + 4) if c["kv"] == "fp8" else n * c["D"] * eb
        pages = min(T, c["requests"] * -(-c["rows"] // max(c["page"], 1))) if c["page"] else 0
        return {"bytes": n * c["D"] * eb + out + 4 * T + 4 * pages, "flops": 3.0 * n * c["rot"] / 2}
    pairs = rows = cached = 0
    for n, L in _lengths(c):
        rows += n
        if c["window"]:
            w, sk = c["window"], c["sinks"]
            pairs += sum(x if x <= w else w + min(sk, x - w) for x in range(L - n + 1, L + 1))
            lo = max(0, L - n + 1 - w)
            cached += L - lo + min(sk, lo)
        else:
            pairs += n * (L - n) + n * (n + 1) // 2
            cached += L
    vec = c["D"] + 4 if c["kv"] == "fp8" else 2 * c["D"]
    return {"bytes": rows * c["Hq"] * (4.0 * c["D"] + 4) + 4 * rows + 2.0 * cached * c["Hkv"] * vec
            + (4.0 * cached / c["page"] if c["page"] else 0),
            "flops": 4.0 * pairs * c["Hq"] * c["D"]}


# ------------------------------------------------------------------------------- 64 bits


def exact(case, seed):
    c = dict(case)
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    return _EXACT[c["op"]](c, s)


def _exact_e4m3(x):
    """The e4m3 values nearest to x / scale, in 64 bits: a step of 2^(e - 3) at 2^e <= |y|,
    2^-9 below 2^-6, ties to the even multiple."""
    amax = x.abs().amax(dim=-1, keepdim=True)
    s = torch.where(amax > 0, (amax / E4M3_MAX).clamp(min=SMALLEST), torch.ones_like(amax))
    y = x / s
    step = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=-6).double() - 3)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX), s.squeeze(-1)


def _exact_append(c, s):
    T = s["pos"].shape[0]
    host, cu_q = s["pos"].cpu(), s["cu_q"]
    at = torch.empty(T, dtype=torch.int64)
    for r in range(c["requests"]):
        p = host[cu_q[r]:cu_q[r + 1]].long()
        at[cu_q[r]:cu_q[r + 1]] = s["cu_k"][r] + p if s["table"] is None else \
            s["table"][r].cpu().long()[p // c["page"]] * c["page"] + p % c["page"]
    at = at.to(DEV)
    k = s["k"].double()
    half = c["rot"] // 2
    for i in range(half):
        a = s["pos"].double() * 10000.0 ** (-2.0 * i / c["rot"])
        co, si = torch.cos(a)[:, None], torch.sin(a)[:, None]
        p, q = (i, i + half) if c["layout"] == "half" else (2 * i, 2 * i + 1)
        u, v = s["k"][..., p].double(), s["k"][..., q].double()
        k[..., p], k[..., q] = u * co - v * si, u * si + v * co
    res = []
    for name, x in (("kc", k), ("vc", s["v"].double())):
        if c["kv"] == "fp8":
            y, sc = _exact_e4m3(x)
            full = s[name].view(torch.float8_e4m3fn).double()
            scale = s[name + "_scale"].double()
            full[at], scale[at] = y, sc
            res += [full, scale]
        else:
            full = s[name].double()
            full[at] = x
            res.append(full)
    return tuple(res)


def _exact_attend(c, s):
    T, D, G = s["pos"].shape[0], c["D"], c["Hq"] // c["Hkv"]
    out = torch.empty((T, c["Hq"], D), dtype=torch.float64, device=DEV)
    lse = torch.empty((T, c["Hq"]), dtype=torch.float64, device=DEV)
    for r, t0, t1, sinks, lo, hi in _pieces(s, 2e8):
        j = torch.cat([torch.arange(sinks, device=DEV), torch.arange(lo, hi, device=DEV)])
        at = _slots_of(s, r, j)
        n = s["lens"][t0:t1].long()
        seen = j[None, :] < n[:, None]
        if c["window"]:
            seen &= (j[None, :] >= (n - c["window"])[:, None]) | (j < c["sinks"])[None, :]
        for h in range(c["Hkv"]):
            kk, vv = s["k"][at, h], s["v"][at, h]
            if c["kv"] == "fp8":
                kk = kk.view(torch.float8_e4m3fn).double() * s["k_scale"][at, h].double()[:, None]
                vv = vv.view(torch.float8_e4m3fn).double() * s["v_scale"][at, h].double()[:, None]
            q = s["q"][t0:t1, h * G:(h + 1) * G].double()
            a = torch.matmul(q, kk.double().T) / math.sqrt(D)
            a.masked_fill_(~seen[:, None, :], -math.inf)
            lse[t0:t1, h * G:(h + 1) * G] = torch.logsumexp(a, dim=-1)
            out[t0:t1, h * G:(h + 1) * G] = torch.matmul(torch.softmax(a, dim=-1), vv.double())
    return out, lse


def _exact_join(c, s):
    l = [x.double() for x in s["lses"]]
    if s["sink"] is not None:
        l.append(s["sink"].double().expand_as(l[0]))
    lse = torch.logsumexp(torch.stack(l), dim=0)
    o = torch.zeros(s["outs"][0].shape, dtype=torch.float64, device=DEV)
    for x, y in zip(s["outs"], l):
        w = torch.where(torch.isinf(y), torch.zeros_like(y), torch.exp(y - lse))
        o += w[..., None] * x.double()
    return o, lse


def _exact_norm(c, s):
    h = s["x"].double()
    if c["residual"]:
        h = h + s["residual"].double()
    rms = torch.sqrt(h.square().sum(dim=-1, keepdim=True) / c["n"] + EPS)
    y = h / rms * s["weight"].double()
    codes = scales = None
    if c["group"]:
        codes, scales = _exact_e4m3(y.reshape(c["rows"], -1, c["group"]))
        codes = codes.reshape(y.shape)
    return _norm_outputs(s, y, h, codes, scales)


_EXACT = {"append": _exact_append, "attend": _exact_attend, "join": _exact_join,
          "norm": _exact_norm}
