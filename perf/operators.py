"""What the operators around the indexer cost: rotary positions, quantised operands and
caches, and attention over the selected keys.

Each case is one pass through one operator as a serving loop calls it.  `own` picks the
side: elementary torch operations in 32 bits (False), or the framework's entry points
(True).  `exact` computes the same outputs in 64 bits, straight from the definitions.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3_MAX = 448.0
SMALLEST = 2.0 ** -126          # smallest scale of a quantised row
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)      # e2m1 magnitudes by code


def listed():
    return [
        # the queries of a decode step: one token of each of 64 requests, the last half of
        # every head rotated; latency counts
        dict(name="rope step 64", op="rope", rows=64, heads=32, D=128, rot=64, offset=64,
             layout="interleaved", dtype="bf16", ctx=200000, factor=1.0, inverse=False),
        # the queries of a long-context chunk, positions scaled for a context 16 times the
        # trained one
        dict(name="rope chunk 16384", op="rope", rows=16384, heads=32, D=128, rot=128, offset=0,
             layout="half", dtype="bf16", ctx=487936, factor=16.0, inverse=False),
        # a ragged batch of few heads of an odd size, fp32, rotated back
        dict(name="rope odd fp32", op="rope", rows=7001, heads=5, D=80, rot=48, offset=16,
             layout="half", dtype="fp32", ctx=65536, factor=4.0, inverse=True),
        # the indexer's queries of a long-context chunk: rotated and quantised to e4m3 with a
        # scale per head vector
        dict(name="quantise queries e4m3", op="quant", rows=16384, heads=32, D=128, rot=64,
             offset=0, layout="interleaved", dtype="bf16", ctx=487936, factor=1.0, fmt="fp8"),
        # the same for e2m1 queries with a scale per 32 elements, one low-ratio chunk
        dict(name="quantise queries e2m1", op="quant", rows=2048, heads=32, D=128, rot=64,
             offset=0, layout="half", dtype="bf16", ctx=200000, factor=1.0, fmt="fp4"),
        # one new key of each of 64 requests written to a paged cache, and read back
        dict(name="cache step 64", op="cache", rows=64, heads=1, D=128, rot=64, offset=0,
             layout="interleaved", dtype="bf16", ctx=150000, factor=1.0, fmt="fp8",
             slots=131072, page=64, read=64),
        # a 2048-row chunk's keys written behind a cached prefix of 150,000, and the whole
        # prefix read back
        dict(name="cache prefix 152048", op="cache", rows=2048, heads=1, D=128, rot=64, offset=0,
             layout="interleaved", dtype="bf16", ctx=152048, factor=1.0, fmt="fp8",
             slots=262144, page=64, read=152048),
        # the smallest: 64 rows ending a 1024-token prompt, four heads of 64, four 8-key blocks
        # each, named by the candidate mask
        dict(name="attend tiny", op="attend", requests=1, rows=64, keys=1024, Hq=4, Hkv=1, D=64,
             block=8, sel=4, dtype="fp16", kv="same", page=0, mask=True),
        # a decode step: one token of each of 64 requests over 2048 selected keys of a paged
        # e4m3 cache
        dict(name="attend step 64", op="attend", requests=64, rows=1, keys=32768, Hq=32, Hkv=1,
             D=128, block=1, sel=2048, dtype="bf16", kv="fp8", page=64, mask=False),
        # a cold 64K chunk, 2048 selected keys a row
        dict(name="attend cold 2048", op="attend", requests=1, rows=2048, keys=65536, Hq=32, Hkv=1,
             D=128, block=1, sel=2048, dtype="bf16", kv="same", page=0, mask=False),
        # two prompts, grouped heads, 8-key blocks named by the candidate mask
        dict(name="attend blocks ragged", op="attend", requests=2, rows=1024, keys=7167, Hq=32,
             Hkv=4, D=64, block=8, sel=64, dtype="bf16", kv="same", page=48, mask=True),
        # a long-context chunk: 16,384 rows, 512 selected keys each of 487,936, paged e4m3 cache
        dict(name="attend long 16384", op="attend", requests=1, rows=16384, keys=487936, Hq=64,
             Hkv=1, D=128, block=1, sel=512, dtype="bf16", kv="fp8", page=64, mask=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "quant", "cache", "attend", "attend", "attend"])
    if op in ("rope", "quant", "cache"):
        D = rng.choice([64, 128, 128] if op != "rope" else [64, 80, 96, 128, 128])
        rot = rng.choice([D, D // 2])
        c = dict(op=op, rows=_log(rng, 1, 16384), heads=rng.choice([1, 4, 8, 16, 32]), D=D, rot=rot,
                 offset=rng.choice([0, D - rot]), layout=rng.choice(["half", "interleaved"]),
                 dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                 ctx=_log(rng, 1024, 487936), factor=rng.choice([1.0, 4.0, 16.0]))
        if op == "rope":
            return dict(c, inverse=rng.random() < 0.3)
        c["fmt"] = rng.choice(["fp8", "fp8", "fp4"])
        if op == "quant":
            return c
        c["heads"] = rng.choice([1, 1, 4])
        slots = _log(rng, 4096, 262144)
        c["rows"] = min(c["rows"], slots // 2)
        page = rng.choice([1, 16, 48, 64])
        return dict(c, slots=slots, page=page, read=rng.randint(1, slots // 2))
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 1, 2, 4])
    block = rng.choice([1, 1, 8, 64])
    mask = block == 8 and rng.random() < 0.5
    keys = _log(rng, 64, 200000)
    picked = _log(rng, 16, 2048)                       # keys a row may attend to
    sel = max(1, picked // block)
    requests = rng.choice([1, 1, 2, 5, 32])
    keys = max(1, min(keys, 400000 // requests))
    most = 4000000 // (sel * block * Hkv)
    rows = _log(rng, 1, max(1, min(4096, keys, most) // requests)) if rng.random() < 0.7 else 1
    return dict(op="attend", requests=requests, rows=min(rows, keys), keys=keys,
                Hq=Hkv * rng.choice([1, 4, 8, 16, 32]), Hkv=Hkv, D=D, block=block, sel=sel,
                dtype=rng.choice(["bf16", "bf16", "fp16"]), kv=rng.choice(["same", "fp8"]),
                page=rng.choice([0, 1, 48, 64]), mask=mask)


# ------------------------------------------------------------------------------ inputs


def _frequencies(c):
    """Angle per position of each rotated pair, 64 bits.  With factor > 1 the pairs that turn
    at most once over the trained context (4096 positions) are slowed by the factor, those
    that turn at least 32 times are kept, and the ones between are mixed linearly."""
    n = c["rot"] // 2
    i = torch.arange(n, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / c["rot"])
    if c["factor"] > 1.0:
        def pair_of(turns):
            return c["rot"] * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
        lo = max(math.floor(pair_of(32.0)), 0)
        hi = min(math.ceil(pair_of(1.0)), c["rot"] - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / c["factor"] * ramp + f * (1 - ramp)
    return f


def _amplitude(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["factor"] > 1.0 else 1.0


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _rand_perm(n, g):
    return torch.randperm(n, generator=g, device=DEV)


def _spread(n, rows_len, g):
    """n distinct ascending indices below each row's length, one from each of n equal parts
    of it (all of them, then -1, where the length is at most n)."""
    L = rows_len.to(torch.int64)[:, None]
    i = torch.arange(n, device=DEV, dtype=torch.int64)[None, :]
    lo, hi = i * L // n, (i + 1) * L // n
    u = torch.rand((L.shape[0], n), generator=g, device=DEV)
    some = lo + torch.minimum((u * (hi - lo)).to(torch.int64), (hi - lo - 1).clamp_(min=0))
    few = torch.where(i < L, i.expand_as(some), torch.full_like(some, -1))
    return torch.where(L > n, some, few).to(torch.int32)


def _e4m3(x):
    """Codes and scales of rows in 32 bits: scale = largest magnitude / 448."""
    s = (x.abs().amax(dim=-1, keepdim=True) / E4M3_MAX).clamp(min=SMALLEST)
    s = torch.where(x.abs().amax(dim=-1, keepdim=True) > 0, s, torch.ones_like(s))
    y = (x / s).clamp(-E4M3_MAX, E4M3_MAX)
    return y.to(torch.float8_e4m3fn), s.squeeze(-1)


def prepare(case, seed):
    c = dict(case)
    g = _generator(seed)
    if c["op"] == "attend":
        return _prepare_attend(c, g)
    dt = DT[c["dtype"]]
    s = dict(case=c, x=torch.randn((c["rows"], c["heads"], c["D"]), generator=g,
                                   device=DEV).to(dt))
    s["positions"] = torch.randint(0, c["ctx"], (c["rows"],), generator=g, device=DEV,
                                   dtype=torch.int32)
    s["freq"] = _frequencies(c).to(DEV)
    if c["op"] == "rope":
        s["out"] = torch.empty_like(s["x"])
    elif c["op"] == "quant":
        s["codes"], s["scales"] = _storage(c, c["rows"])
    else:
        n = c["slots"]
        s["codes"], s["scales"] = _storage(c, n)
        # an occupied cache: random finite codes, scales of ordinary size
        s["codes"].copy_(torch.randint(0, 127, s["codes"].shape, generator=g, device=DEV,
                                       dtype=torch.uint8))
        if c["fmt"] == "fp8":
            s["scales"].copy_(0.005 + 0.01 * torch.rand(s["scales"].shape, generator=g, device=DEV))
        else:
            s["scales"].copy_(torch.randint(118, 130, s["scales"].shape, generator=g, device=DEV,
                                            dtype=torch.uint8))
        # whole pages in a random order; the new tokens are the last of what is read
        page = c["page"]
        pages = _rand_perm(n // page, g)
        all_slots = (pages[:, None] * page + torch.arange(page, device=DEV)[None, :]).reshape(-1)
        used = all_slots[: max(c["read"], c["rows"])].to(torch.int32)
        s["slots"] = used[-c["rows"]:].contiguous()
        s["read_slots"] = used[-c["read"]:].contiguous()
        s["out"] = torch.empty((c["read"], c["heads"], c["D"]), dtype=torch.bfloat16, device=DEV)
    if own:
        import sparse_attention_prefill_tcgen05_gb300 as K
        s["rope"] = K.indexer_rope_create(
            c["D"], c["rot"], rot_offset=c["offset"],
            layout=K.IDX_ROPE_HALF if c["layout"] == "half" else K.IDX_ROPE_INTERLEAVED,
            base=10000.0, factor=c["factor"], original_len=4096, beta_fast=32.0, beta_slow=1.0,
            amplitude=_amplitude(c))
    return s


def _storage(c, n):
    half = c["fmt"] == "fp4"
    codes = torch.empty((n, c["heads"], c["D"] // 2 if half else c["D"]), dtype=torch.uint8,
                        device=DEV)
    scales = torch.empty((n, c["heads"], c["D"] // 32), dtype=torch.uint8, device=DEV) if half \
        else torch.empty((n, c["heads"]), dtype=torch.float32, device=DEV)
    return codes, scales


def _prepare_attend(c, g):
    R, rows, L = c["requests"], c["rows"], c["keys"]
    T, D = R * rows, c["D"]
    dt = DT[c["dtype"]]
    lens = torch.arange(L - rows + 1, L + 1, dtype=torch.int32).repeat(R)
    s = dict(case=c, lens=lens.to(DEV))
    s["q"] = torch.randn((T, c["Hq"], D), generator=g, device=DEV).to(dt)
    if c["page"] > 0:
        per = -(-L // c["page"])
        s["table"] = _rand_perm(R * per, g).to(torch.int32).reshape(R, per)
        slots = R * per * c["page"]
    else:
        s["table"], slots = None, R * L
    s["slots"] = slots
    for name in ("k", "v"):
        x = torch.randn((slots, c["Hkv"], D), generator=g, device=DEV)
        if c["kv"] == "fp8":
            y, sc = _e4m3(x)
            s[name], s[name + "_scale"] = y.view(torch.uint8), sc.contiguous()
        else:
            s[name], s[name + "_scale"] = x.to(dt), None
        del x
    nblk = -(-L // c["block"])
    blocks_of = (s["lens"] + c["block"] - 1) // c["block"]
    sel = _spread(c["sel"], blocks_of, g)
    s["sel"], s["mask"] = sel, None
    if c["mask"]:
        m = torch.zeros((T, nblk + 1), dtype=torch.uint8, device=DEV)
        m.scatter_(1, torch.where(sel < 0, nblk, sel.long()), 1)
        s["mask"] = m[:, :nblk].contiguous()
        s["sel"] = torch.empty((T, c["sel"]), dtype=torch.int32, device=DEV)
    s["out"] = torch.empty((T, c["Hq"], D), dtype=dt, device=DEV)
    s["lse"] = torch.empty((T, c["Hq"]), dtype=torch.float32, device=DEV)
    if own:
        import sparse_attention_prefill_tcgen05_gb300 as K
        cu_q = torch.arange(0, R + 1, dtype=torch.int32) * rows
        cu_k = torch.arange(0, R + 1, dtype=torch.int32) * L
        s["plan"] = K.indexer_plan(cu_q, cu_k, lens, 32, 128, min(2048, c["sel"]))
        s["attn"] = K.indexer_attention_create(
            s["plan"], c["Hq"], c["Hkv"], D, c["sel"], block=c["block"],
            dtype=K.IDX_BF16 if c["dtype"] == "bf16" else K.IDX_FP16,
            kv_format=K.IDX_KV_FP8_E4M3 if c["kv"] == "fp8" else K.IDX_KV_DENSE,
            num_slots=slots, page_size=c["page"])
        s["ws"] = torch.empty(max(256, s["attn"].workspace_bytes), dtype=torch.uint8, device=DEV)
        s["count"] = torch.empty((T,), dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------- the passes


def run(state):
    return _RUN[state["case"]["op"]](state)


def _rotate(x, positions, freq, c):
    """Rotated rows in 32 bits.  The angles are reduced in 64: position 487,935 times a
    32-bit frequency would be off by hundredths of a radian."""
    a = (positions.to(torch.float64)[:, None] * freq[None, :]) % (2 * math.pi)
    a = a.to(torch.float32)[:, None, :]
    m = _amplitude(c)
    cos, sin = torch.cos(a) * m, torch.sin(a) * m
    if c.get("inverse"):
        sin = -sin
    return _turn(x, cos, sin, c)


def _turn(x, cos, sin, c):
    o, r = c["offset"], c["rot"]
    y = x.clone()
    t = x[..., o:o + r]
    if c["layout"] == "half":
        a, b = t[..., : r // 2], t[..., r // 2:]
        y[..., o:o + r] = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    else:
        a, b = t[..., 0::2], t[..., 1::2]
        y[..., o:o + r] = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    return y


def _run_rope(s):
    c = s["case"]
    if own:
        import sparse_attention_prefill_tcgen05_gb300 as K
        K.indexer_rope(s["rope"], s["x"], s["positions"], s["out"], inverse=c["inverse"])
        return s["out"]
    return _rotate(s["x"].float(), s["positions"], s["freq"], c).to(s["x"].dtype)


def _e2m1(x):
    """e2m1 codes and block exponents (biased by 127) of rows in 32 bits, a scale per 32."""
    xb = x.reshape(*x.shape[:-1], -1, 32)
    amax = xb.abs().amax(dim=-1)
    e = (torch.frexp(amax)[1] - 3 + 127).clamp(0, 254)     # floor(log2(amax)) - 2
    e = torch.where(amax > 0, e, torch.full_like(e, 127))
    v = xb * torch.exp2((127 - e).to(x.dtype)).unsqueeze(-1)
    mag = v.abs()
    code = torch.zeros(v.shape, dtype=torch.uint8, device=v.device)
    mids = [(p + q) / 2 for p, q in zip(GRID[:-1], GRID[1:])]
    # a tie goes to the even code: up past the odd midpoints, down at the even ones
    code = (torch.stack([mag >= m if i % 2 else mag > m for i, m in enumerate(mids)])
            .sum(dim=0).to(torch.uint8))
    return code | ((v < 0).to(torch.uint8) << 3), e.to(torch.uint8)


def _e2m1_values(code):
    grid = torch.tensor(GRID + tuple(-x for x in GRID), device=code.device)
    return grid[code.long()]


def _pack(code):
    code = code.reshape(*code.shape[:-2], -1)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _unpack(codes):
    return torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)


def _run_quant(s):
    c = s["case"]
    if own:
        import sparse_attention_prefill_tcgen05_gb300 as K
        fmt = K.IDX_K_FP8_E4M3 if c["fmt"] == "fp8" else K.IDX_K_FP4_E2M1_UE8M0
        K.indexer_cache_write(s["x"], s["codes"], s["scales"], fmt, rope=s["rope"],
                              positions=s["positions"])
        if c["fmt"] == "fp8":
            return s["codes"].view(torch.float8_e4m3fn), s["scales"]
        # 4-bit codes as the values they stand for: the cache's own read, rounded to bf16
        out = torch.empty(s["x"].shape, dtype=torch.bfloat16, device=DEV)
        K.indexer_cache_read(s["codes"], s["scales"], fmt, None, out)
        return out
    x = _rotate(s["x"].float(), s["positions"], s["freq"], c)
    if c["fmt"] == "fp8":
        return _e4m3(x)
    code, e = _e2m1(x)
    s["codes"].copy_(_pack(code))
    s["scales"].copy_(e)
    return _values(s["codes"], s["scales"], "fp4").to(torch.bfloat16)


def _values(codes, scales, fmt):
    if fmt == "fp8":
        return codes.view(torch.float8_e4m3fn).float() * scales[..., None]
    v = _e2m1_values(_unpack(codes))
    return v * torch.exp2(scales.float() - 127).repeat_interleave(32, dim=-1)


def _run_cache(s):
    c = s["case"]
    if own:
        import sparse_attention_prefill_tcgen05_gb300 as K
        fmt = K.IDX_K_FP8_E4M3 if c["fmt"] == "fp8" else K.IDX_K_FP4_E2M1_UE8M0
        K.indexer_cache_write(s["x"], s["codes"], s["scales"], fmt, rope=s["rope"],
                              positions=s["positions"], slots=s["slots"])
        K.indexer_cache_read(s["codes"], s["scales"], fmt, s["read_slots"], s["out"])
        return s["out"]
    x = _rotate(s["x"].float(), s["positions"], s["freq"], c)
    at = s["slots"].long()
    if c["fmt"] == "fp8":
        y, sc = _e4m3(x)
        s["codes"][at] = y.view(torch.uint8)
        s["scales"][at] = sc
    else:
        code, e = _e2m1(x)
        s["codes"][at] = _pack(code)
        s["scales"][at] = e
    src = s["read_slots"].long()
    return _values(s["codes"][src], s["scales"][src], c["fmt"]).to(torch.bfloat16)


def _selected(s):
    """Selected keys of each row, request-local, and their cache slots; -1 where there is none."""
    c = s["case"]
    T = s["q"].shape[0]
    sel = s["sel"]
    if c["mask"]:
        # the kept blocks of each mask row in ascending order, then -1
        n = s["mask"].shape[1]
        at = torch.arange(n, device=DEV, dtype=torch.int32)[None, :]
        sel = torch.where(s["mask"] != 0, at, n).sort(dim=1)[0][:, : c["sel"]]
        sel = torch.where(sel < n, sel, -1)
        if sel.shape[1] < c["sel"]:
            sel = torch.cat([sel, sel.new_full((T, c["sel"] - sel.shape[1]), -1)], dim=1)
    j = sel.long()[:, :, None] * c["block"] + torch.arange(c["block"], device=DEV)
    ok = (sel[:, :, None] >= 0) & (j < s["lens"].long()[:, None, None])
    j, ok = j.flatten(1), ok.flatten(1)
    j = torch.where(ok, j, torch.zeros_like(j))
    r = torch.arange(T, device=DEV) // c["rows"]
    if s["table"] is not None:
        slot = s["table"][r[:, None], j // c["page"]].long() * c["page"] + j % c["page"]
    else:
        slot = r[:, None] * c["keys"] + j
    return sel, slot, ok


def _run_attend(s):
    c = s["case"]
    if own:
        import sparse_attention_prefill_tcgen05_gb300 as K
        count = None
        if c["mask"]:
            K.indexer_mask_blocks(s["plan"], s["mask"], s["lens"], c["block"], s["sel"], s["count"])
            count = s["count"]
        K.indexer_sparse_attention(s["attn"], s["q"], s["k"], s["v"], s["sel"], s["lens"],
                                   s["out"], s["ws"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                   sel_count=count, page_table=s["table"], lse=s["lse"])
        return (s["out"], s["lse"]) + ((s["sel"],) if c["mask"] else ())
    sel, slot, ok = _selected(s)
    T, G = s["q"].shape[0], c["Hq"] // c["Hkv"]
    k, v = s["k"][slot], s["v"][slot]                       # [T, S, Hkv, D]
    if c["kv"] == "fp8":
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    k, v = k.float().transpose(1, 2), v.float().transpose(1, 2)
    if c["kv"] == "fp8":
        k = k * s["k_scale"][slot].transpose(1, 2)[..., None]
        v = v * s["v_scale"][slot].transpose(1, 2)[..., None]
    q = s["q"].float().reshape(T, c["Hkv"], G, c["D"])
    a = torch.matmul(q, k.transpose(2, 3)) * c["D"] ** -0.5
    a = a.masked_fill(~ok[:, None, None, :], -math.inf)
    m = a.amax(dim=-1, keepdim=True)
    p = torch.exp(a - m.clamp(min=-3.0e38))
    z = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, v) / z.clamp(min=1e-30)
    lse = (m + torch.log(z)).reshape(T, c["Hq"])
    o = o.reshape(T, c["Hq"], c["D"]).to(s["q"].dtype)
    return (o, lse) + ((sel.to(torch.int32),) if c["mask"] else ())


_RUN = {"rope": _run_rope, "quant": _run_quant, "cache": _run_cache, "attend": _run_attend}


# ------------------------------------------------------------------------- what it takes


def work(case):
    c = case
    n = c["rows"] * c.get("heads", 1) * c["D"]
    if c["op"] == "attend":
        T = c["requests"] * c["rows"]
        eb, sb = (1, 4) if c["kv"] == "fp8" else (2, 0)
        lens = range(c["keys"] - c["rows"] + 1, c["keys"] + 1)
        picked = c["requests"] * sum(min(c["sel"] * c["block"], x) for x in lens)
        distinct = min(c["requests"] * c["keys"], picked)
        per_row = 4 * c["sel"] if not c["mask"] else 4 * c["sel"] + -(-c["keys"] // c["block"])
        return {"bytes": 4 * T * c["Hq"] * c["D"] + 4 * T * c["Hq"] + T * (per_row + 4)
                + distinct * c["Hkv"] * 2 * (c["D"] * eb + sb),
                "flops": 4.0 * picked * c["Hq"] * c["D"]}
    eb = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "rope":
        return {"bytes": 2 * n * eb + 4 * c["rows"], "flops": 6.0 * n * c["rot"] / c["D"] / 2}
    per = (1.0 + 4.0 / c["D"]) if c["fmt"] == "fp8" else (0.5 + 1.0 / 32)      # of an element
    w = n * eb + n * per + 4 * c["rows"]
    r = 0.0
    if c["op"] == "cache":
        r = c["read"] * (c["heads"] * c["D"] * (per + 2) + 4) + 4 * c["rows"]
    elif c["fmt"] == "fp4":
        r = n * (per + 2)
    return {"bytes": w + r, "flops": 8.0 * n}


# ------------------------------------------------------------------------------- 64 bits


def _exact_rotated(c, x, positions):
    a = positions.double()[:, None] * _frequencies(c).to(DEV)[None, :]
    a = a[:, None, :]
    m = _amplitude(c)
    sign = -1.0 if c.get("inverse") else 1.0
    co, si = m * torch.cos(a), sign * m * torch.sin(a)
    y = x.double().clone()
    half = c["rot"] // 2
    for i in range(half):
        p, q = (i, i + half) if c["layout"] == "half" else (2 * i, 2 * i + 1)
        p, q = p + c["offset"], q + c["offset"]
        u, v = x[..., p].double(), x[..., q].double()
        y[..., p] = u * co[..., i] - v * si[..., i]
        y[..., q] = u * si[..., i] + v * co[..., i]
    return y


def _exact_e4m3(x):
    """The e4m3 values nearest to x / scale, in 64 bits: a step of 2^(e - 3) at 2^e <= |y|,
    2^-9 below 2^-6, ties to the even multiple."""
    amax = x.abs().amax(dim=-1, keepdim=True)
    s = torch.where(amax > 0, (amax / E4M3_MAX).clamp(min=SMALLEST), torch.ones_like(amax))
    y = x / s
    step = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=-6).double() - 3)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX), s.squeeze(-1)


def _exact_e2m1(x):
    """The e2m1 values nearest to x / scale times the scale, in 64 bits."""
    xb = x.reshape(*x.shape[:-1], -1, 32)
    amax = xb.abs().amax(dim=-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)
    s = torch.where(amax > 0, torch.exp2(e.double()), torch.ones_like(amax))
    y = xb / s
    step = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=0).double() - 1)
    return ((torch.round(y / step) * step).clamp(-6, 6) * s).reshape(x.shape)


def exact(case, seed):
    c = dict(case)
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    if c["op"] == "attend":
        return _exact_attend(c, s)
    y = _exact_rotated(c, s["x"], s["positions"])
    if c["op"] == "rope":
        return y
    if c["op"] == "quant":
        return _exact_e4m3(y) if c["fmt"] == "fp8" else _exact_e2m1(y)
    n = c["slots"]
    if c["fmt"] == "fp8":
        v, sc = _exact_e4m3(y)
        new = v * sc[..., None]
        old = s["codes"].view(torch.float8_e4m3fn).double() * s["scales"].double()[..., None]
    else:
        new = _exact_e2m1(y)
        old = _e2m1_values(_unpack(s["codes"])).double() * torch.exp2(
            s["scales"].double() - 127).repeat_interleave(32, dim=-1)
    old[s["slots"].long()] = new
    assert old.shape[0] == n
    return old[s["read_slots"].long()]


def _exact_attend(c, s):
    sel, slot, ok = _selected(s)
    T, G, D = s["q"].shape[0], c["Hq"] // c["Hkv"], c["D"]
    out = torch.empty((T, c["Hq"], D), dtype=torch.float64, device=DEV)
    lse = torch.empty((T, c["Hq"]), dtype=torch.float64, device=DEV)
    step = max(1, 200_000_000 // (slot.shape[1] * c["Hkv"] * D))
    for t in range(0, T, step):
        at, good = slot[t:t + step], ok[t:t + step]
        kk, vv = s["k"][at], s["v"][at]
        if c["kv"] == "fp8":
            kk = kk.view(torch.float8_e4m3fn).double() * s["k_scale"][at].double()[..., None]
            vv = vv.view(torch.float8_e4m3fn).double() * s["v_scale"][at].double()[..., None]
        kk, vv = kk.double(), vv.double()
        for h in range(c["Hkv"]):
            q = s["q"][t:t + step, h * G:(h + 1) * G].double()
            a = torch.bmm(q, kk[:, :, h].transpose(1, 2)) / math.sqrt(D)
            a.masked_fill_(~good[:, None, :], -math.inf)
            lse[t:t + step, h * G:(h + 1) * G] = torch.logsumexp(a, dim=-1)
            out[t:t + step, h * G:(h + 1) * G] = torch.bmm(torch.softmax(a, dim=-1), vv[:, :, h])
    return (out, lse) + ((None,) if c["mask"] else ())
