"""Causal attention in tiles of rows (indexer_causal_attention), whose form is chosen at creation by
estimated times: batches for which it is chosen, asserted, so that its masks, rescaling, cuts and joins
run.  Formulas and tolerances are those of test_causal_attention.
"""
import math

import numpy as np
import pytest
import torch

from sparse_attention_prefill_tcgen05_gb300 import _lib as K
from tests.test_causal_attention import Batch, seen_by

KINDS = [("bf16", "same"), ("fp16", "same"), ("bf16", "fp8"), ("fp16", "fp8")]

# name: requests, Hq, Hkv, window, sinks, page, and what the batch is shared out to:
# "whole" items, parts that a warp ("few") or four ("many") join, None: any
SHAPES = {
    "whole": ([(300, 300)], 2, 2, 0, 0, 16, "whole"),
    "packed": ([(600, 600)], 4, 1, 0, 0, 0, None),
    "many parts": ([(260, 3000)], 8, 1, 0, 0, 48, "many"),
    "few parts": ([(900, 1500), (301, 700), (64, 64)], 16, 4, 0, 0, 64, "few"),
    "long window": ([(800, 3000)], 8, 2, 300, 5, 1, "whole"),
    "window": ([(500, 900)], 4, 2, 60, 3, 16, "whole"),
    "sinks": ([(600, 900), (5, 5)], 8, 2, 33, 130, 100, None),
    "pages": ([(500, 700), (300, 300)], 4, 2, 0, 0, 16, None),
    "pages, window": ([(500, 700), (300, 300)], 4, 2, 90, 20, 16, None),
    "unseen": ([(300, 900), (260, 400)], 4, 2, 100, 5, 48, None),
    "gaps": ([(600, 1000)], 4, 2, 60, 4, 16, None),
    "any lengths": ([(300, 400), (0, 10), (60, 0), (290, 1000)], 4, 2, 0, 0, 16, None),
    "any lengths, window": ([(300, 400), (0, 10), (60, 0), (290, 1000)], 4, 2, 50, 7, 16, None),
    "strides": ([(300, 300)], 4, 2, 40, 2, 16, "whole"),
    "far": ([(400, 400)], 8, 2, 0, 0, 40, None),
    "five heads": ([(300, 900)], 15, 3, 0, 0, 3, "many"),
    "wide group": ([(300, 700)], 160, 1, 0, 0, 64, "few"),
    "wide group, window": ([(200, 700)], 320, 2, 64, 9, 7, "whole"),
}


def batch(name, D=64, dt="bf16", kv="same", **kw):
    requests, Hq, Hkv, window, sinks, page, _ = SHAPES[name]
    return Batch(requests, Hq, Hkv, D, window, sinks, dt, kv, page, **kw)


def run(b, **kw):
    r = b.run(**kw)
    assert b.attn.info()["tiles"] == 1
    return r


def some_rows(b, n=60, seed=0):
    """Row numbers to check: the ends of every request and some between."""
    ends = [t for c in b.cu_q for t in (c - 1, c, c + 1) if 0 <= t < b.T]
    return sorted({*ends, *np.random.default_rng(seed).integers(0, b.T, n)})


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt,kv", KINDS)
def test_form(D, dt, kv):
    """Which of them are cut, and how the parts are joined (four warps a row where a cut item has
    more than four blocks on average)."""
    for name, (requests, Hq, Hkv, window, sinks, page, cut) in SHAPES.items():
        rows, keys = [r for r, _ in requests], [n for _, n in requests]
        plan = K.indexer_plan(np.cumsum([0] + rows), np.cumsum([0] + keys), [0] * sum(rows), 32, 128, 8)
        info = K.indexer_causal_attention_create(
            plan, Hq, Hkv, D, window, sinks, K.IDX_BF16 if dt == "bf16" else K.IDX_FP16,
            K.IDX_KV_FP8_E4M3 if kv == "fp8" else K.IDX_KV_DENSE, 4096, page).info()
        assert info["tiles"] == 1, name
        if cut:
            joined = info["joined"]
            got = "whole" if joined == 0 else "many" if info["blocks"] > 4 * joined else "few"
            assert got == cut, (name, info)
        if name in ("many parts", "few parts"):
            assert info["blocks"] == 152, name


def test_rows_one_by_one_have_no_blocks():
    plan = K.indexer_plan([0, 1], [0, 4000], [4000], 32, 128, 8)
    attn = K.indexer_causal_attention_create(plan, 8, 2, 64)
    assert attn.info() == dict(tiles=0, blocks=0, joined=0)
    assert K.lib().indexer_causal_attention_info(None, None, None, None) == K.IDX_ERR_INVALID_ARG
    assert K.lib().indexer_causal_attention_info(attn.handle, None, None, None) == K.IDX_OK


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("name", ["whole", "packed", "many parts", "few parts", "long window", "sinks"])
def test_formulas(name, dt, kv, D):
    b = batch(name, D, dt, kv, seed=21)
    b.check(*run(b), rows=some_rows(b))


@pytest.mark.gpu
@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("name", ["five heads", "wide group", "wide group, window"])
def test_groups(name, dt, kv):
    """Groups that do not divide a row tile, or fill more than one: queries without a tensor map."""
    b = batch(name, 128, dt, kv, seed=22)
    b.check(*run(b), rows=some_rows(b, 12))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
@pytest.mark.parametrize("name", ["any lengths", "any lengths, window"])
def test_lengths_in_any_order(name, kv):
    rng = np.random.default_rng(23)
    lens = np.concatenate([rng.integers(0, n + 50, r) * (rng.random(r) < 0.7) for r, n in SHAPES[name][0]])
    lens[3], lens[7] = -5, 2 ** 31 - 1
    b = batch(name, kv=kv, lens=lens, seed=23)
    b.check(*run(b))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt,kv", KINDS)
def test_scores_that_grow(dt, kv, D):
    """Each half tile's largest score is far above the one before in most rows, so that the outputs so
    far are rescaled every time; others fall, or stay."""
    b = batch("whole", D, dt, kv, seed=24)
    j = torch.from_numpy(np.concatenate([b.slot_of(0, np.array([x])) for x in range(300)]))
    k = torch.empty(b.slots, 2, D)
    k[:] = 0.05 * torch.randn(k.shape, generator=torch.Generator().manual_seed(24))
    k[j] += 12 * torch.linspace(0, 1, 300)[:, None, None]
    if kv == "fp8":
        b.ks[:] = 2.0
        b.k = (k / 2).to(torch.float8_e4m3fn).view(torch.uint8)
        kk = b.k.view(torch.float8_e4m3fn).float() * 2
    else:
        b.k = k.to(b.dt)
        kk = b.k.float()
    slope = torch.tensor([1.0, 2.0, -1.5, 0.001])[torch.arange(300) % 4]
    b.q = (b.q.float() * 0.01 + slope[:, None, None]).to(b.dt)
    # (a new reference for scores 15 above the one before, in powers of two)
    a = b.scale / math.log(2) * torch.einsum("thd,jhd->thj", b.q.float(), kk[j])
    top = a[:, :, :256].reshape(300, 2, 4, 64).amax(-1)
    assert torch.all((top[1::4, :, 1:] - top[1::4, :, :-1])[:, :, :1] > 15 + 7)
    assert torch.all((top[::4, :, 1:] - top[::4, :, :-1]) > 15 + 7)
    b.check(*run(b))


@pytest.mark.gpu
@pytest.mark.parametrize("dt,kv", KINDS)
def test_large_scores(dt, kv):
    b = batch("whole", 128, dt, kv, spread=16.0, seed=25)
    b.check(*run(b))
    b = batch("many parts", 128, dt, kv, spread=16.0, seed=25)
    b.check(*run(b), rows=some_rows(b, 30))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
@pytest.mark.parametrize("scale", [0.0, 1.0, 2.0 ** -140])
def test_scales(scale, kv):
    b = batch("window", kv=kv, scale=scale, seed=26)
    b.check(*run(b), rows=some_rows(b))


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -90])
def test_smallest_scales(scale):
    """Keys of the smallest scale under a small factor, masked and not: their product is none, and none
    times a masked score would not be a number."""
    b = batch("window", kv="fp8", scale=scale, seed=27)
    b.ks[::3] = 2.0 ** -126
    assert np.float32(2.0 ** -126) * np.float32(scale) == 0
    b.check(*run(b), rows=some_rows(b))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
@pytest.mark.parametrize("name", ["pages", "pages, window"])
def test_unmapped_pages(name, kv):
    b = batch(name, kv=kv, seed=28)
    b.table[0, ::3] = -1
    b.table[0, 4] = 2 ** 31 - 1
    b.table[1] = -7
    b.table[1, 1 if name == "pages" else 18] = b.slots // 16      # the first page past the cache
    b.check(*run(b))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
def test_what_no_row_sees_has_no_effect(kv):
    b = batch("unseen", kv=kv, seed=29)
    b.lens = b.lens.copy()
    b.lens[:300] -= 30
    want = run(b)
    b.check(*want, rows=some_rows(b))
    used = np.zeros(b.slots, bool)
    for t in range(b.T):
        used[b.slot_of(t, seen_by(int(b.lens[t]), b.window, b.sinks))] = True
    bad = torch.from_numpy(~used)
    assert bad.any()
    if kv == "fp8":
        b.k[bad], b.v[bad] = 0x7F, 0xFF
        b.ks[bad], b.vs[bad] = math.nan, math.inf
    else:
        b.k[bad], b.v[bad] = math.nan, math.inf
    got = run(b)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
def test_gaps_between_windows(kv):
    b = batch("gaps", 128, kv=kv, lens=[100] * 300 + [950] * 300, seed=30)
    want = run(b)
    b.check(*want, rows=some_rows(b))
    gap = torch.from_numpy(b.slot_of(0, np.arange(100, 890))).cuda()

    def edit(k, v):
        k[gap], v[gap] = (0x7F, 0x7F) if kv == "fp8" else (math.nan, math.inf)
        return k, v
    if kv == "fp8":
        b.ks[gap.cpu()], b.vs[gap.cpu()] = math.inf, math.nan
    got = run(b, edit=edit)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_strides(D):
    """q, k, v and out as parts of wider tensors, queries by map and heads of one address; the rest of
    out stays."""
    b = batch("strides", D, seed=31)
    want, _ = run(b)
    q = torch.zeros(300, 6, D + 16, dtype=b.dt)
    q[:, 1:5, 8:8 + D] = b.q
    kv = torch.zeros(b.slots, 2, 2, D + 8, dtype=b.dt)
    kv[:, 0, :, :D], kv[:, 1, :, :D] = b.k, b.v
    q, kv, lens, table = q.cuda(), kv.cuda(), torch.from_numpy(b.lens).cuda(), b.table.cuda()
    ws = torch.empty(b.attn.workspace_bytes, dtype=torch.uint8, device="cuda")

    def call(q, out):
        K.indexer_causal_attention(b.attn, q, kv[:, 0, :, :D], kv[:, 1, :, :D], lens, out, ws, page_table=table)
    for pad in (16, 3):                                           # 32-byte stores, or not
        out = torch.full((300, 5, D + pad), 7.0, dtype=b.dt, device="cuda")
        call(q[:, 1:5, 8:8 + D], out[:, :4, :D])
        assert torch.equal(out[:, :4, :D], want)
        assert torch.all(out[:, 4] == 7) and torch.all(out[:, :, D:] == 7)
    b.q[:] = b.q[:, :1].clone()
    want, _ = run(b)
    out = torch.empty(300, 4, D, dtype=b.dt, device="cuda")
    call(q[:, 1:2, 8:8 + D].expand(-1, 4, -1), out)
    assert torch.equal(out, want)
    b.check(want, None, rows=some_rows(b))


@pytest.mark.gpu
def test_far_slots():
    """A cache whose last keys are past 2^32 bytes from its start."""
    n, D = 9_000_000, 128
    b = batch("far", D, seed=32)
    pages = torch.tensor([n // 40 - 1, 0, n // 40 - 7, 215_000, 210_000, 224_990, 1, 7, 150_000, 9], dtype=torch.int32)
    at = (b.table[0].long()[:, None] * 40 + torch.arange(40)).reshape(-1)
    to = (pages.long()[:, None] * 40 + torch.arange(40)).reshape(-1)
    want = run(b)
    b.check(*want, rows=some_rows(b))
    k = torch.zeros(n, 2, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[to.cuda()], v[to.cuda()] = b.k[at].cuda(), b.v[at].cuda()
    b.table, b.slots = pages[None], n
    got = run(b, edit=lambda *_: (k, v))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["many parts", "few parts"])
def test_two_streams_and_a_replay(name):
    """Cut items beside whole ones on two streams; a captured call replayed with other lengths, longer
    and shorter than those its cuts were planned by."""
    b, c = batch(name, 128, seed=33), batch("whole", seed=34)
    want_b, want_c = run(b), run(c)
    args = []
    for x in (b, c):
        args.append([x.attn, x.q.cuda(), x.k.cuda(), x.v.cuda(), torch.from_numpy(x.lens).cuda(),
                     torch.empty(x.T, x.Hq, x.D, dtype=x.dt, device="cuda"),
                     torch.empty(x.attn.workspace_bytes, dtype=torch.uint8, device="cuda")])
    tables = [b.table.cuda(), c.table.cuda()]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for st, a, t in zip(s, args, tables):
            K.indexer_causal_attention(*a, page_table=t, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(args[0][5], want_b[0]) and torch.equal(args[1][5], want_c[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for a, t in zip(args, tables):
            K.indexer_causal_attention(*a, page_table=t)
    rng = np.random.default_rng(33)
    for lens in (np.zeros_like(b.lens), np.minimum(b.lens, 100), b.L, rng.integers(0, b.L + 1)):
        b.lens = lens.astype(np.int32)
        args[0][4].copy_(torch.from_numpy(b.lens))
        for a in args:
            a[5].fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        b.check(args[0][5], None, rows=some_rows(b, 20))
        assert torch.equal(args[1][5], want_c[0])
