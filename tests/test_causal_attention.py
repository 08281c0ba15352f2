"""Causal attention over cached keys (indexer_causal_attention), against the formulas in 64 bits.

Tolerance, from the operations, per row, head and element.  A score is a sum of D products in fp32, off by
D 2^-24 sum |q_i k_i| at most, then scaled and taken from the reference with roundings of 2^-22 of its
size; so a weight is off by a relative 2 da + 2^-20 with da the largest of both.  Weights enter
the product with v rounded: by 2^-8 of their size (bf16), 2^-11 (fp16; and 2^-32 of the row's largest),
2^-16 (two bf16 terms).  The output is rounded once.
"""
import math

import numpy as np
import pytest
import torch

from sparse_attention_prefill_tcgen05_gb300 import _lib as K

DT = {"bf16": (torch.bfloat16, K.IDX_BF16), "fp16": (torch.float16, K.IDX_FP16)}


def seen_by(n, window, sinks):
    """Key positions a row of length n sees."""
    if window <= 0 or n <= window:
        return np.arange(n)
    return np.concatenate([np.arange(min(sinks, n - window)), np.arange(n - window, n)])


class Batch:
    """A ragged batch, requests of (rows, keys); the last row of a request sees every key."""

    def __init__(self, requests, Hq, Hkv, D, window=0, sinks=0, dt="bf16", kv="same", page=0, seed=0, spread=1.0,
                 lens=None, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.dt, self.code = DT[dt]
        self.kv, self.page, self.window, self.sinks = kv, page, window, sinks
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.scale = D ** -0.5 if scale is None else scale
        rows, keys = [r for r, _ in requests], [n for _, n in requests]
        self.cu_q = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.cu_k = np.concatenate([[0], np.cumsum(keys)]).astype(np.int32)
        self.T, self.req = int(self.cu_q[-1]), np.repeat(np.arange(len(rows)), rows)
        self.L = np.array([keys[r] for r in self.req], dtype=np.int64)
        if lens is None:
            lens = np.concatenate([np.clip(n - r + 1 + np.arange(r), 0, n) for r, n in requests])
        self.lens = np.asarray(lens).astype(np.int32)
        self.plan = K.indexer_plan(self.cu_q, self.cu_k, np.clip(self.lens, 0, self.L).astype(np.int32), 32, 128, 8)
        if page:
            per = -(-max(keys) // page)
            self.table = torch.randperm(len(rows) * per, generator=g).int().reshape(len(rows), per)
            self.slots = len(rows) * per * page
        else:
            self.table, self.slots = None, int(self.cu_k[-1])
        self.q = (torch.randn(self.T, Hq, D, generator=g) * spread).to(self.dt)
        kf, vf = (torch.randn(self.slots, Hkv, D, generator=g) for _ in range(2))
        self.ks = self.vs = None
        if kv == "fp8":
            # each vector has its own scale, far apart
            self.ks, self.vs = (torch.exp2(torch.randint(-a, a, (self.slots, Hkv), generator=g).float()) / 100
                                for a in (2, 6))
            self.k, self.v = ((x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x in (kf, vf))
        else:
            self.k, self.v = kf.to(self.dt), vf.to(self.dt)

    def slot_of(self, t, j):
        r = self.req[t]
        if not self.page:
            return self.cu_k[r] + j
        page = self.table[r].numpy()[j // self.page].astype(np.int64)
        at = page * self.page + j % self.page
        return np.where((page >= 0) & (at < self.slots), at, -1)

    def run(self, lse=True, edit=None, ws=None, page_table="own", out=None):
        self.attn = K.indexer_causal_attention_create(
            self.plan, self.Hq, self.Hkv, self.D, self.window, self.sinks, self.code,
            K.IDX_KV_FP8_E4M3 if self.kv == "fp8" else K.IDX_KV_DENSE, self.slots, self.page, self.scale)
        c = lambda t: None if t is None else t.cuda()
        if ws is None:
            ws = torch.full((self.attn.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
        if out is None:
            out = torch.full((self.T, self.Hq, self.D), math.nan, dtype=self.dt, device="cuda")
        z = torch.full((self.T, self.Hq), math.nan, device="cuda") if lse else None
        k, v = c(self.k), c(self.v)
        if edit:
            k, v = edit(k, v)
        K.indexer_causal_attention(self.attn, c(self.q), k, v, torch.from_numpy(self.lens).cuda(), out, ws,
                                   c(self.ks), c(self.vs), c(self.table), z)
        assert K.indexer_status(None, ws) == K.IDX_OK
        return out, z

    def check(self, got, lse, rows=None):
        Hkv, G = self.Hkv, self.Hq // self.Hkv
        val = lambda x, s: x.double().numpy() if s is None else \
            x.view(torch.float8_e4m3fn).double().numpy() * s.double().numpy()[..., None]
        k, v, q = val(self.k, self.ks), val(self.v, self.vs), self.q.double().numpy()
        got = got.double().cpu().numpy()
        z = None if lse is None else lse.double().cpu().numpy()
        up = 2.0 ** -8 if self.dt == torch.bfloat16 else 2.0 ** -16 if self.kv == "fp8" else 2.0 ** -11
        uo = torch.finfo(self.dt).eps / 2
        for t in range(self.T) if rows is None else rows:
            at = self.slot_of(t, seen_by(max(0, min(int(self.lens[t]), self.L[t])), self.window, self.sinks))
            at = at[at >= 0]
            if len(at) == 0:
                assert np.all(got[t] == 0), t
                assert z is None or np.all(np.isneginf(z[t])), t
                continue
            for g in range(Hkv):
                h = slice(g * G, (g + 1) * G)
                kk, vv, qq = k[at, g], v[at, g], q[t, h]
                a = self.scale * (qq @ kk.T)
                mx = a.max(axis=1, keepdims=True)
                e = np.exp(a - mx)
                s = e.sum(axis=1, keepdims=True)
                p = e / s
                out = p @ vv
                da = (abs(self.scale) * self.D * 2.0 ** -24 * (np.abs(qq) @ np.abs(kk).T)
                      + 2.0 ** -22 * np.abs(a)).max(axis=1, keepdims=True)
                tol = (up + 2 * da + 2.0 ** -20) * (p @ np.abs(vv)) + uo * np.abs(out) \
                    + 2.0 ** -32 * len(at) * p.max(axis=1, keepdims=True) * np.abs(vv).max() + 2.0 ** -25
                err = np.abs(got[t, h] - out)
                assert np.all(err <= tol), (t, g, float(np.max(err - tol)), float(err.max()))
                if z is not None:
                    want = (mx + np.log(s))[:, 0]
                    assert np.all(np.abs(z[t, h] - want) <= da[:, 0] + 2.0 ** -20 * (1 + np.abs(want))), (t, g)


CASES = [
    # requests, Hq, Hkv, D, window, sinks, dtype, cache, page
    ([(1, 1)], 1, 1, 64, 0, 0, "bf16", "same", 0),
    ([(16, 77)], 4, 1, 64, 0, 0, "fp16", "same", 0),
    ([(128, 128)], 1, 1, 128, 0, 0, "bf16", "same", 0),
    ([(300, 300)], 2, 2, 128, 0, 0, "bf16", "same", 16),
    ([(1, 200), (3, 129), (70, 70)], 8, 1, 128, 0, 0, "bf16", "same", 48),
    ([(5, 700), (0, 30), (100, 411)], 15, 3, 64, 0, 0, "fp16", "same", 1),
    ([(257, 1000)], 4, 1, 64, 100, 4, "bf16", "same", 64),
    ([(140, 900)], 6, 2, 128, 128, 0, "fp16", "same", 3),
    ([(140, 900), (1, 1), (2, 2)], 16, 2, 128, 33, 130, "bf16", "same", 100),
    ([(64, 512)], 3, 1, 64, 1, 1, "bf16", "same", 16),
    ([(40, 300)], 160, 1, 64, 0, 0, "bf16", "same", 64),         # a group wider than a tile
    ([(9, 600)], 320, 2, 128, 64, 9, "fp16", "same", 7),
    ([(200, 333)], 4, 2, 64, 0, 0, "bf16", "fp8", 16),
    ([(200, 333)], 4, 2, 128, 0, 0, "fp16", "fp8", 48),
    ([(1, 1500), (33, 640)], 8, 1, 128, 200, 4, "bf16", "fp8", 1),
    ([(90, 90), (7, 1000)], 5, 1, 64, 0, 0, "fp16", "fp8", 0),
    ([(600, 2000)], 8, 1, 64, 256, 2, "bf16", "fp8", 64),
    ([(2, 9000)], 8, 2, 128, 0, 0, "bf16", "same", 64),          # split over blocks
    ([(1, 20000)], 4, 4, 64, 0, 0, "fp16", "same", 16),
    ([(3, 5000), (1, 100)], 32, 4, 128, 0, 0, "fp16", "fp8", 64),
    ([(1, 4000)] * 9, 16, 8, 128, 700, 4, "bf16", "fp8", 16),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
def test_formulas(case):
    *args, dt, kv, page = CASES[case]
    b = Batch(*args, dt, kv, page, seed=case)
    rows = None if b.T * b.Hq < 3000 else sorted({0, 1, b.T - 1, b.T // 2, *np.random.default_rng(case).integers(0, b.T, 60)})
    b.check(*b.run(), rows=rows)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 0), (50, 7), (500, 200)])
def test_lengths_in_any_order(window, sinks, kv):
    """Padding rows of length 0 among others, lengths past the request's keys, negative ones."""
    rng = np.random.default_rng(window)
    requests = [(150, 400), (0, 10), (60, 0), (90, 1000)]
    lens = np.concatenate([rng.integers(0, n + 50, r) * (rng.random(r) < 0.7) for r, n in requests])
    lens[3], lens[7] = -5, 2 ** 31 - 1
    b = Batch(requests, 4, 2, 64, window, sinks, kv=kv, page=16, lens=lens, seed=1)
    b.check(*b.run())


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 2 ** 31 - 1), (300, 2 ** 31 - 1), (2, 0), (900, 5), (901, 5)])
@pytest.mark.parametrize("requests", [[(70, 20), (200, 900)], [(1, 900), (1, 5)]])
def test_windows_at_their_limits(window, sinks, requests):
    """Windows and sinks longer than any request, requests with fewer keys than rows."""
    b = Batch(requests, 4, 2, 64, window, sinks, page=16, seed=14)
    b.check(*b.run())


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_large_scores(dt, kv):
    """Weights of one key a row, references that move from tile to tile."""
    b = Batch([(40, 900)], 8, 2, 128, dt=dt, kv=kv, spread=16.0, seed=3)
    b.check(*b.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_scores_that_grow(dt):
    """Every tile's maximum above the one before, and one row whose scores fall."""
    b = Batch([(3, 1300)], 4, 1, 64, dt=dt, seed=4)
    ramp = torch.linspace(0, 1, 1300)[:, None, None]
    b.k = (b.k.float() * 0.05 + ramp * 6).to(b.dt)
    b.q = (b.q.float() * 0.05 + torch.tensor([1.0, 2.0, -1.5])[:, None, None]).to(b.dt)
    b.check(*b.run())


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0, -1e-30])
@pytest.mark.parametrize("kv", ["same", "fp8"])
def test_scales(scale, kv):
    b = Batch([(50, 300)], 4, 2, 64, 60, 3, kv=kv, scale=scale, seed=5)
    b.check(*b.run())


@pytest.mark.gpu
def test_smallest_scales():
    """Keys of the smallest scale under a small factor, masked and not."""
    b = Batch([(70, 300)], 4, 2, 64, 60, 3, kv="fp8", scale=2.0 ** -90, seed=15)
    b.ks[::3] = 2.0 ** -126
    b.check(*b.run())


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
@pytest.mark.parametrize("window", [0, 90])
def test_unmapped_pages(kv, window):
    """Negative entries and slots past the cache are left out, in any place of the list."""
    b = Batch([(70, 500), (1, 300)], 4, 2, 64, window, 20, kv=kv, page=16, seed=6)
    b.table[0, ::3] = -1
    b.table[0, 4] = 2 ** 31 - 1
    b.table[1] = -7
    b.table[1, 1 if window == 0 else 18] = b.slots // 16          # the first page past the cache
    b.check(*b.run())


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
def test_what_no_row_sees_has_no_effect(kv):
    """NaN and infinities in keys, values and scales that no row sees, in pages that are partly seen."""
    b = Batch([(20, 700), (33, 200)], 4, 2, 64, 100, 5, kv=kv, page=48, seed=7)
    lens = b.lens.copy()
    lens[:20] -= 30
    b.lens = lens
    want = b.run()
    used = np.zeros(b.slots, bool)
    for t in range(b.T):
        used[b.slot_of(t, seen_by(int(b.lens[t]), b.window, b.sinks))] = True
    bad = torch.from_numpy(~used)
    if kv == "fp8":
        b.k[bad], b.v[bad] = 0x7F, 0xFF
        b.ks[bad], b.vs[bad] = math.nan, math.inf
    else:
        b.k[bad], b.v[bad] = math.nan, math.inf
    got = b.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
@pytest.mark.parametrize("rows,window", [(300, 0), (300, 70), (2, 0)])
def test_what_some_rows_do_not_see(kv, rows, window):
    """Values (16-bit) and keys that are not finite change nothing in rows that do not see them, and
    give none that see them a number where the formula has none."""
    b = Batch([(rows, 500), (40, 90)], 4, 2, 64, window, 3, kv=kv, page=16, seed=12)
    want = b.run()
    first = 500 - rows // 2                                       # keys of the second half's rows
    at = torch.from_numpy(b.slot_of(0, np.arange(first, 500)))
    bad = at[::3]
    sees = np.array([r == 0 and n > first for r, n in zip(b.req, b.lens)])

    def edit(k, v):
        if kv == "fp8":
            k[bad[::2].cuda()] = 0x7F
            v[bad[1::2].cuda()] = 0xFF
        else:
            k[bad[::2].cuda(), :, 5] = math.nan
            v[bad[1::2].cuda(), :, 7] = math.inf
            v[bad[1::4].cuda(), :, 9] = math.nan
        return k, v
    got = b.run(edit=edit)
    assert torch.equal(got[0][~sees], want[0][~sees]) and torch.equal(got[1][~sees], want[1][~sees])
    last = [t for t in range(b.T) if sees[t]][-1]
    assert torch.isnan(got[0][last]).any(-1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
def test_gaps_between_windows(kv):
    """Keys between two rows' windows that neither sees."""
    lens = [100] * 20 + [950] * 20
    b = Batch([(40, 1000)], 4, 2, 128, 60, 4, kv=kv, page=16, lens=lens, seed=13)
    want = b.run()
    gap = torch.from_numpy(b.slot_of(0, np.arange(100, 890))).cuda()

    def edit(k, v):
        k[gap], v[gap] = (0x7F, 0x7F) if kv == "fp8" else (math.nan, math.inf)
        return k, v
    if kv == "fp8":
        b.ks[gap.cpu()], b.vs[gap.cpu()] = math.inf, math.nan
    got = b.run(edit=edit)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_strides():
    """q, k, v and out as parts of wider tensors; no log-sum-exp asked for; the rest stays."""
    b = Batch([(50, 300)], 4, 2, 64, 40, 2, page=16, seed=8)
    want, _ = b.run()
    q = torch.zeros(50, 6, 80, dtype=b.dt)
    q[:, 1:5, 8:72] = b.q
    kv = torch.zeros(b.slots, 2, 2, 72, dtype=b.dt)
    kv[:, 0, :, :64], kv[:, 1, :, :64] = b.k, b.v
    kv = kv.cuda()
    for pad in (80, 67):                                          # 16-byte stores, or not
        out = torch.full((50, 5, pad), 7.0, dtype=b.dt, device="cuda")
        attn = b.attn
        ws = torch.empty(attn.workspace_bytes, dtype=torch.uint8, device="cuda")
        K.indexer_causal_attention(attn, q.cuda()[:, 1:5, 8:72], kv[:, 0, :, :64], kv[:, 1, :, :64],
                                   torch.from_numpy(b.lens).cuda(), out[:, :4, :64], ws, page_table=b.table.cuda())
        assert torch.equal(out[:, :4, :64], want)
        assert torch.all(out[:, 4] == 7) and torch.all(out[:, :, 64:] == 7)


@pytest.mark.gpu
def test_far_slots():
    """A cache whose last keys are past 2^32 bytes from its start."""
    n, D = 18_000_000, 128
    k = torch.zeros(n, 1, D, dtype=torch.bfloat16, device="cuda")
    b = Batch([(3, 200)], 4, 1, D, page=40, seed=9)
    pages = torch.tensor([n // 40 - 1, 0, n // 40 - 7, 430_000, 420_000], dtype=torch.int32)
    at = b.table[0].long()[:, None] * 40 + torch.arange(40)
    to = (pages.long()[:, None] * 40 + torch.arange(40)).reshape(-1)
    want = b.run()
    v = torch.zeros_like(k)
    k[to.cuda()], v[to.cuda()] = b.k[at.reshape(-1)].cuda(), b.v[at.reshape(-1)].cuda()
    b.table, b.slots = pages[None], n
    got = b.run(edit=lambda *_: (k, v))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_two_streams_and_a_replay():
    """Two calls at once with a workspace each, a captured one replayed with other lengths."""
    b = Batch([(2, 3000), (1, 700)], 8, 2, 128, page=64, seed=10)
    c = Batch([(100, 400)], 4, 4, 64, 50, 1, seed=11)
    want_b, want_c = b.run(), c.run()
    args = []
    for x in (b, c):
        args.append([x.attn, x.q.cuda(), x.k.cuda(), x.v.cuda(), torch.from_numpy(x.lens).cuda(),
                     torch.empty(x.T, x.Hq, x.D, dtype=x.dt, device="cuda"),
                     torch.empty(x.attn.workspace_bytes, dtype=torch.uint8, device="cuda")])
    tables = [b.table.cuda(), None]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for st, a, t in zip(s, args, tables):
            K.indexer_causal_attention(*a, page_table=t, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(args[0][5], want_b[0]) and torch.equal(args[1][5], want_c[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for a, t in zip(args, tables):
            K.indexer_causal_attention(*a, page_table=t)
    b.lens = b.lens - np.array([900, 17, 699], dtype=np.int32)
    args[0][4].copy_(torch.from_numpy(b.lens))
    for a in args:
        a[5].fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    b.check(args[0][5], None)
    assert torch.equal(args[1][5], want_c[0])


def plan_of(rows, keys):
    return K.indexer_plan([0, rows], [0, keys], [keys] * rows, 32, 128, 8)


def test_refusals():
    p = plan_of(4, 100)
    make = K.indexer_causal_attention_create
    for kw in [dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(Hq=1026, Hkv=2), dict(window=-1), dict(sinks=-1),
               dict(dtype=K.IDX_FP32), dict(kv_format=2), dict(num_slots=-1), dict(page_size=-1),
               dict(scale=2e38), dict(scale=math.nan), dict(D=0)]:
        with pytest.raises(K.IndexerError) as e:
            make(p, **dict(dict(Hq=4, Hkv=2, D=64), **kw))
        assert e.value.code == K.IDX_ERR_INVALID_ARG, kw
    with pytest.raises(K.IndexerError) as e:
        make(p, 4, 2, 96)
    assert e.value.code == K.IDX_ERR_UNSUPPORTED
    lib = K.lib()
    base = dict(q=1024, k=1024, v=1024, out=1024, ks=0, vs=0, clen=1024, table=1024, lse=0, q_row=256, q_head=64,
                k_slot=128, k_head=64, v_slot=128, v_head=64, out_row=256, out_head=64, ld=7)
    dense, fp8 = make(p, 4, 2, 64, page_size=16), make(p, 4, 2, 64, page_size=16, kv_format=K.IDX_KV_FP8_E4M3)

    def call(a=dense, ws=4096, n=None, **kw):
        return lib.indexer_causal_attention(a.handle, K._CAUSAL_IO(*dict(base, **kw).values()), ws,
                                            a.workspace_bytes if n is None else n, None)
    for kw in [dict(q=0), dict(k=0), dict(v=0), dict(out=0), dict(clen=0), dict(table=0), dict(ld=6), dict(q=1032),
               dict(k=1032), dict(v=1032), dict(out=1025), dict(clen=1026), dict(table=1026), dict(lse=1026),
               dict(q_row=-8), dict(q_row=4), dict(q_head=4), dict(k_slot=4), dict(k_head=4), dict(v_slot=4),
               dict(v_head=4), dict(out_row=63), dict(out_head=63), dict(ws=0), dict(ws=128),
               dict(a=fp8), dict(a=fp8, ks=1024), dict(a=fp8, ks=1024, vs=1026),
               dict(a=fp8, ks=1024, vs=1024, k_slot=136)]:
        assert call(**kw) == K.IDX_ERR_INVALID_ARG, kw
    assert call(n=dense.workspace_bytes - 1) == K.IDX_ERR_WORKSPACE
    assert lib.indexer_causal_attention(None, K._CAUSAL_IO(*base.values()), 4096, 256, None) == K.IDX_ERR_INVALID_ARG
    if not torch.cuda.is_available():
        assert call() == K.IDX_ERR_UNSUPPORTED                    # nothing wrong but the device
        assert call(fp8, ks=1024, vs=1024) == K.IDX_ERR_UNSUPPORTED
    x = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                               # not on a GPU
        K.indexer_causal_attention(dense, x, x, x, x, x)
