"""Attention over the selected keys (indexer_sparse_attention) and the block lists of
candidate masks (indexer_mask_blocks), against the formulas in 64 bits.

Tolerance, from the operations, per row, head and element.  A score is a product of D terms
summed in fp32 (and, for e4m3 caches, of a query split into e4m3 terms whose rest is below
2^-20 of its largest element): off by at most
    ds = scale (D 2^-24 sum_i |q_i k_i| + 2^-20 max|q| sum_i |k_i|),
so a weight is off by a relative 2 max(ds) + 2^-20.  Weights enter the product with v with a
relative rounding of u_p (2^-8 for bf16 and for two e4m3 terms, 2^-11 for fp16) and an absolute
one of 2^-18 of the row's largest weighted scale.  The output is rounded once (u_o).
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from sparse_attention_prefill_tcgen05_gb300 import _lib as K

DT = {"bf16": (torch.bfloat16, K.IDX_BF16, 2.0 ** -8), "fp16": (torch.float16, K.IDX_FP16, 2.0 ** -11)}


def selected(sel, count, lens, L, block):
    """Per row the selected key positions, as they are listed."""
    rows = []
    for t in range(sel.shape[0]):
        n = sel.shape[1] if count is None else max(0, min(sel.shape[1], int(count[t])))
        keys = []
        for e in sel[t, :n].tolist():
            if e >= 0:
                keys += [e * block + i for i in range(block) if e * block + i < min(int(lens[t]), L[t])]
        rows.append(keys)
    return rows


def reference(q, k, v, keys, slot_of, Hkv, scale, ds_only=False):
    """out, lse and the tolerance's terms in 64 bits; slot_of(t, j) is the cache row or -1."""
    T, Hq, D = q.shape
    G = Hq // Hkv
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    ds, wabs, vabs, pmax = np.zeros((T, Hq)), np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for t in range(T):
        at = [s for s in (slot_of(t, j) for j in keys[t]) if s >= 0]
        if not at:
            continue
        for g in range(Hkv):
            kk, vv = k[at, g], v[at, g]
            qq = q[t, g * G:(g + 1) * G]
            a = scale * (qq @ kk.T)
            mx = a.max(axis=1, keepdims=True)
            e = np.exp(a - mx)
            z = e.sum(axis=1, keepdims=True)
            p = e / z
            h = slice(g * G, (g + 1) * G)
            out[t, h] = p @ vv
            lse[t, h] = (mx + np.log(z))[:, 0]
            ds[t, h] = abs(scale) * (D * 2.0 ** -24 * (np.abs(qq) @ np.abs(kk).T)
                                     + 2.0 ** -20 * np.abs(qq).max(axis=1, keepdims=True)
                                     * np.abs(kk).sum(axis=1)[None]).max(axis=1)
            wabs[t, h] = p @ np.abs(vv)
            # e4m3 weights carry v's scale: relative to the row's largest p * |v|
            vabs[t, h] = len(at) * np.abs(vv).max()
            pmax[t, h] = p.max()
    return out, lse, ds, wabs, vabs, pmax


def check(got, lse, ref, up, uo):
    out, want_lse, ds, wabs, vabs, pmax = ref
    g = got.double().cpu().numpy()
    tol = (up + 2 * ds[..., None] + 2.0 ** -20) * wabs + 2.0 ** -18 * (pmax[..., None] * vabs) \
        + uo * np.abs(out) + 2.0 ** -25
    assert np.all(np.isfinite(g))
    assert np.all(np.abs(g - out) <= tol), float(np.max(np.abs(g - out) - tol))
    e = np.isneginf(want_lse)
    if lse is not None:
        z = lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(z), e)
        assert np.all(np.abs(z[~e] - want_lse[~e]) <= ds[~e] + 2.0 ** -20 * (1 + np.abs(want_lse[~e])))
    assert np.all(g[e] == 0)


class Batch:
    """A ragged batch: requests of (rows, keys); the last row of a request sees every key."""

    def __init__(self, requests, Hq, Hkv, D, nsel, block=1, dt="bf16", kv="same", page=0, seed=0,
                 spread=1.0, lens=None):
        self.g = torch.Generator().manual_seed(seed)
        self.dt, self.code, self.u = DT[dt]
        self.kv, self.page, self.block, self.nsel = kv, page, block, nsel
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        rows, keys = [r for r, _ in requests], [n for _, n in requests]
        self.cu_q = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.cu_k = np.concatenate([[0], np.cumsum(keys)]).astype(np.int32)
        self.T, self.req = int(self.cu_q[-1]), np.repeat(np.arange(len(rows)), rows)
        self.L = np.array([keys[r] for r in self.req], dtype=np.int64)
        if lens is None:
            lens = np.concatenate([np.clip(n - r + 1 + np.arange(r), 0, n) for r, n in requests]) \
                if self.T else np.zeros(0)
        self.lens = np.asarray(lens).astype(np.int32)
        self.plan = K.indexer_plan(self.cu_q, self.cu_k, np.minimum(self.lens, self.L).astype(np.int32),
                                   32, 128, 8)
        if page:
            per = -(-max(keys) // page)
            self.table = torch.randperm(len(rows) * per, generator=self.g).to(torch.int32).reshape(
                len(rows), per)
            self.slots = len(rows) * per * page
        else:
            self.table, self.slots = None, int(self.cu_k[-1])
        rnd = lambda *s: torch.randn(s, generator=self.g)
        self.q = (rnd(self.T, Hq, D) * spread).to(self.dt)
        kf, vf = rnd(self.slots, Hkv, D), rnd(self.slots, Hkv, D)
        if kv == "fp8":
            # each vector has its own scale, far apart
            self.ks = torch.exp2(torch.randint(-3, 3, (self.slots, Hkv), generator=self.g).float()) / 200
            self.vs = torch.exp2(torch.randint(-6, 6, (self.slots, Hkv), generator=self.g).float()) / 200
            self.k = (kf * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            self.v = (vf * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            self.ks = self.vs = None
            self.k, self.v = kf.to(self.dt), vf.to(self.dt)
        # distinct selected entries of every row's valid ones, in random order, then -1
        self.sel = torch.full((self.T, nsel), -1, dtype=torch.int32)
        for t in range(self.T):
            nb = -(-int(min(self.lens[t], self.L[t])) // block)
            pick = torch.randperm(max(nb, 0), generator=self.g)[:nsel]
            self.sel[t, :len(pick)] = pick.to(torch.int32)
        self.count = None

    def slot_of(self, t, j):
        r = int(self.req[t])
        if self.page == 0:
            s = int(self.cu_k[r]) + j
        else:
            pg = int(self.table[r, j // self.page])
            s = pg * self.page + j % self.page if pg >= 0 else -1
        return s if 0 <= s < self.slots else -1

    def values(self):
        if self.kv == "fp8":
            f = lambda c, s: (c.view(torch.float8_e4m3fn).double() * s.double()[..., None]).numpy()
            return f(self.k, self.ks), f(self.v, self.vs)
        return self.k.double().numpy(), self.v.double().numpy()

    def attention(self, scale=None):
        return K.indexer_attention_create(
            self.plan, self.Hq, self.Hkv, self.D, self.nsel, block=self.block, dtype=self.code,
            kv_format=K.IDX_KV_FP8_E4M3 if self.kv == "fp8" else K.IDX_KV_DENSE,
            num_slots=self.slots, page_size=self.page, scale=scale)

    def run(self, scale=None, attn=None, ws=None, with_lse=True):
        c = lambda x: None if x is None else x.cuda()
        attn = attn or self.attention(scale)
        out = torch.full((self.T, self.Hq, self.D), 7.0, dtype=self.dt, device="cuda")
        lse = torch.full((self.T, self.Hq), 7.0, device="cuda") if with_lse else None
        if ws is None:
            ws = torch.empty(max(attn.workspace_bytes, 256), dtype=torch.uint8, device="cuda")
        K.indexer_sparse_attention(attn, c(self.q), c(self.k), c(self.v), c(self.sel),
                                   torch.from_numpy(self.lens).cuda(), out, ws, k_scale=c(self.ks),
                                   v_scale=c(self.vs), sel_count=c(self.count),
                                   page_table=c(self.table), lse=lse)
        assert K.indexer_status(None, ws) == K.IDX_OK
        return out, lse

    def check(self, scale=None, **kw):
        out, lse = self.run(scale, **kw)
        keys = selected(self.sel, self.count, self.lens, self.L, self.block)
        kf, vf = self.values()
        ref = reference(self.q.double().numpy(), kf, vf, keys, self.slot_of, self.Hkv,
                        self.D ** -0.5 if scale is None else scale)
        up = 2.0 ** -8 if self.kv == "fp8" else self.u
        check(out, lse, ref, up, self.u)
        return out, lse


# ------------------------------------------------------------------------- refusals


def _plan(T=4, L=100):
    return K.indexer_plan(np.array([0, T], np.int32), np.array([0, L], np.int32),
                          np.full(T, L, np.int32), 32, 128, 8)


def test_spec_refusals():
    plan = _plan()

    def create(**kw):
        a = dict(Hq=8, Hkv=2, D=128, num_sel=16)
        a.update(kw)
        return K.indexer_attention_create(plan, **a)
    create()
    create(D=64, block=128, page_size=16, kv_format=K.IDX_KV_FP8_E4M3, dtype=K.IDX_FP16)
    for code, kw in [(K.IDX_ERR_INVALID_ARG, x) for x in (
            dict(Hq=0), dict(Hkv=0), dict(Hq=9), dict(Hq=1025, Hkv=1), dict(block=3), dict(block=0),
            dict(block=256), dict(num_sel=0), dict(num_sel=65537), dict(dtype=K.IDX_FP32),
            dict(kv_format=2), dict(num_slots=-1), dict(page_size=-1), dict(scale=math.nan),
            dict(D=0))] + [(K.IDX_ERR_UNSUPPORTED, dict(D=96)), (K.IDX_ERR_UNSUPPORTED, dict(D=256))]:
        with pytest.raises(K.IndexerError) as e:
            create(**kw)
        assert e.value.code == code, kw
    L = K.lib()
    assert L.indexer_attention_create(None, None, None, None) == K.IDX_ERR_INVALID_ARG


def test_call_refusals():
    L, plan = K.lib(), _plan()
    A, odd = 0x100000, 0x100008
    for fmt in (K.IDX_KV_DENSE, K.IDX_KV_FP8_E4M3):
        attn = K.indexer_attention_create(plan, 8, 2, 128, 16, kv_format=fmt, page_size=16)
        good = dict(q=A, k=A, v=A, out=A, sel=A, compress_len=A, page_table=A, q_row=1024, q_head=128,
                    k_slot=256, k_head=128, v_slot=256, v_head=128, out_row=1024, out_head=128,
                    ld_sel=16, ld_page_table=7, k_scale=A, v_scale=A)

        def call(attn=attn, ws=ctypes.c_void_p(A), n=1 << 30, **kw):
            io = K._AttentionIo(**{**good, **kw})
            return L.indexer_sparse_attention(attn.handle if attn else None, ctypes.byref(io), ws, n,
                                              None)
        bad = [dict(attn=None), dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(sel=None),
               dict(compress_len=None), dict(page_table=None), dict(ld_page_table=6), dict(ld_sel=15),
               dict(q=odd), dict(k=odd), dict(v=odd), dict(q_row=1028), dict(q_row=-1024),
               dict(k_slot=260), dict(v_head=132), dict(out_row=100), dict(out_head=64),
               dict(out=0x100001), dict(lse=0x100002), dict(sel=0x100001)]
        if fmt == K.IDX_KV_FP8_E4M3:
            bad += [dict(k_scale=None), dict(v_scale=None), dict(k_slot=264)]
        for kw in bad:
            assert call(**kw) == K.IDX_ERR_INVALID_ARG, kw
        assert L.indexer_sparse_attention(attn.handle, None, None, 0, None) == K.IDX_ERR_INVALID_ARG
        if attn.workspace_bytes:
            assert call(n=attn.workspace_bytes - 1) == K.IDX_ERR_WORKSPACE
            assert call(ws=ctypes.c_void_p(A + 16)) == K.IDX_ERR_INVALID_ARG
            assert call(ws=None) == K.IDX_ERR_INVALID_ARG


def test_mask_blocks_refusals():
    L, plan, A, N = K.lib(), _plan(), ctypes.c_void_p(0x100000), ctypes.c_void_p(0)
    f = L.indexer_mask_blocks
    for args in ((None, A, 13, A, 8, A, 4, A), (plan.handle, N, 13, A, 8, A, 4, A),
                 (plan.handle, A, 12, A, 8, A, 4, A), (plan.handle, A, 13, N, 8, A, 4, A),
                 (plan.handle, A, 13, A, 0, A, 4, A), (plan.handle, A, 13, A, 8, N, 4, A),
                 (plan.handle, A, 13, A, 8, A, 0, A)):
        assert f(*args, N) == K.IDX_ERR_INVALID_ARG


# --------------------------------------------------------------------------- numbers

SHAPES = [
    # requests, Hq, Hkv, D, nsel, block
    (((64, 1024),), 4, 1, 64, 32, 1),
    (((3, 700),), 32, 1, 128, 300, 1),
    (((1, 1),), 1, 1, 128, 1, 1),
    (((5, 40), (1, 600), (2, 129)), 32, 4, 128, 20, 8),
    (((4, 2000),), 64, 1, 128, 128, 1),
    (((2, 500), (3, 0), (2, 3)), 16, 2, 64, 129, 1),
    (((6, 900),), 40, 1, 64, 257, 1),                 # a group that is no power of two
    (((2, 800),), 96, 1, 128, 130, 1),                # more heads than one tile
    (((3, 1000),), 8, 8, 128, 7, 64),                 # one head a group, blocks past the tile's half
    (((2, 3000),), 20, 4, 64, 9, 128),
    (((300, 310),), 8, 2, 64, 16, 2),                 # more rows than SMs
    (((7, 6000),), 32, 1, 64, 2048, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [0, 16, 48])
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_the_formula(shape, dt, kv, page):
    requests, Hq, Hkv, D, nsel, block = shape
    Batch(requests, Hq, Hkv, D, nsel, block, dt, kv, page, seed=Hq + nsel).check()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
@pytest.mark.parametrize("scale,spread", [(1.0, 3.0), (-0.5, 1.0), (0.0, 1.0), (0.05, 40.0)])
def test_scales_and_peaked_rows(scale, spread, kv):
    """Rows whose weight sits on a few keys, equal scores, and falling ones."""
    Batch(((9, 800),), 32, 1, 128, 400, 1, "bf16", kv, 16, seed=5, spread=spread).check(scale)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_a_maximum_that_moves_through_the_list(order, kv):
    """Scores that rise (or fall) by hundreds over the list: the running maximum is replaced in
    every tile, and everything before it loses its weight."""
    b = Batch(((3, 640),), 16, 1, 64, 640, 1, "bf16", kv, 0, seed=6)
    b.sel = torch.arange(640, dtype=torch.int32).repeat(3, 1)
    ramp = torch.linspace(-1, 1, 640) * (1 if order == "rising" else -1)
    b.q = torch.full((3, 16, 64), 8.0).to(b.dt)
    if kv == "fp8":
        b.k = (ramp[:, None, None] * 400).expand(640, 1, 64).to(torch.float8_e4m3fn).view(
            torch.uint8).contiguous()
        b.ks = torch.full((640, 1), 0.01)
    else:
        b.k = (ramp[:, None, None] * 4).expand(640, 1, 64).to(b.dt).contiguous()
    b.lens[:] = 640
    b.check(scale=0.25)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,G,Hkv,D,kv,dt,kernel", [
    (40, 8, 1, 64, "same", "bf16", True), (33, 5, 2, 64, "fp8", "bf16", False),
    (64, 32, 1, 128, "fp8", "bf16", False), (48, 40, 1, 128, "same", "fp16", False),
    (16, 16, 1, 64, "fp8", "fp16", True),
    (30, 16, 1, 64, "fp8", "fp16", False), (5, 70, 1, 128, "same", "bf16", False),
    (9, 9, 3, 128, "same", "bf16", False), (1, 64, 1, 128, "fp8", "bf16", True),
    (2, 3, 2, 64, "same", "fp16", True),
])
def test_split_rows(rows, G, Hkv, D, kv, dt, kernel):
    """Rows too few for the SMs, over 2,048 keys each: joined within a cluster or, in three parts or
    more than four, by a kernel, which shows in the workspace; lists that leave splits empty."""
    b = Batch(((rows, 2100),), G * Hkv, Hkv, D, 2048, 1, dt, kv, 16, seed=rows + G)
    for t, n in enumerate((2048, 0, 1, 128, 129, 700, 1024, 1025, 1920)):
        if t + 1 < rows:
            b.sel[t, n:] = -1
    attn = b.attention()
    assert (attn.workspace_bytes > 256) == kernel
    b.check(attn=attn)
    b.count = torch.tensor([(0, 3, 2048, 1100, 257)[t % 5] for t in range(rows)], dtype=torch.int32)
    b.check(attn=attn)
    b.check(attn=attn, with_lse=False)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
@pytest.mark.parametrize("block", [1, 8])
def test_rows_that_select_nothing_and_lists_with_holes(block, kv):
    b = Batch(((12, 600),), 32, 2, 128, 200, block, "bf16", kv, 16, seed=7,
              lens=[600, 0, 599, 5, 600, 600, 600, 600, 1, 600, 600, 601])
    big = 2 ** 31 - 1
    b.sel[2, ::2] = -1                                # holes
    b.sel[3, :] = 50 // block + 1                     # past the row's length
    b.sel[4, :] = -1
    b.sel[5, 1:] = big                                # far past it (the product passes 32 bits)
    b.sel[6, :150] = -2 ** 31
    b.sel[7, :] = 3                                   # one entry, 200 times over
    b.sel[8, :] = -1
    b.sel[8, 199] = 0                                 # one key, at the end of the list
    b.sel[9, :] = 600 // block                        # the request's last, part of it past the end
    b.sel[11, 0] = 600 // block
    b.table[0, 4] = -1                                # an unmapped page
    b.table[0, 5] = b.slots // 16 + 3                 # a page past the cache
    b.check()
    b.count = torch.tensor([200, 200, 7, 200, 0, -3, 199, 129, 200, 128, 127, 500], dtype=torch.int32)
    b.check()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
def test_nan_and_infinities_outside_the_selection_do_not_matter(kv):
    b = Batch(((5, 301),), 32, 1, 128, 30, 8, "bf16", kv, 16, seed=8, lens=[297, 298, 299, 300, 301])
    used = torch.zeros(b.slots, dtype=torch.bool)
    keys = selected(b.sel, None, b.lens, b.L, 8)
    for t in range(5):
        for j in keys[t]:
            used[b.slot_of(t, j)] = True
    want = b.run()
    for bad in (float("nan"), float("inf"), -float("inf")):
        if kv == "fp8":
            b.k[~used], b.v[~used] = 0x7F, 0xFF
            b.ks[~used], b.vs[~used] = bad, bad
        else:
            b.k[~used], b.v[~used] = bad, bad
        got = b.run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a key past the row's length in a block that the row selects: only later rows see it
    b.sel[:, 0] = 37                                  # keys 296..303 of 301
    last = b.slot_of(0, 300)
    if kv == "same":
        b.v[last] = 1.0
        b.k[last] = 1.0
        clean = b.run()
        b.v[last] = float("nan")
        got = b.run()
        assert torch.equal(got[0][:4], clean[0][:4]) and bool(torch.isnan(got[0][4]).any())


@pytest.mark.gpu
def test_nan_in_a_selected_key_shows():
    b = Batch(((3, 200),), 16, 1, 64, 20, 1, seed=9)
    b.k[b.slot_of(0, int(b.sel[1, 3])), 0, 5] = float("nan")
    out, lse = b.run()
    has = [int(b.sel[1, 3]) in b.sel[t].tolist() for t in range(3)]
    for t in range(3):
        assert bool(torch.isnan(out[t]).all()) == has[t] and bool(torch.isnan(lse[t]).all()) == has[t]


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_head_that_is_not_finite_leaves_the_others_alone(bad, kv):
    b = Batch(((3, 300),), 32, 1, 128, 150, 1, "bf16", kv, 0, seed=15)
    q = b.q.clone()
    b.q[1, 5, 17] = bad
    got, lse = b.run()
    assert bool(torch.isnan(got[1, 5]).all()) and bool(torch.isnan(lse[1, 5]))
    kf, vf = b.values()
    keys = selected(b.sel, None, b.lens, b.L, 1)
    ref = reference(q.double().numpy(), kf, vf, keys, b.slot_of, 1, 128 ** -0.5)
    got[1, 5] = torch.from_numpy(ref[0][1, 5]).to(got)          # the others are held to the formula
    lse[1, 5] = float(ref[1][1, 5])
    check(got, lse, ref, 2.0 ** -8, 2.0 ** -8)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
def test_strides(kv):
    """q and out inside wider tensors, heads outermost, k and v side by side in one cache."""
    b = Batch(((40, 300),), 32, 4, 128, 60, 1, "bf16", kv, 0, seed=10)
    want, want_lse = b.run()
    attn = b.attention()
    ws = torch.empty(max(attn.workspace_bytes, 256), dtype=torch.uint8, device="cuda")
    wide = torch.zeros((40, 50, 256), dtype=b.dt, device="cuda")
    q = wide[:, 5:37, 64:192]
    q.copy_(b.q)
    both = torch.empty((300, 2, 4, 128), dtype=b.k.dtype, device="cuda")
    both[:, 0], both[:, 1] = b.k.cuda(), b.v.cuda()
    out = torch.full((33, 40, 131), 9.0, dtype=b.dt, device="cuda")   # heads first, 2-byte aligned
    o = out[1:, :, 3:].transpose(0, 1)
    sel = torch.full((40, 77), -1, dtype=torch.int32, device="cuda")
    sel[:, :60] = b.sel.cuda()
    c = lambda x: None if x is None else x.cuda()
    args = dict(k_scale=c(b.ks), v_scale=c(b.vs))
    lens = torch.from_numpy(b.lens).cuda()
    K.indexer_sparse_attention(attn, q, both[:, 0], both[:, 1], sel[:, :60], lens, o, ws, **args)
    assert torch.equal(o, want)
    assert torch.all(out[0] == 9) and torch.all(out[:, :, :3] == 9)
    kh = both[:, 0].permute(1, 0, 2).contiguous().permute(1, 0, 2)    # [Hkv, slots, D] cache
    K.indexer_sparse_attention(attn, q, kh, both[:, 1], sel[:, :60], lens, o, ws, **args)
    assert torch.equal(o, want)


@pytest.mark.gpu
def test_broadcast_queries_and_shared_keys():
    """Zero strides: one query row for all, one key row for all."""
    b = Batch(((6, 100),), 16, 1, 64, 30, 1, seed=11)
    attn = b.attention()
    ws = torch.empty(max(attn.workspace_bytes, 256), dtype=torch.uint8, device="cuda")
    q = b.q[:1].cuda().expand(6, 16, 64)
    k = b.k[:1].cuda().expand(100, 1, 64)
    out = torch.empty((6, 16, 64), dtype=b.dt, device="cuda")
    K.indexer_sparse_attention(attn, q, k, b.v.cuda(), b.sel.cuda(), torch.from_numpy(b.lens).cuda(),
                               out, ws)
    b.q, b.k = b.q[:1].repeat(6, 1, 1), b.k[:1].repeat(100, 1, 1)
    want, _ = b.run()
    assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
def test_runs_and_streams_give_the_same_bits(kv):
    b = Batch(((3, 3000),), 32, 1, 128, 1500, 1, "bf16", kv, 16, seed=12)
    first, lse = b.run()
    ws = torch.full((max(b.attention().workspace_bytes, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        again, lse2 = b.run(ws=ws)
        assert torch.equal(first, again) and torch.equal(lse, lse2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other, _ = b.run(with_lse=False)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["same", "fp8"])
def test_cache_offsets_past_32_bits(kv):
    """Slots whose byte offsets pass 2^31 and 2^32 in a long paged cache."""
    b = Batch(((2, 256),), 16, 1, 128, 100, 1, "bf16", kv, 64, seed=13)
    want, _ = b.run()
    bytes_row = 128 if kv == "fp8" else 256
    n = ((5 << 30) // bytes_row) // 64 * 64
    old, new = b.table.clone(), torch.tensor([[1, n // 64 - 1, (n // 64) // 2, 7]], dtype=torch.int32)
    big = {}
    for name in ("k", "v"):
        t = torch.empty((n, 1, 128), dtype=getattr(b, name).dtype, device="cuda")
        for i in range(4):
            o, w = int(old[0, i]) * 64, int(new[0, i]) * 64
            t[w:w + 64] = getattr(b, name)[o:o + 64].cuda()
        big[name] = t
        sc = getattr(b, name + "s")
        if sc is not None:
            s = torch.zeros((n, 1), device="cuda")
            for i in range(4):
                o, w = int(old[0, i]) * 64, int(new[0, i]) * 64
                s[w:w + 64] = sc[o:o + 64].cuda()
            big[name + "s"] = s
    attn = K.indexer_attention_create(b.plan, 16, 1, 128, 100, kv_format=int(kv == "fp8"), num_slots=n,
                                      page_size=64)
    ws = torch.empty(max(attn.workspace_bytes, 256), dtype=torch.uint8, device="cuda")
    out = torch.empty((2, 16, 128), dtype=b.dt, device="cuda")
    K.indexer_sparse_attention(attn, b.q.cuda(), big["k"], big["v"], b.sel.cuda(),
                               torch.from_numpy(b.lens).cuda(), out, ws, k_scale=big.get("ks"),
                               v_scale=big.get("vs"), page_table=new.cuda())
    assert torch.equal(out, want)


@pytest.mark.gpu
def test_no_rows():
    cu = np.array([0, 0], np.int32)
    plan = K.indexer_plan(cu, np.array([0, 10], np.int32), np.zeros(0, np.int32), 32, 128, 8)
    attn = K.indexer_attention_create(plan, 8, 1, 64, 4)
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
    i = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
    K.indexer_sparse_attention(attn, e(0, 8, 64), e(10, 1, 64), e(10, 1, 64), i(0, 4), i(0), e(0, 8, 64))


# ------------------------------------------------------------------------ mask lists


@pytest.mark.gpu
@pytest.mark.parametrize("block,nsel", [(8, 64), (8, 3), (1, 500), (48, 7)])
def test_mask_blocks(block, nsel):
    g = torch.Generator().manual_seed(block)
    requests = ((40, 900), (3, 0), (5, 33), (1, 40000))
    cu_q = np.concatenate([[0], np.cumsum([r for r, _ in requests])]).astype(np.int32)
    cu_k = np.concatenate([[0], np.cumsum([n for _, n in requests])]).astype(np.int32)
    L = np.repeat([n for _, n in requests], [r for r, _ in requests])
    lens = (L - torch.randint(0, 30, (len(L),), generator=g).numpy()).clip(0).astype(np.int32)
    plan = K.indexer_plan(cu_q, cu_k, lens, 32, 128, 8)
    ld = -(-40000 // block) + 5
    mask = (torch.rand((len(L), ld), generator=g) < 0.3).to(torch.uint8) * 255
    mask[1], mask[2] = 0, 1
    blocks = torch.full((len(L), nsel), 99, dtype=torch.int32, device="cuda")
    count = torch.full((len(L),), 99, dtype=torch.int32, device="cuda")
    dl = torch.from_numpy(lens).cuda()
    K.indexer_mask_blocks(plan, mask.cuda(), dl, block, blocks, count)
    again = torch.empty_like(blocks)
    K.indexer_mask_blocks(plan, mask.cuda(), dl, block, again)
    assert torch.equal(blocks, again)
    for t in range(len(L)):
        nb = -(-int(lens[t]) // block)
        want = torch.nonzero(mask[t, :nb])[:, 0][:nsel].tolist()
        assert int(count[t]) == len(want)
        assert blocks[t].tolist() == want + [-1] * (nsel - len(want))


@pytest.mark.gpu
def test_candidate_mask_to_attention():
    """The blocks a candidate mask names are what attention with that many blocks reads."""
    b = Batch(((10, 400),), 16, 2, 64, 25, 8, seed=14)
    mask = torch.zeros((10, 50), dtype=torch.uint8)
    for t in range(10):
        mask[t, b.sel[t][b.sel[t] >= 0].long()] = 1
    blocks = torch.empty((10, 25), dtype=torch.int32, device="cuda")
    count = torch.empty((10,), dtype=torch.int32, device="cuda")
    K.indexer_mask_blocks(b.plan, mask.cuda(), torch.from_numpy(b.lens).cuda(), 8, blocks, count)
    b.sel, b.count = blocks.cpu(), count.cpu()
    b.check()
