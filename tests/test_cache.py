"""Quantised operands and caches (indexer_cache_write / _read, indexer_page_slots).

What a written vector must be, from the definition in 64 bits: with y the rotated vector (off
by at most 1e-6 (|a| + |b|) as in the rotation's own tests, 0 without a rotation) and s the
stored scale, every code is the grid's nearest value to y / s up to that error and a relative
2^-21 for the two roundings of s and 1/s; the scale is max|y| / 448 within 4e-6 (e4m3), or
the power of two floor(log2(max|y|)) - 2 (e2m1).
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import oracle as O
from sparse_attention_prefill_tcgen05_gb300 import _lib as K

from .test_rope import frequencies, rotated

FP8, FP4 = K.IDX_K_FP8_E4M3, K.IDX_K_FP4_E2M1_UE8M0
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6.0])


def storage(slots, heads, D, fmt, fill=0x5A):
    n = D // 2 if fmt == FP4 else D
    codes = torch.full((slots, heads, n), fill, dtype=torch.uint8, device="cuda")
    if fmt == FP4:
        return codes, torch.full((slots, heads, D // 32), 100, dtype=torch.uint8, device="cuda")
    return codes, torch.full((slots, heads), 3.0, device="cuda")


def decoded(codes, scales, fmt):
    """Code values and per-element scales in 64 bits, by the formats' definitions."""
    c = codes.cpu().numpy()
    if fmt == FP8:
        table = np.array([O.lib().oracle_e4m3_value(i) for i in range(256)])
        v = table[c]
        return v, np.broadcast_to(scales.double().cpu().numpy()[..., None], v.shape)
    v = np.stack([E2M1[c & 15], E2M1[c >> 4]], axis=-1).reshape(*c.shape[:-1], -1)
    s = 2.0 ** (scales.cpu().numpy().astype(np.float64) - 127)
    return v, np.repeat(s, 32, axis=-1)


def half_step(v, fmt):
    """Half the distance between the grid's neighbours around |v|."""
    lo, top, bits = (-6, 448.0, 3) if fmt == FP8 else (0, 6.0, 1)
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** lo)))
    return 2.0 ** (np.minimum(e, np.floor(np.log2(top))) - bits - 1)


def check_vectors(codes, scales, fmt, y, err):
    v, s = decoded(codes, scales, fmt)
    amax = np.abs(y).max(axis=-1)
    if fmt == FP8:
        want = np.where(amax > 0, np.maximum(amax / 448, 2.0 ** -126), 1.0)
        got = scales.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= 4e-6 * want)
    else:
        blocks = np.abs(y).reshape(*y.shape[:-1], -1, 32).max(axis=-1)
        got = scales.cpu().numpy().astype(np.int64) - 127
        near = [np.floor(np.log2(np.maximum(blocks * f, 1e-300))) - 2 for f in (1 - 4e-6, 1 + 4e-6)]
        ok = (got == near[0]) | (got == near[1]) | ((blocks == 0) & (got == 0)) | \
             ((got == -127) & (near[1] <= -127))
        assert np.all(ok)
    top = 448.0 if fmt == FP8 else 6.0
    want = np.clip(y / s, -top, top)
    # nearest: no further than half the wider of the steps on both sides
    tol = np.maximum(half_step(want, fmt), half_step(v, fmt)) + 2.0 ** -21 * np.abs(want) + err / s
    assert np.all(np.abs(v - want) <= tol), float(np.max(np.abs(v - want) - tol))


def test_refusals():
    L, A, N = K.lib(), ctypes.c_void_p(0x100000), ctypes.c_void_p(0)
    r = K.indexer_rope_create(64, 64)

    def write(rope=None, x=A, dt=K.IDX_BF16, rows=4, heads=1, D=128, rs=128, hs=128, pos=A, slots=A,
              n=8, fmt=FP8, codes=A, scales=A):
        return L.indexer_cache_write(rope, x, dt, rows, heads, D, rs, hs, pos, slots, n, fmt, codes,
                                     scales, N)
    for kw in (dict(x=N), dict(codes=N), dict(scales=N), dict(dt=3), dict(rows=-1), dict(heads=0),
               dict(D=48), dict(D=0), dict(D=288), dict(n=-1), dict(fmt=2), dict(rs=-1),
               dict(rope=r.handle), dict(slots=N, rows=9), dict(codes=ctypes.c_void_p(0x100008)),
               dict(scales=ctypes.c_void_p(0x100002)), dict(x=ctypes.c_void_p(0x100001))):
        assert write(**kw) == K.IDX_ERR_INVALID_ARG, kw
    assert write(rope=r.handle, D=64, pos=N) == K.IDX_ERR_INVALID_ARG

    def read(codes=A, scales=A, fmt=FP8, n=8, heads=1, D=128, slots=A, rows=4, dt=K.IDX_BF16, out=A,
             osc=N):
        return L.indexer_cache_read(codes, scales, fmt, n, heads, D, slots, rows, dt, out, osc, N)
    for kw in (dict(codes=N), dict(scales=N), dict(out=N), dict(fmt=5), dict(n=-1), dict(heads=0),
               dict(D=40), dict(rows=-1), dict(dt=4), dict(dt=K.IDX_CODES),
               dict(out=ctypes.c_void_p(0x100004)), dict(slots=N, rows=9)):
        assert read(**kw) == K.IDX_ERR_INVALID_ARG, kw
    cu = np.array([0, 4], np.int32)
    plan = K.indexer_plan(cu, np.array([0, 100], np.int32), np.full(4, 100, np.int32), 32, 128, 8)
    page = L.indexer_page_slots
    assert page(plan.handle, A, 6, 16, A, N) == K.IDX_ERR_INVALID_ARG      # 100 / 16 -> 7 pages
    assert page(plan.handle, A, 7, 0, A, N) == K.IDX_ERR_INVALID_ARG
    assert page(plan.handle, N, 7, 16, A, N) == K.IDX_ERR_INVALID_ARG
    assert page(plan.handle, A, 7, 16, N, N) == K.IDX_ERR_INVALID_ARG
    assert page(None, A, 7, 16, A, N) == K.IDX_ERR_INVALID_ARG


WRITES = [
    # rows, heads, D, rot, offset, interleaved, dtype
    (64, 1, 128, 64, 0, True, torch.bfloat16),
    (37, 32, 128, 128, 0, False, torch.bfloat16),
    (1, 4, 64, 32, 32, False, torch.float16),
    (53, 3, 96, 32, 8, False, torch.float32),
    (20, 2, 32, 32, 0, True, torch.float32),
    (31, 2, 160, 48, 24, False, torch.float16),
    (25, 5, 256, 256, 0, False, torch.bfloat16),
    (29, 2, 96, 24, 4, False, torch.bfloat16),         # no whole units
    (40, 2, 128, 0, 0, False, torch.float32),          # no rotation
]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [FP8, FP4])
@pytest.mark.parametrize("rows,heads,D,rot,offset,inter,dt", WRITES)
def test_written_vectors(rows, heads, D, rot, offset, inter, dt, fmt):
    g = torch.Generator().manual_seed(rows * D)
    x = (torch.randn((rows, heads, D), generator=g) * torch.exp2(
        torch.randint(-12, 12, (rows, heads, 1), generator=g).float())).to(dt)
    x[0] = 0                                           # a zero vector
    x = x.cuda()
    pos = torch.randint(0, 150000, (rows,), generator=g, dtype=torch.int32).cuda()
    n = rows + 13
    slots = torch.randperm(n, generator=g)[:rows].to(torch.int32)
    if rows > 3:
        slots[2], slots[3] = -1, n                     # skipped rows
    codes, scales = storage(n, heads, D, fmt)
    before = codes.clone(), scales.clone()
    rope = K.indexer_rope_create(D, rot, offset, int(inter)) if rot else None
    K.indexer_cache_write(x, codes, scales, fmt, rope=rope, positions=pos if rot else None,
                          slots=slots.cuda())
    y, mag = x.double().cpu().numpy(), np.zeros((rows, heads, D))
    if rot:
        y, mag = rotated(y, pos.cpu().numpy(), rot, offset, inter, frequencies(rot))
    ok = (slots >= 0) & (slots < n)
    at = slots[ok].long().cuda()
    check_vectors(codes[at], scales[at], fmt, y[ok.numpy()], 1e-6 * mag[ok.numpy()])
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(codes[rest], before[0][rest]) and torch.equal(scales[rest], before[1][rest])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [FP8, FP4])
def test_exact_values_ties_and_extremes(fmt):
    """Inputs whose scale is a power of two: every rounding is known exactly."""
    D = 64
    x = torch.zeros((6, 1, D))
    top, tie, even = (448.0, 17.0, 16.0) if fmt == FP8 else (4.0, 2.5, 2.0)
    x[0, 0, :] = top
    x[0, 0, 1::2] = tie                                # halfway, to the even code
    x[1, 0, :] = -top * 2.0 ** -100
    x[2, 0, 5] = float("nan")
    x[2, 0, 40] = top
    x[3, 0, 7] = float("inf")
    x[3, 0, 8] = -float("inf")
    x[4, 0, :] = 2.0 ** -149                           # subnormal
    x[5, 0, 0] = 3.4028234e38
    codes, scales = storage(6, 1, D, fmt)
    K.indexer_cache_write(x.cuda(), codes, scales, fmt)
    v, s = decoded(codes, scales, fmt)
    w = v * s
    assert np.all(w[0, 0, 0::2] == top) and np.all(w[0, 0, 1::2] == even)
    assert np.all(np.isfinite(w)) and np.all(s > 0) and np.all(np.isfinite(s))
    assert np.all(w[1, 0] == -top * 2.0 ** -100)
    assert w[2, 0, 5] == 0 and w[2, 0, 40] == top
    big = 448.0 if fmt == FP8 else 6.0
    assert v[3, 0, 7] == big and v[3, 0, 8] == -big
    assert np.all(np.abs(w[4, 0]) <= 2.0 ** -127) 
    assert v[5, 0, 0] == big
    if fmt == FP8:
        assert not np.any((codes.cpu().numpy() & 0x7F) == 0x7F)     # no NaN code


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [FP8, FP4])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,heads,D", [(50, 1, 128), (7, 3, 96), (1, 1, 32), (300, 4, 64)])
def test_read_back(rows, heads, D, dt, fmt):
    g = torch.Generator().manual_seed(D + rows)
    n = 64
    codes, scales = storage(n, heads, D, fmt)
    codes.copy_(torch.randint(0, 127, codes.shape, generator=g).to(torch.uint8))
    if fmt == FP8:
        scales.copy_(torch.rand(scales.shape, generator=g) + 0.01)
    else:
        scales.copy_(torch.randint(120, 132, scales.shape, generator=g).to(torch.uint8))
    slots = torch.randint(0, n, (rows,), generator=g, dtype=torch.int32)
    if rows > 4:
        slots[1], slots[3] = -1, n
    out = torch.full((rows, heads, D), 9.0, dtype=dt, device="cuda")
    K.indexer_cache_read(codes, scales, fmt, slots.cuda(), out)
    v, s = decoded(codes, scales, fmt)
    ok = ((slots >= 0) & (slots < n)).numpy()
    at = np.where(ok, slots.numpy(), 0)
    f32 = (v[at].astype(np.float32) * s[at].astype(np.float32))
    f32[~ok] = 0
    assert torch.equal(out.cpu(), torch.from_numpy(f32).to(dt))
    # as stored
    oc, os_ = storage(rows, heads, D, fmt)
    K.indexer_cache_read(codes, scales, fmt, slots.cuda(), oc, os_)
    wc, ws = codes.cpu()[at], scales.cpu()[at]
    wc[~ok], ws[~ok] = 0, (127 if fmt == FP4 else 1.0)
    assert torch.equal(oc.cpu(), wc) and torch.equal(os_.cpu(), ws)


@pytest.mark.gpu
def test_strided_input_and_whole_batch_without_slots():
    g = torch.Generator().manual_seed(8)
    wide = torch.randn((30, 6, 200), generator=g).to(torch.bfloat16).cuda()
    for lo in (8, 3):                                  # aligned and unaligned rows
        x = wide[:, ::2, lo:lo + 128]
        for fmt in (FP8, FP4):
            a, b = storage(30, 3, 128, fmt), storage(30, 3, 128, fmt)
            K.indexer_cache_write(x, *a, fmt)
            K.indexer_cache_write(x.contiguous(), *b, fmt)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    codes, scales = storage(4, 1, 64, FP8)
    K.indexer_cache_write(torch.empty((0, 1, 64), device="cuda"), codes, scales, FP8)
    K.indexer_cache_read(codes, scales, FP8, torch.empty(0, dtype=torch.int32, device="cuda"),
                         torch.empty((0, 1, 64), device="cuda"))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Slots whose byte offsets pass 2^31 and 2^32."""
    n, D = (1 << 25) + 64, 128                         # 4 GiB of codes
    codes = torch.empty((n, 1, D), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n, 1), device="cuda")
    slots = torch.tensor([0, (1 << 24) + 3, n - 1, 1 << 25], dtype=torch.int32).cuda()
    codes[slots.long()] = 0
    x = torch.randn((4, 1, D), generator=torch.Generator().manual_seed(9)).cuda()
    K.indexer_cache_write(x, codes, scales, FP8, slots=slots)
    small = storage(4, 1, D, FP8)
    K.indexer_cache_write(x, *small, FP8)
    assert torch.equal(codes[slots.long()], small[0])
    assert torch.equal(scales[slots.long()], small[1])
    a, b = (torch.empty((4, 1, D), device="cuda") for _ in range(2))
    K.indexer_cache_read(codes, scales, FP8, slots, a)
    K.indexer_cache_read(*small, FP8, None, b)
    assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [1, 16, 48])
def test_page_slots(page):
    g = torch.Generator().manual_seed(page)
    lens = [100, 0, 1, 333]
    cu_k = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    cu_q = np.arange(5, dtype=np.int32)
    plan = K.indexer_plan(cu_q, cu_k, np.array(lens, np.int32), 32, 128, 8)
    ld = -(-max(lens) // page) + 2
    table = torch.randint(0, 5000, (4, ld), generator=g, dtype=torch.int32)
    table[3, 0] = -1                                   # unmapped
    table[0, 0] = 2 ** 31 - 1 if page > 1 else 7       # a slot past int32
    got = K.indexer_page_slots(plan, table.cuda(), page).cpu().numpy()
    want = []
    for r, n in enumerate(lens):
        for j in range(n):
            pg = int(table[r, j // page])
            s = pg * page + j % page
            want.append(s if pg >= 0 and s <= 2 ** 31 - 1 else -1)
    assert got.tolist() == want


@pytest.mark.gpu
def test_written_operands_feed_the_indexer():
    """Keys written to a paged cache and packed back, queries quantised by the same call:
    the indexer's logits are those of the formula on the decoded operands."""
    T, L, H, D, page = 16, 300, 32, 128, 16
    g = torch.Generator().manual_seed(10)
    rope = K.indexer_rope_create(D, 64)
    kf = torch.randn((L, 1, D), generator=g).to(torch.bfloat16).cuda()
    qf = torch.randn((T, H, D), generator=g).to(torch.bfloat16).cuda()
    w = (torch.rand((T, H), generator=g) / H ** 0.5).cuda()
    pages = -(-L // page)
    table = torch.randperm(pages, generator=g).to(torch.int32)[None].cuda()
    clen = torch.arange(L - T + 1, L + 1, dtype=torch.int32)
    plan = K.indexer_plan(np.array([0, T], np.int32), np.array([0, L], np.int32), clen, H, D, 8)
    slots = K.indexer_page_slots(plan, table, page)
    pool, pool_s = storage(pages * page, 1, D, FP8)
    pos = torch.arange(L, dtype=torch.int32).cuda()
    K.indexer_cache_write(kf, pool, pool_s, FP8, rope=rope, positions=pos, slots=slots)
    k, ks = storage(L, 1, D, FP8)
    K.indexer_cache_read(pool, pool_s, FP8, slots, k, ks)
    q, qs = storage(T, H, D, FP8)
    K.indexer_cache_write(qf, q, qs, FP8, rope=rope, positions=pos[L - T:].contiguous())
    logits = torch.empty((T, L), device="cuda")
    ws = torch.empty(max(plan.workspace_bytes, 256), dtype=torch.uint8, device="cuda")
    K.indexer_logits(plan, q, qs, w, k, ks, clen.cuda(), logits, ws)
    assert K.indexer_status(plan, ws) == K.IDX_OK
    qv, qsc = decoded(q, qs, FP8)
    kv, ksc = decoded(k, ks, FP8)
    ref = np.einsum("thd,jd->thj", qv * qsc, (kv * ksc)[:, 0])
    ref = (np.maximum(ref, 0) * w.double().cpu().numpy()[:, :, None]).sum(axis=1)
    got = logits.double().cpu().numpy()
    for t in range(T):
        n = int(clen[t])
        assert np.all(np.abs(got[t, :n] - ref[t, :n]) <= 1e-3 * (1 + np.abs(ref[t, :n])))
