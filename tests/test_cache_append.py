"""New keys and values into their caches (indexer_cache_append), against the formulas in 64 bits.

Tolerances: a rotation's angle is off by 3e-7 rad at most and its two products and sum by three
fp32 roundings, so a turned element is off by (3e-7 + 3 * 2^-24) of its pair's length before the one
rounding to the cache's type; e4m3 codes are off by half a step (2^-4 of the value, or 2^-10 of
the scale among the smallest).  Unturned 16-bit elements are copies.
"""
import math

import numpy as np
import pytest
import torch

from sparse_attention_prefill_tcgen05_gb300 import _lib as K

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def plan_of(requests, slots_needed=None):
    """requests: (new rows, keys with them) each."""
    cu_q = np.concatenate([[0], np.cumsum([n for n, _ in requests])]).astype(np.int32)
    cu_k = np.concatenate([[0], np.cumsum([k for _, k in requests])]).astype(np.int32)
    pos = np.concatenate([np.arange(k - n, k) for n, k in requests] or [np.zeros(0)]).astype(np.int32)
    plan = K.indexer_plan(cu_q, cu_k, np.minimum(pos + 1, 1 << 30).astype(np.int32), 32, 128, 8)
    return plan, torch.from_numpy(pos), torch.from_numpy(np.repeat(np.arange(len(requests)),
                                                                  [n for n, _ in requests]))


def turned(x, pos, rot, offset, interleaved, base=10000.0):
    """x turned in 64 bits, and the length of every element's pair (0: not turned)."""
    y, ln = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = a + offset, b + offset
        u = pos.double() * base ** (-2.0 * i / rot)
        c, s = torch.cos(u)[:, None], torch.sin(u)[:, None]
        xa, xb = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = xa * c - xb * s, xa * s + xb * c
        ln[..., a] = ln[..., b] = torch.hypot(xa, xb)
    return y, ln


def compare(got, scale, want, ln, dtype):
    """got, scale: the cache's rows; want: 64-bit values."""
    err = (3e-7 + 3 * 2.0 ** -24) * ln
    if scale is None:
        g = got.double().cpu()
        assert torch.all((g - want).abs() <= err + torch.finfo(dtype).eps / 2 * (want.abs() + err))
        return
    s = scale.double().cpu()
    amax = want.abs().amax(-1)
    worst = err.amax(-1)
    assert torch.all((s - torch.where(amax > 0, amax / 448, 1.0)).abs()
                     <= worst / 448 + 2.0 ** -23 * amax / 448)
    g = got.view(torch.float8_e4m3fn).double().cpu() * s[..., None]
    slack = err + 2.0 ** -22 * want.abs() + worst[..., None] / 448
    assert torch.all((g - want).abs() <= torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * s[..., None])
                     + 2 * slack)


CASES = [
    # requests, heads, D, rot, offset, interleaved, dtype, cache, page
    ([(1, 1)], 1, 64, 64, 0, False, "bf16", "same", 0),
    ([(1, 40), (1, 7), (1, 129)], 8, 128, 64, 0, True, "bf16", "same", 16),
    ([(5, 5), (0, 9), (33, 70)], 2, 128, 128, 0, False, "fp16", "same", 48),
    ([(257, 300)], 3, 96, 48, 48, True, "bf16", "fp8", 1),
    ([(700, 900), (1, 3)], 4, 128, 64, 64, False, "fp32", "fp8", 64),
    ([(90, 90)], 1, 32, 32, 0, True, "fp16", "fp8", 0),
    ([(1500, 1501)], 1, 32, 0, 0, False, "bf16", "same", 64),
    ([(40, 64)], 2, 64, 20, 6, False, "bf16", "fp8", 8),         # parts of units
    ([(40, 64)], 2, 80, 20, 6, True, "fp32", "bf16", 8),
    ([(17, 30)], 5, 7, 6, 1, False, "fp16", "same", 5),          # odd head size
    ([(64, 64)], 2, 72, 64, 0, True, "fp32", "fp16", 64),        # eight elements left over
    ([(3, 40)], 2, 8, 0, 0, True, "bf16", "same", 4),
    ([(3, 40)], 300, 256, 256, 0, False, "bf16", "fp8", 4),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("layout", ["packed", "strided"])
def test_rows_and_the_rest_of_the_cache(case, layout):
    requests, H, D, rot, off, inter, dt, kv, page = CASES[case]
    g = torch.Generator().manual_seed(case)
    plan, pos, req = plan_of(requests)
    T = pos.numel()
    fp8 = kv == "fp8"
    ct = DT[dt] if kv == "same" else DT.get(kv)
    if page:
        per = -(-max(k for _, k in requests) // page)
        table = torch.randperm(len(requests) * per + 3, generator=g)[:len(requests) * per].int().view(-1, per)
        n = (len(requests) * per + 3) * page
        at = table[req, pos.long() // page].long() * page + pos.long() % page
    else:
        table, n = None, sum(k for _, k in requests) + 3
        at = torch.tensor(np.concatenate([[0], np.cumsum([k for _, k in requests])]))[req] + pos.long()
    x = (torch.randn(T, 2, H, D + (24 if layout == "strided" else 0), generator=g)).to(DT[dt])
    k, v = x[:, 0, :, :D], x[:, 1, :, :D]                        # halves of one tensor
    if fp8:
        old = torch.randint(0, 127, (n, 2, H, D + (8 if layout == "strided" else 0)), generator=g).byte()
        scales = [torch.rand(n, H, generator=g) for _ in range(2)]
    else:
        old = torch.randn(n, 2, H, D + (8 if layout == "strided" else 0), generator=g).to(ct)
        scales = [None, None]
    dev = old.cuda()
    dsc = [None if s is None else s.cuda() for s in scales]
    xd = x.cuda()
    rope = K.indexer_rope_create(D, rot, rot_offset=off, layout=K.IDX_ROPE_INTERLEAVED if inter
                                 else K.IDX_ROPE_HALF) if rot else None
    K.indexer_cache_append(plan, xd[:, 0, :, :D], xd[:, 1, :, :D], dev[:, 0, :, :D], dev[:, 1, :, :D],
                           pos.cuda(), rope=rope, page_table=None if table is None else table.cuda(),
                           page_size=page, k_scale=dsc[0], v_scale=dsc[1])
    got = dev.cpu()
    rest = torch.ones(n, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(got[rest].view(torch.uint8), old[rest].view(torch.uint8))
    assert torch.equal(got[..., D:].view(torch.uint8), old[..., D:].view(torch.uint8))
    for i, y in enumerate((k, v)):
        want, ln = turned(y, pos, rot if i == 0 else 0, off, inter)
        s = None
        if fp8:
            s = dsc[i].cpu()
            assert torch.equal(s[rest], scales[i][rest])
            s = s[at]
        compare(got[at][:, i, :, :D], s, want, ln, ct)
        if not fp8 and i == 1:
            assert torch.equal(got[at][:, 1, :, :D], v.to(ct))


@pytest.mark.gpu
@pytest.mark.parametrize("D,rot", [(128, 64), (64, 20)])
def test_codes_are_the_cache_writes(D, rot):
    """The same codes and scales as indexer_cache_write's, NaN, infinities and zero rows too."""
    T, H, n = 200, 3, 333
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, H, D, generator=g) * torch.exp2(torch.randint(-30, 30, (T, H, 1), generator=g).float())
    x[3] = 0
    x[4, 1, 5] = math.nan
    x[5, 0, 7] = math.inf
    x[6, 2] = -math.inf
    x = x.cuda()
    slots = torch.randperm(n, generator=g)[:T].int()
    slots[7], slots[8] = -1, n
    slots, pos = slots.cuda(), torch.arange(T, dtype=torch.int32).cuda() * 1001
    rope = K.indexer_rope_create(D, rot)
    kc, vc, kc2, vc2 = (torch.full((n, H, D), 7, dtype=torch.uint8, device="cuda") for _ in range(4))
    ks, vs, ks2, vs2 = (torch.full((n, H), 5.0, device="cuda") for _ in range(4))
    K.indexer_cache_append(None, x, x, kc, vc, pos, rope=rope, slots=slots, k_scale=ks, v_scale=vs)
    K.indexer_cache_write(x, kc2, ks2, rope=rope, positions=pos, slots=slots)
    K.indexer_cache_write(x, vc2, vs2, slots=slots)
    for a, b in ((kc, kc2), (vc, vc2), (ks, ks2), (vs, vs2)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_rows_without_a_place_are_skipped():
    plan, pos, req = plan_of([(6, 20), (4, 40)])
    table = torch.tensor([[0, 1, -1], [4, 99, 1 << 30]], dtype=torch.int32)   # pages of 16
    pos = torch.tensor([0, 15, 16, 20, -1, -2 ** 31, 17, 39, 40, 2 ** 31 - 1], dtype=torch.int32)
    # request 0: 0 -> slot 0, 15 -> 15, 16 -> 16, 20: no key of it; request 1: unmapped or far pages
    k = torch.randn(10, 2, 64).bfloat16()
    kc, vc = (torch.zeros(6 * 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    K.indexer_cache_append(plan, k.cuda(), k.cuda(), kc, vc, pos.cuda(), page_table=table.cuda(),
                           page_size=16)
    want = torch.zeros(6 * 16, 2, 64, dtype=torch.bfloat16)
    want[[0, 15, 16]] = k[:3]
    assert torch.equal(kc.cpu(), want) and torch.equal(vc.cpu(), want)


@pytest.mark.gpu
def test_far_slots():
    """Slots whose elements are past 2^31 from the cache's start."""
    n, H, D = 9_000_000, 2, 128
    kc = torch.zeros(n, H, D, dtype=torch.uint8, device="cuda")
    vc = torch.zeros(n, H, D, dtype=torch.uint8, device="cuda")
    ks, vs = (torch.zeros(n, H, device="cuda") for _ in range(2))
    slots = torch.tensor([n - 1, 8_400_000, 5], dtype=torch.int32, device="cuda")
    x = torch.ones(3, H, D, device="cuda", dtype=torch.bfloat16)
    K.indexer_cache_append(None, x, 2 * x, kc, vc, None, slots=slots, k_scale=ks, v_scale=vs)
    at = slots.long()
    for c, s, want in ((kc, ks, 1.0), (vc, vs, 2.0)):
        y = c[at].view(torch.float8_e4m3fn).float() * s[at][..., None]
        assert torch.allclose(y, torch.full_like(y, want), rtol=2.0 ** -20)
        assert int(torch.count_nonzero(s)) == 3 * H


@pytest.mark.gpu
def test_captured_and_replayed_with_other_positions():
    plan, pos, req = plan_of([(1, 64), (1, 64)])
    k, v = (torch.randn(2, 2, 64, device="cuda").bfloat16() for _ in range(2))
    kc, vc = (torch.zeros(128, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    p = torch.tensor([3, 5], dtype=torch.int32, device="cuda")
    rope = K.indexer_rope_create(64, 32)
    table = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda")

    def call(kc, vc):
        K.indexer_cache_append(plan, k, v, kc, vc, p, rope=rope, page_table=table, page_size=64)
    call(kc, vc)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(kc, vc)
    p += 9
    k.mul_(2)
    graph.replay()
    want = torch.zeros_like(kc), torch.zeros_like(vc)
    k.div_(2)
    p -= 9
    call(*want)
    k.mul_(2)
    p += 9
    call(*want)
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


def test_refusals():
    plan, pos, _ = plan_of([(4, 9)])
    rope = K.indexer_rope_create(64, 64)
    lib = K.lib()
    base = dict(k=1024, v=1024, kc=4096, vc=4096, ks=0, vs=0, pos=1024, slots=0, table=1024, k_row=128,
                k_head=64, v_row=128, v_head=64, kc_slot=128, kc_head=64, vc_slot=128, vc_head=64,
                ld=1, rows=4, heads=2, D=64, dtype=K.IDX_BF16, cache=K.IDX_BF16, n=64, page=16)

    def call(plan=plan, rope=None, **kw):
        io = K._APPEND_IO(*dict(base, **kw).values())
        return lib.indexer_cache_append(plan.handle if plan else None, rope.handle if rope else None,
                                        io, None)
    bad = [dict(k=0), dict(v=0), dict(pos=0), dict(kc=0), dict(vc=0), dict(k=1025), dict(kc=4097),
           dict(pos=1026), dict(table=1026), dict(rows=-1), dict(rows=3), dict(heads=0), dict(heads=1025),
           dict(D=0), dict(D=257), dict(dtype=3), dict(cache=K.IDX_FP32), dict(cache=K.IDX_FP16),
           dict(n=-1), dict(page=-1), dict(table=0), dict(ld=0), dict(k_row=-1), dict(kc_slot=-1),
           dict(kc_slot=63), dict(vc_head=63), dict(cache=K.IDX_CODES), dict(plan=None),
           dict(cache=K.IDX_CODES, ks=1024, vs=1026), dict(cache=K.IDX_CODES, ks=1024, vs=1024, kc=4100),
           dict(cache=K.IDX_CODES, ks=1024, vs=1024, kc_slot=129),
           dict(cache=K.IDX_CODES, ks=1024, vs=1024, D=40, k_head=40, kc_head=64),
           dict(rope=K.indexer_rope_create(128, 64)), dict(plan=None, slots=1024, pos=0, rope=rope)]
    for kw in bad:
        assert call(**kw) == K.IDX_ERR_INVALID_ARG, kw
    assert lib.indexer_cache_append(plan.handle, None, None, None) == K.IDX_ERR_INVALID_ARG
    if not torch.cuda.is_available():
        assert call() == K.IDX_ERR_UNSUPPORTED                  # nothing wrong but the device


def test_binding_refusals():
    plan, pos, _ = plan_of([(4, 9)])
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                             # not on a GPU
        K.indexer_cache_append(plan, x, x, x, x, pos)
