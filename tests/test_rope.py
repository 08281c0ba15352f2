"""Rotary positions (indexer_rope) against the formula in 64 bits.

Tolerance, from the operations: the angle is off by at most 3e-7 rad (one rounding of the
reduced phase to fp32), sine and cosine by 2 ulp, and a rotated element takes three more
roundings, so it is within 1e-6 * m * (|a| + |b|) of m (a cos u -+ b sin u); an output of 16
bits adds half a unit of its last place.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from sparse_attention_prefill_tcgen05_gb300 import _lib as K

HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def frequencies(rot, base=10000.0, factor=1.0, original=0.0, fast=32.0, slow=1.0):
    i = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2.0 * i / rot)
    if factor > 1 and original > 0:
        def pair(n):
            return rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return f / factor * ramp + f * (1 - ramp)
    return f / factor


def rotated(x, pos, rot, offset, interleaved, f, m=1.0, inverse=False):
    """The rotated rows in 64 bits, and |a| + |b| of each rotated element (0 elsewhere)."""
    x = x.astype(np.float64)
    y, mag = x.copy(), np.zeros_like(x)
    u = pos.astype(np.float64)[:, None] * f[None, :]
    c, s = np.cos(u)[:, None, :], np.sin(u)[:, None, :] * (-1 if inverse else 1)
    ia = offset + (np.arange(0, rot, 2) if interleaved else np.arange(rot // 2))
    ib = ia + (1 if interleaved else rot // 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = m * (a * c - b * s), m * (a * s + b * c)
    mag[..., ia] = mag[..., ib] = abs(m) * (np.abs(a) + np.abs(b))
    return y, mag


def check(out, x, pos, rot, offset, interleaved, f, m=1.0, inverse=False):
    want, mag = rotated(x.double().cpu().numpy(), pos.cpu().numpy(), rot, offset, interleaved, f,
                        m, inverse)
    got = out.double().cpu().numpy()
    tol = 1e-6 * mag + (mag > 0) * (HALF_ULP[out.dtype] * np.abs(want) + 2.0 ** -25)
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) - tol))


def test_spec_refusals():
    def bad(**kw):
        a = dict(D=128, rot_dim=64)
        a.update(kw)
        with pytest.raises(K.IndexerError) as e:
            K.indexer_rope_create(**a)
        assert e.value.code == K.IDX_ERR_INVALID_ARG
    K.indexer_rope_create(128, 64)
    K.indexer_rope_create(80, 80, layout=K.IDX_ROPE_INTERLEAVED, factor=8.0, original_len=4096)
    for kw in (dict(rot_dim=63), dict(rot_dim=0), dict(rot_dim=130), dict(D=257, rot_dim=2),
               dict(rot_offset=65), dict(rot_offset=-1), dict(layout=2), dict(base=0.0),
               dict(base=math.nan), dict(factor=0.5), dict(factor=math.inf),
               dict(amplitude=math.nan), dict(factor=2.0, original_len=4096, beta_slow=0.0),
               dict(factor=2.0, original_len=4096, beta_fast=1.0, beta_slow=2.0),
               dict(factor=2.0, original_len=4096, base=1.0)):
        bad(**kw)
    L = K.lib()
    assert L.indexer_rope_create(None, None) == K.IDX_ERR_INVALID_ARG


def test_call_refusals():
    L, A, N = K.lib(), ctypes.c_void_p(0x100000), ctypes.c_void_p(0)
    B = ctypes.c_void_p(0x200000)
    r = K.indexer_rope_create(128, 64)

    def call(rope=r.handle, x=A, dt=K.IDX_BF16, rows=4, heads=2, rs=256, hs=128, pos=A, inv=0,
             out=B, ors=256, ohs=128):
        return L.indexer_rope(rope, x, dt, rows, heads, rs, hs, pos, inv, out, ors, ohs, N)
    for kw in (dict(rope=None), dict(x=N), dict(out=N), dict(pos=N), dict(dt=3), dict(dt=-1),
               dict(rows=-1), dict(heads=0), dict(heads=1025), dict(rs=-1), dict(inv=2),
               dict(ors=127), dict(ohs=64), dict(x=ctypes.c_void_p(0x100001)),
               dict(out=A, ors=512), dict(out=A, rs=512)):
        assert call(**kw) == K.IDX_ERR_INVALID_ARG, kw


CASES = [
    # rows, heads, D, rot, offset, interleaved, dtype
    (64, 32, 128, 128, 0, False, torch.bfloat16),
    (1, 1, 128, 64, 64, True, torch.bfloat16),
    (300, 3, 64, 64, 0, True, torch.float16),
    (77, 5, 80, 48, 16, False, torch.float32),
    (33, 4, 96, 24, 0, False, torch.bfloat16),          # half of 24: no whole units
    (50, 2, 128, 32, 8, True, torch.float32),
    (19, 3, 6, 2, 3, False, torch.float16),
    (41, 1, 256, 256, 0, True, torch.bfloat16),
    (9, 2, 104, 64, 40, False, torch.float16),          # an odd number of vectors left alone
]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,heads,D,rot,offset,inter,dt", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_matches_the_formula(rows, heads, D, rot, offset, inter, dt, inverse):
    g = torch.Generator().manual_seed(rows + D)
    x = torch.randn((rows, heads, D), generator=g).to(dt).cuda()
    pos = torch.randint(0, 487936, (rows,), generator=g, dtype=torch.int32).cuda()
    r = K.indexer_rope_create(D, rot, offset,
                              K.IDX_ROPE_INTERLEAVED if inter else K.IDX_ROPE_HALF)
    out = K.indexer_rope(r, x, pos, inverse=inverse)
    check(out, x, pos, rot, offset, inter, frequencies(rot), inverse=inverse)


@pytest.mark.gpu
@pytest.mark.parametrize("factor,original", [(4.0, 0.0), (16.0, 4096.0), (40.0, 65536.0)])
def test_scaled_for_long_contexts(factor, original):
    x = torch.randn((257, 2, 128), generator=torch.Generator().manual_seed(1)).cuda()
    pos = torch.arange(0, 257 * 1900, 1900, dtype=torch.int32).cuda()
    m = 0.1 * math.log(factor) + 1
    r = K.indexer_rope_create(128, 128, factor=factor, original_len=original, amplitude=m)
    check(K.indexer_rope(r, x, pos), x, pos, 128, 0, False,
          frequencies(128, factor=factor, original=original), m)


@pytest.mark.gpu
def test_extreme_positions():
    """Angles stay exact for the largest and for negative positions."""
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, -487936],
                       dtype=torch.int32).cuda()
    x = torch.randn((7, 2, 64), generator=torch.Generator().manual_seed(2)).cuda()
    out = K.indexer_rope(K.indexer_rope_create(64, 64), x, pos).double().cpu().numpy()
    # 64-bit angles of positions near 2^31 are themselves off by 2^31 * 2^-53 rad: below 3e-7
    want, mag = rotated(x.double().cpu().numpy(), pos.cpu().numpy(), 64, 0, False,
                        frequencies(64))
    assert np.all(np.abs(out - want) <= 2e-6 * mag)
    assert torch.equal(torch.from_numpy(out[0]).float(), x[0].cpu())   # position 0


@pytest.mark.gpu
@pytest.mark.parametrize("rot,offset", [(128, 0), (64, 64), (24, 4)])
def test_strided_in_place_and_other_alignments(rot, offset):
    g = torch.Generator().manual_seed(3)
    r = K.indexer_rope_create(128, rot, offset)
    f = frequencies(rot)
    big = torch.randn((40, 7, 3, 136), generator=g).to(torch.bfloat16).cuda()
    pos = torch.randint(0, 5000, (40,), generator=g, dtype=torch.int32).cuda()
    for part in (big[:, :, 1, :128], big[:, :, 1, 3:131]):      # aligned rows, unaligned rows
        out = K.indexer_rope(r, part, pos)
        check(out, part, pos, rot, offset, False, f)
    heads_first = big[:, :, 0, :128].transpose(0, 1).contiguous().transpose(0, 1)
    before = heads_first.clone()
    rest = big[:, :, 2].clone()
    K.indexer_rope(r, heads_first, pos, out=heads_first)        # in place, heads outermost
    check(heads_first, before, pos, rot, offset, False, f)
    inside = big[:, :, 1, :128]
    before = inside.clone()
    K.indexer_rope(r, inside, pos, out=inside)
    check(inside, before, pos, rot, offset, False, f)
    assert torch.equal(big[:, :, 2], rest)                      # neighbours untouched


@pytest.mark.gpu
def test_inverse_is_the_gradient():
    """d/dx of <g, rope(x)> is the inverse rotation of g: against differences."""
    r = K.indexer_rope_create(32, 16, 8, amplitude=1.25)
    g = torch.Generator().manual_seed(4)
    x, dy = (torch.randn((3, 2, 32), generator=g).cuda() for _ in range(2))
    pos = torch.tensor([3, 40000, 7], dtype=torch.int32).cuda()
    dx = K.indexer_rope(r, dy, pos, inverse=True)
    for e in (0, 8, 13, 15, 16, 23, 24):
        d = torch.zeros_like(x)
        d[:, :, e] = 1.0
        # the rotation is linear: a difference of any size is its derivative
        diff = ((K.indexer_rope(r, x + d, pos) - K.indexer_rope(r, x, pos)) * dy).sum(dim=-1)
        # three fp32 results of magnitude <= 8 cancel: 32 products off by 3e-6 each
        want = dx[:, :, e] if 8 <= e < 24 else dy[:, :, e]
        assert torch.all((diff - want).abs() <= 1e-4)


@pytest.mark.gpu
def test_no_rows_and_another_stream():
    r = K.indexer_rope_create(64, 64)
    empty = torch.empty((0, 4, 64), device="cuda")
    K.indexer_rope(r, empty, torch.empty(0, dtype=torch.int32, device="cuda"))
    x = torch.randn((4096, 8, 64), generator=torch.Generator().manual_seed(5)).cuda()
    pos = torch.arange(4096, dtype=torch.int32).cuda()
    want = K.indexer_rope(r, x, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = K.indexer_rope(r, x, pos)
    b = torch.empty_like(x)
    torch.cuda.current_stream().wait_stream(side)
    K.indexer_rope(r, x, pos, out=b, stream=torch.cuda.current_stream())
    assert torch.equal(a, want) and torch.equal(b, want)


def test_binding_refusals():
    x = torch.zeros((2, 2, 64))
    with pytest.raises(ValueError):                             # not on the device
        K.indexer_rope(K.indexer_rope_create(64, 64), x, torch.zeros(2, dtype=torch.int32))
