"""The norm in front of the projections (indexer_rms_norm) and the join of attention parts
(indexer_attention_join), against the formulas in 64 bits.

Tolerances.  Norm: a row's sum of squares is added up in fp32 from at most 64 terms a thread and 10
levels of a tree, each square rounded once: a relative 76 * 2^-24 at most, half of that of its
root; with the root, the quotient and three products 44 * 2^-24 < 2^-18 of y.  Join: weights
exp2((lse - m) log2 e) are off by a relative 2^-22 (1 + |lse - m|), and count for little where that
is large: w (1 + |lse - m|) stays below 2, so the output is off by 2^-20 of the parts' sizes.
Both are rounded once to their type.
"""
import math

import pytest
import torch

from sparse_attention_prefill_tcgen05_gb300 import _lib as K

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def norm_reference(x, r, w, eps):
    h = x.double() + (0 if r is None else r.double())
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    return h, y * (1 if w is None else w.double())


def check_values(got, want, dtype, rel):
    # (fp32's smallest steps, fp16's are 2^-24)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -140
    err = rel * want.abs()
    assert torch.all((got.double().cpu() - want).abs()
                     <= err + torch.finfo(dtype).eps / 2 * (want.abs() + err) + tiny)


def check_codes(codes, scales, want, group):
    y = want.reshape(want.shape[0], -1, group)
    s = scales.double().cpu()
    amax = y.abs().amax(-1)
    assert torch.all((s - torch.where(amax > 0, amax / 448, 1.0)).abs() <= 2.0 ** -17 * amax / 448)
    g = codes.view(torch.float8_e4m3fn).double().cpu().reshape(y.shape) * s[..., None]
    half = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s[..., None])
    assert torch.all((g - y).abs() <= half + 2.0 ** -16 * y.abs() + 2.0 ** -17 * amax[..., None] / 448)


NORMS = [
    # rows, n, dtype, weight, residual, group
    (1, 1, "fp32", "same", False, 0), (1, 8, "bf16", "same", True, 8), (3, 7, "bf16", "fp32", True, 7),
    (5, 64, "fp16", "same", True, 32), (64, 7168, "bf16", "same", True, 128),
    (2, 7168, "bf16", "fp32", False, 256), (9, 1000, "fp16", None, True, 1000),
    (33, 992, "fp32", "same", True, 32), (2, 2049, "bf16", "same", True, 0),
    (2, 16384, "bf16", "same", True, 64), (1, 40960, "fp16", "same", True, 128),
    (1, 65536, "bf16", None, True, 65536), (1, 65535, "fp32", "same", True, 0),
    (2, 8200, "fp32", "same", False, 8200), (700, 96, "bf16", "same", True, 96), (0, 64, "bf16", "same", True, 32),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(NORMS)))
@pytest.mark.parametrize("layout", ["packed", "strided", "unaligned", "in place"])
def test_norm(case, layout):
    rows, n, dt, wt, res, group = NORMS[case]
    dt = DT[dt]
    g = torch.Generator().manual_seed(case)
    pad = {"strided": 40, "unaligned": 9}.get(layout, 0)
    first = 1 if layout == "unaligned" else 0

    def matrix(scale=1.0):
        return (torch.randn(rows, n + pad, generator=g) * scale).to(dt)
    x, r = matrix(), matrix(3.0) if res else None
    w = None if wt is None else (1 + torch.randn(n, generator=g)).to(dt if wt == "same" else torch.float32)
    cut = lambda t: None if t is None else t[:, first:first + n]
    h, y = norm_reference(cut(x), cut(r), w, 1e-5)
    xd, rd = x.cuda(), None if r is None else r.cuda()
    if layout == "in place":
        out, total = xd, rd
    else:
        out, total = torch.full_like(xd, 7), None if r is None else torch.full_like(xd, 7)
    codes = scales = None
    if group:
        codes = torch.empty(rows, n, dtype=torch.uint8, device="cuda")
        scales = torch.empty(rows, n // group, device="cuda")
    K.indexer_rms_norm(cut(xd), None if w is None else w.cuda(), 1e-5, residual=cut(rd), total=cut(total),
                       out=cut(out), codes=codes, scales=scales)
    check_values(cut(out), y, dt, 2.0 ** -18)
    if res:
        check_values(cut(total), h, dt, 2.0 ** -24)
    if group and rows:
        check_codes(codes, scales, y, group)
    if pad and layout != "in place":                            # what lies between rows stays
        assert torch.all(out[:, first + n:] == 7) and torch.all(out[:, :first] == 7)


@pytest.mark.gpu
@pytest.mark.parametrize("unaligned", [0, 1])
def test_norm_of_special_rows(unaligned):
    """Zero rows, NaN, infinities, rows of very different sizes: each row by itself."""
    x = torch.randn(8, 256 + unaligned)[:, unaligned:].contiguous()
    x[0] = 0
    x[1, 3] = math.nan
    x[2, 5] = math.inf
    x[3] *= 1e15
    x[4] *= 1e-15
    big = torch.zeros(8, 256 + unaligned, device="cuda")
    big[:, unaligned:] = x.cuda()
    codes = torch.empty(8, 256, dtype=torch.uint8, device="cuda")
    scales = torch.empty(8, 8, device="cuda")
    out = K.indexer_rms_norm(big[:, unaligned:], None, 1e-6, codes=codes, scales=scales,
                             out=torch.empty(8, 256, device="cuda"))
    _, y = norm_reference(x, None, None, 1e-6)
    ok = [0, 3, 4, 5, 6, 7]
    check_values(out[ok], y[ok], torch.float32, 2.0 ** -18)
    check_codes(codes[ok], scales[ok], y[ok], 32)
    assert torch.isnan(out[1]).all() and torch.isnan(out[2, 5])
    assert torch.all(out[2, :5] == 0)
    v = codes.view(torch.float8_e4m3fn).float()
    assert torch.isfinite(v).all() and torch.isfinite(scales).all()
    assert torch.all(scales[1] == 1) and torch.all(v[0] == 0) and torch.all(v[1] == 0)


@pytest.mark.gpu
def test_norm_makes_its_output():
    x = torch.randn(3, 64, device="cuda").bfloat16()
    out = K.indexer_rms_norm(x)
    _, y = norm_reference(x.cpu(), None, None, 1e-6)
    check_values(out, y, torch.bfloat16, 2.0 ** -18)
    codes, scales = torch.empty(3, 64, dtype=torch.uint8, device="cuda"), torch.empty(3, 2, device="cuda")
    assert K.indexer_rms_norm(x, codes=codes, scales=scales) is None
    check_codes(codes, scales, y, 32)


def join_reference(outs, lses, sink):
    l = [x.double() for x in lses]
    a = l + ([] if sink is None else [sink.double().expand_as(l[0])])
    lse = torch.logsumexp(torch.stack(a), 0)
    o = torch.zeros(outs[0].shape, dtype=torch.float64)
    size = torch.zeros_like(o)
    for x, y in zip(outs, l):
        w = torch.where(torch.isneginf(y), 0.0, torch.exp(y - lse))[..., None]
        x = torch.where(w > 0, x.double(), 0.0)
        o += w * x
        size += w * x.abs()
    return o, lse, size


JOINS = [
    # rows, heads, D, parts, part type, out type, sink
    (1, 1, 64, 1, "bf16", "bf16", True), (5, 3, 128, 2, "fp16", "fp16", False),
    (64, 32, 128, 2, "bf16", "bf16", True), (7, 5, 80, 3, "fp32", "bf16", True),
    (9, 2, 256, 8, "fp32", "fp16", False), (33, 4, 7, 5, "fp32", "fp32", True),
    (3, 300, 8, 4, "bf16", "bf16", False), (0, 4, 64, 2, "bf16", "bf16", True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(JOINS)))
@pytest.mark.parametrize("layout", ["packed", "strided", "unaligned", "in place"])
def test_join(case, layout):
    rows, heads, D, parts, dt, ot, sink = JOINS[case]
    dt, ot = DT[dt], DT[ot]
    if layout == "in place" and dt != ot:
        pytest.skip("types differ")
    g = torch.Generator().manual_seed(case)
    pad, first = {"strided": 24, "unaligned": 5}.get(layout, 0), 1 if layout == "unaligned" else 0
    outs = [(torch.randn(rows, heads, D + pad, generator=g) * 4).to(dt) for _ in range(parts)]
    lses = [torch.randn(rows, heads, generator=g) * 10 for _ in range(parts)]
    for i, l in enumerate(lses):                                # parts without a key
        none = torch.rand(l.shape, generator=g) < 0.3
        l[none] = -math.inf
        outs[i][none] = math.nan
    cut = lambda t: t[..., first:first + D]
    s = torch.randn(heads, generator=g) * 10 if sink else None
    if sink and heads > 1:
        s[0] = -math.inf
    o, lse, size = join_reference([cut(x) for x in outs], lses, s)
    od, ld = [x.cuda() for x in outs], [x.cuda() for x in lses]
    if layout == "in place":
        out, glse = od[-1], ld[-1]
    else:
        out = torch.full((rows, heads, D + pad), 7.0, device="cuda", dtype=ot)
        glse = torch.empty(rows, heads, device="cuda")
    K.indexer_attention_join([cut(x) for x in od], ld, cut(out), lse=glse,
                             sink=None if s is None else s.cuda())
    got, z = cut(out).double().cpu(), glse.double().cpu()
    err = 2.0 ** -20 * size
    tiny = 2.0 ** -25 if ot == torch.float16 else 2.0 ** -140
    assert torch.all((got - o).abs() <= err + torch.finfo(ot).eps / 2 * (o.abs() + err) + tiny)
    empty = torch.isneginf(lse)
    assert torch.equal(torch.isneginf(z), empty) and torch.all(got[empty] == 0)
    assert torch.all((z - lse)[~empty].abs() <= 2.0 ** -20 * (1 + lse[~empty].abs()))
    if pad:
        assert torch.all(out[..., first + D:] == 7) and torch.all(out[..., :first] == 7)


@pytest.mark.gpu
def test_join_of_far_log_sum_exps():
    """Sizes whose exponentials are in no type's range, and one part that outweighs all others."""
    lses = [torch.tensor([[1e30, -1e30, 3e4, -3e4]]).cuda(), torch.tensor([[1e30, -1e30, 0.0, -2.9e4]]).cuda()]
    outs = [torch.full((1, 4, 64), v, device="cuda") for v in (1.0, 3.0)]
    lse = torch.empty(1, 4, device="cuda")
    out = K.indexer_attention_join(outs, lses, lse=lse)
    assert torch.equal(out[0, :, 0].cpu(), torch.tensor([2.0, 2.0, 1.0, 3.0]))
    assert torch.equal(lse.cpu(), torch.tensor([[1e30, -1e30, 3e4, -2.9e4]]))


def test_join_refusals():
    lib = K.lib()
    base = dict(part=1024, part2=0, plse=1024, row=128, head=64, out=1024, lse=0, sink=0, out_row=128,
                out_head=64, parts=1, rows=4, heads=2, D=64, pt=K.IDX_BF16, ot=K.IDX_BF16)

    def call(**kw):
        c = dict(base, **kw)
        io = K._JOIN_IO(c["part"], c["part2"], *[0] * 6, c["plse"], *[0] * 7, c["row"], *[0] * 7, c["head"],
                        *[0] * 7, *list(c.values())[5:])
        return lib.indexer_attention_join(io, None)
    for kw in [dict(part=0), dict(plse=0), dict(part=1025), dict(plse=1026), dict(row=-1), dict(head=-1),
               dict(out=0), dict(out=1025), dict(lse=1026), dict(sink=1026), dict(out_row=63),
               dict(out_head=63), dict(parts=0), dict(parts=9), dict(parts=2), dict(rows=-1), dict(heads=0),
               dict(heads=1025), dict(D=0), dict(D=257), dict(pt=3), dict(ot=K.IDX_FP16), dict(ot=K.IDX_FP32),
               dict(rows=2 ** 31 - 1)]:
        assert call(**kw) == K.IDX_ERR_INVALID_ARG, kw
    assert lib.indexer_attention_join(None, None) == K.IDX_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        K.indexer_attention_join([], [])


def test_norm_refusals():
    lib = K.lib()
    base = dict(x=1024, residual=1024, weight=1024, total=1024, out=1024, codes=1024, scales=1024, x_row=64,
                residual_row=64, total_row=64, out_row=64, rows=2, n=64, group=32, dtype=K.IDX_BF16,
                wt=K.IDX_BF16, eps=1e-6)

    def call(**kw):
        return lib.indexer_rms_norm(K._NORM_IO(*dict(base, **kw).values()), None)
    for kw in [dict(x=0), dict(x=1025), dict(residual=1025), dict(weight=1025), dict(total=1025), dict(out=1025),
               dict(scales=0), dict(scales=1026), dict(residual=0), dict(x_row=-1), dict(total_row=63),
               dict(out_row=63), dict(rows=-1), dict(n=0), dict(n=65537), dict(group=16), dict(group=0),
               dict(group=128), dict(dtype=3), dict(wt=K.IDX_FP16), dict(eps=-1.0), dict(eps=math.nan),
               dict(eps=math.inf), dict(out=0, codes=0, total=0)]:
        assert call(**kw) == K.IDX_ERR_INVALID_ARG, kw
    assert lib.indexer_rms_norm(None, None) == K.IDX_ERR_INVALID_ARG
