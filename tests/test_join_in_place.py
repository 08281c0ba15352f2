"""Joins whose output is one of their parts (indexer_attention_join): with that part's type and strides
each thread reads what it overwrites before it writes; with others it would write what threads of
other vectors have yet to read, so such calls are refused."""
import pytest
import torch

from sparse_attention_prefill_tcgen05_gb300 import _lib as K

BASE = dict(rows=4, heads=2, D=64, row=128, head=64, out_row=128, out_head=64, pt=K.IDX_FP32, ot=K.IDX_FP32)


def call(out, parts=(1024, 65536), **kw):
    c = dict(BASE, **kw)
    n, pad = len(parts), (0,) * (K.IDX_MAX_PARTS - len(parts))
    return K.lib().indexer_attention_join(
        K._JOIN_IO(*parts, *pad, *(4096,) * n, *pad, *(c["row"],) * n, *pad, *(c["head"],) * n, *pad, out, 0, 0,
                   c["out_row"], c["out_head"], n, c["rows"], c["heads"], c["D"], c["pt"], c["ot"]), None)


@pytest.mark.parametrize("out", [1024, 65536])
def test_another_type_or_stride_over_a_part_is_refused(out):
    for kw in [dict(ot=K.IDX_BF16), dict(ot=K.IDX_FP16), dict(ot=K.IDX_BF16, rows=1, heads=1),
               dict(ot=K.IDX_BF16, out_row=256, out_head=128), dict(out_row=256), dict(out_head=256),
               dict(row=256), dict(head=0), dict(out_row=64, out_head=256, row=128, head=64)]:
        assert call(out, **kw) == K.IDX_ERR_INVALID_ARG, kw


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are none of a device's")
def test_what_may_be_in_place():
    """The part's own type and strides (those of a single row or head say nothing), or no part's place."""
    for kw in [dict(), dict(pt=K.IDX_BF16, ot=K.IDX_BF16), dict(rows=1, out_row=64), dict(heads=1, head=7)]:
        assert call(65536, **kw) == K.IDX_ERR_UNSUPPORTED, kw
    assert call(1 << 20, ot=K.IDX_BF16) == K.IDX_ERR_UNSUPPORTED
    assert call(1 << 20, row=0, head=0) == K.IDX_ERR_UNSUPPORTED


@pytest.mark.gpu
def test_through_the_binding():
    a = torch.randn(4, 2, 64, device="cuda")
    kept, lse = a.clone(), torch.zeros(4, 2, device="cuda")
    out = a.view(torch.bfloat16).view(-1).as_strided((4, 2, 64), (128, 64, 1))
    with pytest.raises(K.IndexerError) as e:
        K.indexer_attention_join([torch.ones_like(a), a], [lse, lse], out)
    assert e.value.code == K.IDX_ERR_INVALID_ARG and torch.equal(a, kept)
    K.indexer_attention_join([torch.ones_like(a), a], [lse, lse], a)
    assert torch.allclose(a, (1 + kept) / 2, rtol=0, atol=2.0 ** -20 * float(1 + kept.abs().max()))
