"""What the binding refuses before a call: tensors that hold less than the kernels read, and types that
are not what a cache holds."""
import numpy as np
import pytest
import torch

import sparse_attention_prefill_tcgen05_gb300 as K


def _plan(T=4, keys=(100, 37)):
    cu_k = np.concatenate([[0], np.cumsum(keys)]).astype(np.int32)
    cu_q = np.array([0, T // 2, T], np.int32)
    return K.indexer_plan(cu_q, cu_k, np.repeat(np.array(keys, np.int32), T // 2), 32, 128, 8)


def _attention_call(plan, table=None, page=16, dev="cuda", **kw):
    fmt = kw.pop("fmt", K.IDX_KV_DENSE)
    a = K.indexer_attention_create(plan, 8, 1, 128, 16, page_size=page, num_slots=160, kv_format=fmt)
    e = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    args = dict(q=e(4, 8, 128), k=e(160, 1, 128), v=e(160, 1, 128), sel=i(4, 16), lens=i(4), out=e(4, 8, 128))
    args.update(kw)
    ws = torch.zeros(max(a.workspace_bytes, 256), dtype=torch.uint8, device=dev)
    scales = {n: torch.ones((160, 1), device=dev) for n in ("k_scale", "v_scale")} if fmt else {}
    K.indexer_sparse_attention(a, args["q"], args["k"], args["v"], args["sel"], args["lens"], args["out"], ws,
                               page_table=table, **scales)


@pytest.mark.gpu
def test_a_page_table_too_narrow_for_the_longest_request():
    plan = _plan()
    whole = torch.zeros((2, 20), dtype=torch.int32, device="cuda")
    _attention_call(plan, whole[:, :7])                        # 7 pages of 16 for 100 keys
    for table in (whole[:, :6], whole[:, 14:], torch.zeros((2, 6), dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError, match="page_table"):
            _attention_call(plan, table)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_a_mask_too_narrow_for_the_longest_request():
    plan = _plan()
    whole = torch.ones((4, 40), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([100, 100, 37, 37], dtype=torch.int32, device="cuda")
    blocks = torch.empty((4, 16), dtype=torch.int32, device="cuda")
    K.indexer_mask_blocks(plan, whole[:, :13], lens, 8, blocks)  # 13 blocks of 8 for 100 keys
    assert blocks.tolist() == [list(range(13)) + [-1] * 3] * 2 + [list(range(5)) + [-1] * 11] * 2
    for mask in (whole[:, :12], whole[:, 30:]):
        with pytest.raises(ValueError, match="cand_mask"):
            K.indexer_mask_blocks(plan, mask, lens, 8, blocks)
    with pytest.raises(K.IndexerError):                        # no block at all: the library's refusal
        K.indexer_mask_blocks(plan, whole, lens, 0, blocks)


OTHERS = [torch.float8_e5m2, torch.float8_e4m3fnuz, torch.bool]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", OTHERS)
def test_codes_of_another_type(kind):
    plan = _plan()
    table = torch.zeros((2, 7), dtype=torch.int32, device="cuda")
    codes = torch.zeros((160, 1, 128), dtype=torch.uint8, device="cuda")
    for good in (codes, codes.view(torch.float8_e4m3fn), codes.view(torch.int8)):
        _attention_call(plan, table, fmt=K.IDX_KV_FP8_E4M3, k=good, v=good)
    for bad in (dict(k=codes.view(kind), v=codes), dict(k=codes, v=codes.view(kind))):
        with pytest.raises(ValueError):
            _attention_call(plan, table, fmt=K.IDX_KV_FP8_E4M3, **bad)
    x = torch.ones((160, 1, 128), dtype=torch.bfloat16, device="cuda")
    s = torch.empty((160, 1), device="cuda")
    e4, e8 = codes[:, :, :64].contiguous(), torch.empty((160, 1, 4), dtype=torch.uint8, device="cuda")
    K.indexer_cache_write(x, codes.view(torch.float8_e4m3fn), s)
    K.indexer_cache_write(x, e4, e8, K.IDX_K_FP4_E2M1_UE8M0)
    for call in (lambda: K.indexer_cache_write(x, codes.view(kind), s),
                 lambda: K.indexer_cache_write(x, e4.view(kind), e8, K.IDX_K_FP4_E2M1_UE8M0),
                 lambda: K.indexer_cache_write(x, e4, e8.view(kind), K.IDX_K_FP4_E2M1_UE8M0),
                 lambda: K.indexer_cache_write(x, e4.view(torch.float8_e4m3fn), e8,
                                               K.IDX_K_FP4_E2M1_UE8M0),
                 lambda: K.indexer_cache_read(codes.view(kind), s, K.IDX_K_FP8_E4M3, None, x)):
        with pytest.raises(ValueError, match="cache"):
            call()
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_masks_of_truth_values_and_of_another_type():
    plan = _plan()
    lens = torch.tensor([100, 100, 37, 37], dtype=torch.int32, device="cuda")
    mask = torch.arange(52, device="cuda").view(4, 13) % 3 == 0
    a, b = (torch.empty((4, 8), dtype=torch.int32, device="cuda") for _ in "ab")
    K.indexer_mask_blocks(plan, mask, lens, 8, a)
    K.indexer_mask_blocks(plan, mask.to(torch.uint8), lens, 8, b)
    assert torch.equal(a, b)
    # -0.0 is a byte that is not zero
    for kind in (torch.float8_e4m3fn, torch.float8_e5m2):
        with pytest.raises(ValueError, match="cand_mask"):
            K.indexer_mask_blocks(plan, mask.to(torch.uint8).view(kind), lens, 8, a)


@pytest.mark.gpu
def test_a_single_column_of_any_stride():
    """Lists of one entry, tables of one page and masks of one block taken out of wider tensors."""
    cu = np.array([0, 1, 2, 3], np.int32)
    plan = K.indexer_plan(cu, cu * 8, np.full(3, 8, np.int32), 32, 128, 8)
    a = K.indexer_attention_create(plan, 4, 1, 64, 1, block=8, page_size=8, num_slots=24)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((3, 4, 64), generator=g, device="cuda").bfloat16()
    k, v = (torch.randn((24, 1, 64), generator=g, device="cuda").bfloat16() for _ in "kv")
    lens = torch.full((3,), 8, dtype=torch.int32, device="cuda")
    ws = torch.zeros(max(a.workspace_bytes, 256), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[2], [0], [1]], dtype=torch.int32, device="cuda")
    sel = torch.zeros((3, 1), dtype=torch.int32, device="cuda")
    want, got = torch.empty_like(q), torch.empty_like(q)
    K.indexer_sparse_attention(a, q, k, v, sel, lens, want, ws, page_table=table)
    blocks = torch.empty((3, 1), dtype=torch.int32, device="cuda")
    wide = torch.ones((3, 4), dtype=torch.uint8, device="cuda")
    K.indexer_mask_blocks(plan, wide[:, ::2][:, :1], lens, 8, blocks)
    assert torch.equal(blocks, sel)
    wide_sel = torch.zeros((3, 6), dtype=torch.int32, device="cuda")
    wide_sel[:, 1::2] = 99
    wide_table = torch.full((3, 6), 77, dtype=torch.int32, device="cuda")
    wide_table[:, :1] = table
    K.indexer_sparse_attention(a, q, k, v, wide_sel[:, ::2][:, :1], lens, got, ws,
                               page_table=wide_table[:, ::3][:, :1])
    assert torch.equal(got, want)
