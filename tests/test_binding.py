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
