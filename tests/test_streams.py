"""Outputs that a call makes for itself on a stream that is not the current one."""
import numpy as np
import pytest
import torch

import sparse_attention_prefill_tcgen05_gb300 as K

pytestmark = pytest.mark.gpu

L, PAGE = 1 << 19, 16


def _plan():
    return K.indexer_plan(np.array([0, 64], np.int32), np.array([0, L], np.int32), np.full(64, L, np.int32),
                          32, 128, 2048)


def _calls():
    pos = torch.arange(2048, dtype=torch.int32, device="cuda")
    x = torch.randn((2048, 4, 128), device="cuda")
    rope = K.indexer_rope_create(128, 64)
    yield x.shape, x.dtype, lambda **kw: K.indexer_rope(rope, x, pos, **kw)
    plan = _plan()
    table = torch.randperm(L // PAGE, device="cuda").to(torch.int32).view(1, -1)
    yield (L,), torch.int32, lambda **kw: K.indexer_page_slots(plan, table, PAGE, **kw)
    raw = torch.randint(0, L, (64, 2048), device="cuda", dtype=torch.int32)
    yield raw.shape, raw.dtype, lambda **kw: K.indexer_page_indices(plan, raw, table, PAGE, **kw)


@pytest.mark.parametrize("which", [0, 1, 2])
def test_a_new_output_is_not_memory_the_current_stream_still_writes(which):
    shape, dtype, call = list(_calls())[which]
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    junk = torch.empty(shape, dtype=dtype, device="cuda")
    at = junk.data_ptr()
    torch.cuda._sleep(20_000_000)                        # the fill comes some 10 ms later
    junk.fill_(7)
    del junk                                             # its memory is the current stream's again
    got = call(stream=side)
    assert got.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(got, want)
