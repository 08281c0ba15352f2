"""The operators together, as examples/sparse_layer.py uses them: chunked prefill and decode
over paged caches, against the layer in 64 bits.

With as many selected keys as there are, the layer is causal attention, whatever the indexer
scores: that pins positions, slots, page tables and lengths of all calls.  The projections only
pick elements of the hidden state, so they are exact in any order of summation.

Tolerance of the attention's output, 16-bit caches: q and k are rounded to bf16 once after the
rotation (2^-9 of an element; the rotation itself is below 2^-18), so a score is off by at most
ds = scale (2 x 2^-9 + 2^-16) max_j sum_i |q_i k_i|, the last term with a margin for the fp32
sums; weights by 2 ds relative and 2^-8 from their own rounding; the output by 2^-8 of itself.
e4m3 caches: k and v are off by 2^-4 of an element, or of 2^-6 of the largest of its vector where
the element is smaller, so 2^-4 takes the place of k's 2^-9 and v adds as much.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import sparse_attention_prefill_tcgen05_gb300 as K

HIDDEN, HQ, HKV, D = 256, 8, 2, 64


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "sparse_layer.py")
    spec = importlib.util.spec_from_file_location("sparse_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_imports_without_a_gpu():
    assert example().SparseLayer.forward


def make(topk, pages, page, blocks, e4m3):
    layer = example().SparseLayer(HIDDEN, HQ, HKV, D, topk, pages, page, blocks, e4m3)
    eye = torch.eye(HIDDEN).bfloat16()
    for i, name in enumerate(("w_iq", "w_ik", "w_iw", "w_q", "w_k", "w_v")):
        w = getattr(layer, name)
        rows = torch.randint(HIDDEN, (w.shape[0],), generator=torch.Generator().manual_seed(i))
        setattr(layer, name, eye[rows].to(w.device))
    return layer


def run(layer, x, table, chunks):
    """x [requests, positions, hidden] in chunks; the attention's outputs and selections."""
    out, sel = [], []
    at = 0
    for n in chunks:
        b = layer.plan([(at, n)] * x.shape[0])
        layer.forward(x[:, at:at + n].reshape(-1, HIDDEN), b, table)
        torch.cuda.synchronize()
        assert K.indexer_status(b["plan"], b["ws"]) == K.IDX_OK
        assert K.indexer_status(None, b["ws_a"]) == K.IDX_OK
        out.append(layer.last["out"].view(x.shape[0], n, HQ, D).cpu())
        sel.append(layer.last["sel"].view(x.shape[0], n, -1).cpu())
        at += n
    return torch.cat(out, 1), torch.cat(sel, 1)


def turned(a):
    """Rotated in 64 bits: the first half of the head, halves, base 10,000."""
    n, r = a.shape[0], D // 2
    f = 10000.0 ** (-2.0 * np.arange(r // 2) / r)
    u = np.arange(n)[:, None, None] * f
    c, s = np.cos(u), np.sin(u)
    o = a.copy()
    o[..., :r // 2] = a[..., :r // 2] * c - a[..., r // 2:r] * s
    o[..., r // 2:r] = a[..., :r // 2] * s + a[..., r // 2:r] * c
    return o


def check(layer, x, out, sel, block, e4m3):
    scale = D ** -0.5
    uk = 2.0 ** -4 if e4m3 else 2.0 ** -9
    for r in range(x.shape[0]):
        q, k, v = (turned(p.double().cpu().numpy().reshape(x.shape[1], -1, D)) if turn
                   else p.double().cpu().numpy().reshape(x.shape[1], -1, D)
                   for p, turn in ((x[r] @ layer.w_q.T, True), (x[r] @ layer.w_k.T, True),
                                   (x[r] @ layer.w_v.T, False)))
        for t in range(x.shape[1]):
            js = sorted({e * block + i for e in sel[r, t].tolist() if e >= 0 for i in range(block)
                         if e * block + i <= t})
            for h in range(HQ):
                kk, vv = k[js, h // (HQ // HKV)], v[js, h // (HQ // HKV)]
                ak = np.abs(kk) + (np.abs(kk).max(1, keepdims=True) * 2.0 ** -6 if e4m3 else 0)
                av = np.abs(vv) + (np.abs(vv).max(1, keepdims=True) * 2.0 ** -6 if e4m3 else 0)
                a = scale * (kk @ q[t, h])
                p = np.exp(a - a.max())
                p /= p.sum()
                want = p @ vv
                ds = scale * (uk + 2.0 ** -9 + 2.0 ** -16) * (ak @ np.abs(q[t, h])).max()
                tol = (np.expm1(2 * ds) + 2.0 ** -8 + (uk if e4m3 else 0)) * (p @ av) \
                    + 2.0 ** -8 * np.abs(want) + 2.0 ** -20
                err = np.abs(out[r, t, h].double().numpy() - want)
                assert np.all(err <= tol), (r, t, h, float((err - tol).max()))


@pytest.mark.gpu
@pytest.mark.parametrize("blocks,e4m3", [(False, False), (False, True), (True, False), (True, True)])
def test_layer_is_causal_attention_when_everything_is_selected(blocks, e4m3):
    n, page = 77, 16
    layer = make(80, 3 * 6, page, blocks, e4m3)
    g = torch.Generator().manual_seed(3)
    table = torch.randperm(3 * 6, generator=g).int().view(3, 6).cuda()
    x = torch.randn(3, n, HIDDEN, generator=g).bfloat16().cuda()
    out, sel = run(layer, x, table, [40, 33, 1, 1, 1, 1])
    block = 8 if blocks else 1
    for t in range(n):
        want = set(range(t // block + 1))
        assert all(set(sel[r, t].tolist()) - {-1} == want for r in range(3)), t
    check(layer, x, out, sel, block, e4m3)


@pytest.mark.gpu
@pytest.mark.parametrize("blocks,e4m3", [(False, False), (True, True)])
def test_chunks_and_steps_select_and_attend_as_one_call(blocks, e4m3):
    n, page = 150, 16
    g = torch.Generator().manual_seed(4)
    table = torch.randperm(2 * 10, generator=g).int().view(2, 10).cuda()
    x = torch.randn(2, n, HIDDEN, generator=g).bfloat16().cuda()
    res = []
    for chunks in ([n], [64, 64, 20, 1, 1]):
        layer = make(8, 20, page, blocks, e4m3)
        res.append(run(layer, x, table, chunks))
        check(layer, x, *res[-1], 8 if blocks else 1, e4m3)
    assert torch.equal(res[0][1].sort(-1).values, res[1][1].sort(-1).values)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,e4m3", [(1, False), (24, True), (60, False)])
def test_a_captured_decode_step_replays(rows, e4m3):
    """The operators in a CUDA graph (rows split over a kernel's, four and two blocks), replayed on
    new inputs, give what the calls give."""
    g = torch.Generator().manual_seed(rows)
    L, Hq, Hkv, nsel, page = 2100, 8, 1, 2048, 4
    plan = K.indexer_plan(np.arange(rows + 1), np.arange(rows + 1) * L,
                          np.full(rows, L), 32, 128, 8)
    table = torch.randperm(rows * -(-L // page), generator=g).int().view(rows, -1).cuda()
    n = table.numel() * page
    attn = K.indexer_attention_create(
        plan, Hq, Hkv, 128, nsel, num_slots=n, page_size=page,
        kv_format=K.IDX_KV_FP8_E4M3 if e4m3 else K.IDX_KV_DENSE)
    ws = torch.empty(max(256, attn.workspace_bytes), dtype=torch.uint8, device="cuda")
    rope = K.indexer_rope_create(128, 64)
    x = torch.zeros(rows, Hkv, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(rows, Hq, 128, dtype=torch.bfloat16, device="cuda")
    pos = torch.full((rows,), L - 1, dtype=torch.int32, device="cuda")
    slots = (table[:, (L - 1) // page] * page + (L - 1) % page).contiguous()
    lens = torch.full((rows,), L, dtype=torch.int32, device="cuda")
    codes = torch.randint(0, 120, (n, Hkv, 128), generator=g, dtype=torch.uint8).cuda()
    scales = torch.full((n, Hkv), 2.0 ** -7, device="cuda")
    kv = codes if e4m3 else torch.randn(n, Hkv, 128, generator=g).bfloat16().cuda()
    sel = torch.stack([torch.randperm(L, generator=g)[:nsel] for _ in range(rows)]).int().cuda()
    turned_q, read, out = torch.empty_like(q), torch.empty_like(x), torch.empty_like(q)

    def step():
        K.indexer_rope(rope, q, pos, out=turned_q)
        K.indexer_cache_write(x, codes, scales, rope=rope, positions=pos, slots=slots)
        K.indexer_cache_read(codes, scales, K.IDX_K_FP8_E4M3, slots, read)
        K.indexer_sparse_attention(attn, turned_q, kv, kv, sel, lens, out, ws, page_table=table,
                                   k_scale=scales if e4m3 else None,
                                   v_scale=scales if e4m3 else None)

    step()                                               # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        q.copy_(torch.randn(q.shape, generator=g).bfloat16())
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (turned_q, read, out)]
        for t in (turned_q, read, out):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert K.indexer_status(None, ws) == K.IDX_OK
        assert all(torch.equal(a, b) for a, b in zip(want, (turned_q, read, out)))
        assert torch.isfinite(out.float()).all() and out.float().abs().max() > 0
