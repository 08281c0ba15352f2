"""The operators of a layer's dense branch together: norm, cache append, rotation, selection behind a
window, attention over both and their join, as examples/sparse_layer.py uses them; and in a CUDA graph.

Where everything behind the window is selected, the two branches are disjoint and all of the keys, so
their join is causal attention.  Tolerance of the joined output as that of the layer without a
window (tests/test_layer.py), and 2^-8 of the parts' sizes for the rounding of each part's output.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import sparse_attention_prefill_tcgen05_gb300 as K

HIDDEN, HQ, HKV, D = 256, 8, 2, 64


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_layer.py")
    spec = importlib.util.spec_from_file_location("sparse_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def make(pages, page, e4m3, window, norm):
    layer = example().SparseLayer(HIDDEN, HQ, HKV, D, 160, pages, page, False, e4m3, window=window, norm=norm)
    eye = torch.eye(HIDDEN).bfloat16()
    for i, name in enumerate(("w_iq", "w_ik", "w_iw", "w_q", "w_k", "w_v")):
        w = getattr(layer, name)
        rows = torch.randint(HIDDEN, (w.shape[0],), generator=torch.Generator().manual_seed(i))
        setattr(layer, name, eye[rows].to(w.device))                # picks elements: exact
    return layer


def turned(a):
    n, r = a.shape[0], D // 2
    u = np.arange(n)[:, None, None] * 10000.0 ** (-2.0 * np.arange(r // 2) / r)
    c, s = np.cos(u), np.sin(u)
    o = a.copy()
    o[..., :r // 2] = a[..., :r // 2] * c - a[..., r // 2:r] * s
    o[..., r // 2:r] = a[..., :r // 2] * s + a[..., r // 2:r] * c
    return o


def check(layer, x, out, e4m3, sink):
    """x [positions, hidden] as the projections saw it; out [positions, HQ, D]."""
    q, k, v = ((x @ w.T).double().cpu().numpy().reshape(x.shape[0], -1, D) for w in (layer.w_q, layer.w_k, layer.w_v))
    q, k = turned(q), turned(k)
    uk, scale = 2.0 ** -4 if e4m3 else 2.0 ** -9, D ** -0.5
    for t in range(x.shape[0]):
        for h in range(HQ):
            kk, vv = k[:t + 1, h // (HQ // HKV)], v[:t + 1, h // (HQ // HKV)]
            ak = np.abs(kk) + (np.abs(kk).max(1, keepdims=True) * 2.0 ** -6 if e4m3 else 0)
            av = np.abs(vv) + (np.abs(vv).max(1, keepdims=True) * 2.0 ** -6 if e4m3 else 0)
            a = np.append(scale * (kk @ q[t, h]), sink)
            p = np.exp(a - a.max())
            p = (p / p.sum())[:-1]
            want = p @ vv
            ds = scale * (uk + 2.0 ** -9 + 2.0 ** -16) * (ak @ np.abs(q[t, h])).max()
            tol = (np.expm1(2 * ds) + 2 * 2.0 ** -8 + (uk if e4m3 else 0)) * (p @ av) + 2.0 ** -8 * np.abs(want) \
                + 2.0 ** -20
            err = np.abs(out[t, h].double().numpy() - want)
            assert np.all(err <= tol), (t, h, float((err - tol).max()))


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3,window,sink", [(False, 24, -np.inf), (True, 24, 1.0), (False, 100, 0.5), (False, 1, 2.0)])
def test_selection_behind_a_window_and_the_window_are_causal_attention(e4m3, window, sink):
    n, page = 77, 16
    layer = make(2 * 6, page, e4m3, window, norm=True)
    layer.sink.fill_(sink)
    g = torch.Generator().manual_seed(3)
    table = torch.randperm(2 * 6, generator=g).int().view(2, 6).cuda()
    x, res = (torch.randn(2, n, HIDDEN, generator=g).bfloat16().cuda() for _ in range(2))
    at, out = 0, []
    for m in (40, 33, 1, 1, 1, 1):
        b = layer.plan([(at, m)] * 2)
        layer.forward(x[:, at:at + m].reshape(-1, HIDDEN), b, table, res[:, at:at + m].reshape(-1, HIDDEN))
        for ws, plan in ((b["ws"], b["plan"]), (b["ws_a"], None), (b["ws_w"], None)):
            assert K.indexer_status(plan, ws) == K.IDX_OK
        assert torch.equal(layer.total, (x + res)[:, at:at + m].reshape(-1, HIDDEN))
        out.append(layer.last["out"].view(2, m, HQ, D).cpu())
        at += m
    out = torch.cat(out, 1)
    for r in range(2):
        # the norm alone, call by call the same as row by row
        h = K.indexer_rms_norm(x[r], layer.norm, residual=res[r])
        check(layer, h, out[r], e4m3, sink)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,e4m3", [(1, False), (3, True), (70, False)])
def test_a_captured_step_replays(rows, e4m3):
    """Norm, append, attention over all keys and under a window, and the join, captured once and
    replayed on other inputs, lengths and positions: what the calls give."""
    g = torch.Generator().manual_seed(rows)
    L, Hq, Hkv, page = 1500, 8, 2, 16
    plan = K.indexer_plan(np.arange(rows + 1), np.arange(rows + 1) * L, np.full(rows, L), 32, 128, 8)
    per = -(-L // page)
    table = torch.randperm(rows * per, generator=g).int().view(rows, per).cuda()
    n = rows * per * page
    kv = dict(num_slots=n, page_size=page, kv_format=K.IDX_KV_FP8_E4M3 if e4m3 else K.IDX_KV_DENSE)
    everything = K.indexer_causal_attention_create(plan, Hq, Hkv, 128, **kv)
    near = K.indexer_causal_attention_create(plan, Hq, Hkv, 128, window=200, sinks=3, **kv)
    ws = [torch.empty(a.workspace_bytes, dtype=torch.uint8, device="cuda") for a in (everything, near)]
    rope = K.indexer_rope_create(128, 64)
    hidden = 2 * Hkv * 128
    x, res = (torch.zeros(rows, hidden, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(rows, Hq, 128, dtype=torch.bfloat16, device="cuda")
    pos, lens = (torch.full((rows,), L - 1 + i, dtype=torch.int32, device="cuda") for i in range(2))
    if e4m3:
        kc, vc = (torch.randint(0, 120, (n, Hkv, 128), generator=g, dtype=torch.uint8).cuda() for _ in range(2))
        ks, vs = (torch.full((n, Hkv), 2.0 ** -7, device="cuda") for _ in range(2))
    else:
        kc, vc = (torch.randn(n, Hkv, 128, generator=g).bfloat16().cuda() for _ in range(2))
        ks = vs = None
    h, total, a, b, out = (torch.empty_like(t) for t in (x, x, q, q, q))
    la, lb = (torch.empty(rows, Hq, device="cuda") for _ in range(2))

    def step():
        K.indexer_rms_norm(x, None, residual=res, total=total, out=h)
        new = h.view(rows, 2, Hkv, 128)
        K.indexer_cache_append(plan, new[:, 0], new[:, 1], kc, vc, pos, rope=rope, page_table=table, page_size=page,
                               k_scale=ks, v_scale=vs)
        K.indexer_causal_attention(everything, q, kc, vc, lens, a, ws[0], ks, vs, table, la)
        K.indexer_causal_attention(near, q, kc, vc, lens, b, ws[1], ks, vs, table, lb)
        K.indexer_attention_join([a, b], [la, lb], out)

    step()                                               # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        res.copy_(torch.randn(x.shape, generator=g).bfloat16())
        q.copy_(torch.randn(q.shape, generator=g).bfloat16())
        pos.copy_(torch.randint(0, L, (rows,), generator=g).int())
        lens.copy_(pos + 1)
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (h, total, a, b, out, la, lb)]
        for t in (h, total, a, b, out, la, lb):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(K.indexer_status(None, w) == K.IDX_OK for w in ws)
        assert all(torch.equal(s, t) for s, t in zip(want, (h, total, a, b, out, la, lb)))
        assert torch.isfinite(out.float()).all() and out.float().abs().max() > 0


@pytest.mark.gpu
def test_outputs_made_for_another_stream():
    """Outputs that the calls make are that stream's memory, and follow what is queued there."""
    s = torch.cuda.Stream()
    x = torch.randn(64, 256, device="cuda").bfloat16()
    parts = [torch.randn(64, 4, 64, device="cuda") for _ in range(2)]
    lses = [torch.randn(64, 4, device="cuda") for _ in range(2)]
    want = K.indexer_rms_norm(x), K.indexer_attention_join(parts, lses)
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append((K.indexer_rms_norm(x, stream=s), K.indexer_attention_join(parts, lses, stream=s)))
    s.synchronize()
    assert all(torch.equal(a, b) for pair in got for a, b in zip(pair, want))
