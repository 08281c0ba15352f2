"""A sparse-attention layer from the library's operators: chunked prefill and decode over
paged caches.

    python examples/sparse_layer.py [--chunk N] [--steps N] [--blocks] [--e4m3] [--window N]

Per call the layer norms its hidden states (with a norm: indexer_rms_norm, which adds the residual),
projects them and then
  1. turns and quantises the indexer's keys into their cache (indexer_cache_write) and appends the
     attention's keys and values to theirs (indexer_cache_append),
  2. turns and quantises the indexer's queries (indexer_cache_write without slots),
  3. packs the prefix out of the pages for the indexer (indexer_page_slots,
     indexer_cache_read),
  4. selects keys (indexer_fused_topk) or 8-key blocks (indexer_candidate_blocks and
     indexer_mask_blocks),
  5. attends over them through the page table (indexer_rope, indexer_sparse_attention),
  6. with a window: selects among the keys behind it only, attends over the window too
     (indexer_causal_attention) and joins the two (indexer_attention_join).
A decode step is the same call with one row per request.  Weights are random.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_prefill_tcgen05_gb300 as K  # noqa: E402

H, DI = 32, 128     # the indexer's heads and head size


class SparseLayer:
    def __init__(self, hidden, Hq, Hkv, D, topk, pages, page=64, blocks=False, e4m3=False,
                 device="cuda", seed=0, window=0, norm=False):
        self.Hq, self.Hkv, self.D, self.topk, self.page = Hq, Hkv, D, topk, page
        self.blocks, self.e4m3, self.window = blocks, e4m3, window
        g = torch.Generator().manual_seed(seed)

        def weight(n):
            return (torch.randn(n, hidden, generator=g) * hidden ** -0.5).to(device, torch.bfloat16)

        self.w_iq, self.w_ik, self.w_iw = weight(H * DI), weight(DI), weight(H)
        self.w_q, self.w_k, self.w_v = weight(Hq * D), weight(Hkv * D), weight(Hkv * D)
        self.w_o = (torch.randn(hidden, Hq * D, generator=g) * (Hq * D) ** -0.5).to(device,
                                                                                 torch.bfloat16)
        self.norm = torch.ones(hidden, dtype=torch.bfloat16, device=device) if norm else None
        # a learned logit of attending to nothing (joins only)
        self.sink = torch.full((Hq,), float("-inf"), device=device)
        self.rope_i = K.indexer_rope_create(DI, 64)
        self.rope = K.indexer_rope_create(D, D // 2)
        n = pages * page
        self.ik = torch.zeros(n, 1, DI, dtype=torch.uint8, device=device)
        self.ik_s = torch.ones(n, 1, device=device)
        if e4m3:
            self.k = torch.zeros(n, Hkv, D, dtype=torch.uint8, device=device)
            self.v = torch.zeros_like(self.k)
            self.k_s = torch.ones(n, Hkv, device=device)
            self.v_s = torch.ones_like(self.k_s)
        else:
            self.k = torch.zeros(n, Hkv, D, dtype=torch.bfloat16, device=device)
            self.v = torch.zeros_like(self.k)
            self.k_s = self.v_s = None

    def plan(self, batch):
        """What every layer of a model shares: plans and workspaces of one batch, a list of
        (positions already cached, new rows) per request, and their device tensors."""
        dev = self.ik.device
        rows = [n for _, n in batch]
        keys = [p + n for p, n in batch]
        cu_q = torch.tensor([0] + rows).cumsum(0).int()
        cu_k = torch.tensor([0] + keys).cumsum(0).int()
        pos = torch.cat([torch.arange(p, p + n) for p, n in batch]).int()
        req = torch.repeat_interleave(torch.arange(len(rows)), torch.tensor(rows))
        lens = (pos + 1 - self.window).clamp_(min=0)         # what the indexer selects from
        p = K.indexer_plan(cu_q, cu_k, lens, H, DI, self.topk,
                           cand_block=8 if self.blocks else 0,
                           cand_topk=self.topk if self.blocks else 0)
        kv = dict(kv_format=K.IDX_KV_FP8_E4M3 if self.e4m3 else K.IDX_KV_DENSE,
                  num_slots=self.ik.shape[0], page_size=self.page)
        a = K.indexer_attention_create(p, self.Hq, self.Hkv, self.D, self.topk,
                                       block=8 if self.blocks else 1, **kv)
        ws = torch.zeros(p.workspace_bytes, dtype=torch.uint8, device=dev)
        ws_a = torch.zeros(max(256, a.workspace_bytes), dtype=torch.uint8, device=dev)
        b = dict(plan=p, attn=a, ws=ws, ws_a=ws_a, rows=int(cu_q[-1]), keys=int(cu_k[-1]),
                 max_keys=max(keys), pos=pos.to(dev), lens=lens.to(dev), req=req.to(dev))
        if self.window:
            w = K.indexer_causal_attention_create(p, self.Hq, self.Hkv, self.D,
                                                  window=self.window, **kv)
            b.update(near=w, seen=(pos + 1).to(dev),
                     ws_w=torch.zeros(max(256, w.workspace_bytes), dtype=torch.uint8, device=dev))
        return b

    def forward(self, x, b, table, residual=None):
        """x [rows, hidden] bf16 (with a norm: what is added to residual before it, the sum into
        self.total); b: plan()'s batch; table int32 [requests, pages]."""
        T, dev = b["rows"], x.device
        pos, plan = b["pos"], b["plan"]
        if self.norm is not None:
            self.total = x if residual is None else torch.empty_like(x)
            x = K.indexer_rms_norm(x, self.norm, residual=residual,
                                   total=None if residual is None else self.total)
        slots = (table[b["req"], (pos // self.page).long()] * self.page + pos % self.page).int()

        # 1. caches
        K.indexer_cache_write((x @ self.w_ik.T).view(T, 1, DI), self.ik, self.ik_s,
                              rope=self.rope_i, positions=pos, slots=slots)
        k, v = (x @ self.w_k.T).view(T, self.Hkv, self.D), (x @ self.w_v.T).view(T, self.Hkv, self.D)
        K.indexer_cache_append(plan, k, v, self.k, self.v, pos, rope=self.rope, page_table=table,
                               page_size=self.page, k_scale=self.k_s, v_scale=self.v_s)

        # 2. the indexer's queries
        iq = torch.empty(T, H, DI, dtype=torch.uint8, device=dev)
        s_q = torch.empty(T, H, device=dev)
        K.indexer_cache_write((x @ self.w_iq.T).view(T, H, DI), iq, s_q, rope=self.rope_i,
                              positions=pos)
        w = (x @ self.w_iw.T).float()

        # 3. the prefix, packed
        packed = torch.empty(b["keys"], 1, DI, dtype=torch.uint8, device=dev)
        packed_s = torch.empty(b["keys"], 1, device=dev)
        K.indexer_cache_read(self.ik, self.ik_s, K.IDX_K_FP8_E4M3,
                             K.indexer_page_slots(plan, table, self.page), packed, packed_s)

        # 4. selection
        sel = torch.empty(T, self.topk, dtype=torch.int32, device=dev)
        if self.blocks:
            ld = (b["max_keys"] + 127) // 128 * 16
            mask = torch.empty(T, ld, dtype=torch.uint8, device=dev)
            K.indexer_candidate_blocks(plan, iq, s_q, w, packed, packed_s, b["lens"], mask, b["ws"])
            count = torch.empty(T, dtype=torch.int32, device=dev)
            K.indexer_mask_blocks(plan, mask, b["lens"], 8, sel, count)
        else:
            K.indexer_fused_topk(plan, iq, s_q, w, packed, packed_s, b["lens"], None, sel, None,
                                 b["ws"])
            count = None

        # 5. attention
        q = (x @ self.w_q.T).view(T, self.Hq, self.D)
        K.indexer_rope(self.rope, q, pos, out=q)
        out = torch.empty_like(q)
        lse = torch.empty(T, self.Hq, device=dev) if self.window else None
        K.indexer_sparse_attention(b["attn"], q, self.k, self.v, sel, b["lens"], out, b["ws_a"],
                                   k_scale=self.k_s, v_scale=self.v_s, sel_count=count,
                                   page_table=table, lse=lse)

        # 6. the window
        if self.window:
            near, near_lse = torch.empty_like(q), torch.empty_like(lse)
            K.indexer_causal_attention(b["near"], q, self.k, self.v, b["seen"], near, b["ws_w"],
                                       k_scale=self.k_s, v_scale=self.v_s, page_table=table,
                                       lse=near_lse)
            K.indexer_attention_join([out, near], [lse, near_lse], out, lse=lse, sink=self.sink)
        self.last = dict(q=q, sel=sel, out=out)
        return out.view(T, -1) @ self.w_o.T


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--prompt", type=int, default=16384, help="tokens of every prompt")
    ap.add_argument("--chunk", type=int, default=2048, help="prefill rows per request and call")
    ap.add_argument("--steps", type=int, default=16, help="decode steps")
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--topk", type=int, default=512, help="keys (or blocks) a row attends over")
    ap.add_argument("--blocks", action="store_true", help="select 8-key blocks, not keys")
    ap.add_argument("--e4m3", action="store_true", help="e4m3 keys and values")
    ap.add_argument("--window", type=int, default=0, help="keys that every row attends over besides")
    a = ap.parse_args()
    page, hidden = 64, 2048
    per = -(-(a.prompt + a.steps) // page)
    layer = SparseLayer(hidden, 32, 2, 128, a.topk, per * a.requests, page, a.blocks, a.e4m3,
                        window=a.window, norm=True)
    table = torch.randperm(per * a.requests).int().view(a.requests, per).cuda()
    g = torch.Generator(device="cuda").manual_seed(1)

    def call(batch):
        b = layer.plan(batch)
        x = torch.randn(b["rows"], hidden, generator=g, device="cuda").bfloat16()
        torch.cuda.synchronize()
        t = time.perf_counter()
        layer.forward(x, b, table)
        torch.cuda.synchronize()
        for ws, plan in ((b["ws"], b["plan"]), (b["ws_a"], None), (b.get("ws_w"), None)):
            if ws is not None and K.indexer_status(plan, ws) != K.IDX_OK:
                raise RuntimeError("a device-side wait gave up")
        return (time.perf_counter() - t) * 1e3

    ms = [call([(p, min(a.chunk, a.prompt - p))] * a.requests) for p in range(0, a.prompt, a.chunk)]
    print(f"prefill: {len(ms)} chunks of {a.requests} x {a.chunk} rows, last {ms[-1]:.2f} ms")
    ms = sorted(call([(a.prompt + i, 1)] * a.requests) for i in range(a.steps))
    if ms:
        print(f"decode: {a.requests} rows a step, median {ms[len(ms) // 2]:.2f} ms")


if __name__ == "__main__":
    main()
