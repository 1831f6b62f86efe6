"""An attention layer on the quantised projections and the 8-bit paged cache: prompts, then tokens from a CUDA graph.

    x -> qkv = W_qkv x            (gemm: 4-bit weights)
      -> queries, keys normed and rotated, keys and values into the cache   (kv_append)
      -> attention over the cache                                           (attention)
      -> y = W_o a + x            (gemm, the residual in its epilogue)

Run from the repository's root: python examples/attention_layer.py [--hidden 5120 --heads 40 --kv-heads 8 --dim 128]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import prefill_dequant_gemv_gb300 as q  # noqa: E402
import workloads as wl  # noqa: E402


class AttentionLayer:
    """Random NVFP4 projections, a cache of its own and one set of workspaces a call shape, kept between calls."""

    def __init__(self, hidden, heads, kv_heads, dim, n_seqs, max_len, page=64, seed=0):
        self.heads, self.kv_heads, self.dim, self.max_len = heads, kv_heads, dim, max_len
        rows = (heads + 2 * kv_heads) * dim
        self.w_qkv = q.PackedWeight.from_logical(wl.weight(wl.NVFP4, rows, hidden, seed=seed))
        self.w_o = q.PackedWeight.from_logical(wl.weight(wl.NVFP4, hidden, heads * dim, seed=seed + 1))
        angle = np.arange(max_len)[:, None] * 10000.0 ** (-np.arange(0, dim, 2) / dim)
        table = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
        ones = torch.ones(dim, dtype=torch.bfloat16, device="cuda")
        self.norm_rope = q.NormRope(ones, ones, cos_sin=table)
        per = -(-max_len // page)
        self.cache = q.KVCache.empty(n_seqs * per, kv_heads, page, dim)
        self.pages = torch.randperm(n_seqs * per).int().cuda().view(n_seqs, per)  # a sequence's pages lie anywhere
        self.spaces = {}

    def __call__(self, x, batch):
        n = x.shape[0]
        key = (n, batch.max_new, batch.max_len)
        if key not in self.spaces:
            self.spaces[key] = [q.Workspace(b) for b in (
                q.qg_gemm_workspace_size(self.w_qkv.fmt, self.w_qkv.n, self.w_qkv.k, n), q.qkv_append_workspace_size(),
                q.attention_workspace_size(self.cache, batch, n, self.heads),
                q.qg_gemm_workspace_size(self.w_o.fmt, self.w_o.n, self.w_o.k, n))]
        ws = self.spaces[key]
        qkv = q.gemm(self.w_qkv, x, workspace=ws[0]).view(n, -1, self.dim)
        h, kv = self.heads, self.kv_heads
        queries = q.kv_append(self.cache, batch, qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:], self.norm_rope,
                              out=qkv[:, :h], workspace=ws[1])  # in place
        mixed = q.attention(self.cache, batch, queries, workspace=ws[2])
        return q.gemm(self.w_o, mixed.view(n, -1), residual=x, workspace=ws[3])

    def status(self):
        """The first status other than 0 of any workspace (a bounded wait that gave up, an invalid batch)."""
        return next((s for ws in self.spaces.values() for s in (w.status() for w in ws) if s), 0)


def run(hidden=5120, heads=40, kv_heads=8, dim=128, prompts=(700, 45, 1), steps=24, seed=0):
    """Outputs [sequence][token] of prompts in one call, then `steps` tokens of each sequence, one a step; and the
    largest difference from one call over the whole sequences, over its largest output less the residual."""
    n_seqs, max_len = len(prompts), max(prompts) + steps
    dev = dict(dtype=torch.int32, device="cuda")
    torch.manual_seed(seed)
    x = [torch.randn(p + steps, hidden, device="cuda").bfloat16() for p in prompts]

    def batch(layer, news, lens, max_new, max_len):
        starts = torch.tensor([0, *np.cumsum(news)], **dev)
        return q.KVBatch(starts, torch.tensor(lens, **dev), layer.pages, max_new, max_len)

    layer = AttentionLayer(hidden, heads, kv_heads, dim, n_seqs, max_len, seed=seed)
    prompt = layer(torch.cat([t[:p] for t, p in zip(x, prompts)]), batch(layer, prompts, prompts, max(prompts), max(prompts)))
    outs = [list(t) for t in prompt.split(list(prompts))]

    # one token of every sequence: captured once; a step's input and the lengths change in place
    step = batch(layer, [1] * n_seqs, prompts, 1, max_len)
    inp = torch.zeros(n_seqs, hidden, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # workspaces are made outside the graph; this call's tokens are written again below
        step.lens.add_(1)
        layer(inp, step)
        step.lens.sub_(1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.lens.add_(1)
        out = layer(inp, step)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for i in range(steps):
        inp.copy_(torch.stack([t[p + i] for t, p in zip(x, prompts)]))
        graph.replay()
        for b in range(n_seqs):
            outs[b].append(out[b].clone())
    end.record()
    torch.cuda.synchronize()

    whole = AttentionLayer(hidden, heads, kv_heads, dim, n_seqs, max_len, seed=seed)
    news = [len(t) for t in x]
    ref = whole(torch.cat(x), batch(whole, news, news, max_len, max_len)).float()
    got = torch.cat([torch.stack(o) for o in outs]).float()
    diff = float((got - ref).abs().max() / (ref - torch.cat(x).float()).abs().max())
    if layer.status() or whole.status():
        raise RuntimeError("attention layer: a workspace reports an error")
    return outs, diff, start.elapsed_time(end) / steps * 1e3


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    for name, value in (("hidden", 5120), ("heads", 40), ("kv-heads", 8), ("dim", 128), ("steps", 24)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    outs, diff, us = run(a.hidden, a.heads, a.kv_heads, a.dim, steps=a.steps)
    print(f"{len(outs)} sequences of {', '.join(str(len(o)) for o in outs)} tokens: {us:.1f} us a token step (its copies "
          f"included), largest difference from one call over the whole sequences {diff:.1e} of the layer's largest output")
