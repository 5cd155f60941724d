"""A decoder layer's step on one GPU: the attention side's operators around the
MoE step, with the layer captured into a CUDA graph for single tokens.

    add_norm_x8   residual + attention norm (bf16 for the projection here, MXFP8
                  beside it)
    q, k, v       one bf16 product (cuBLAS)
    kv_append_x8  the new keys and values into the 8-bit paged cache
    attn_x8       the query rows over the cache (a sliding window with sinks)
    o             one bf16 product (cuBLAS), added to the residual
    MoeDecode     the FFN half (its own norm, router, experts)

    python examples/decode_layer.py [--steps N]

draws a small random layer, writes a prompt in chunks of at most 48 rows, then
decodes token by token and prints the time of a step.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mxfp8_moe_decode_gb300 import (MoeDecode, add_norm_x8, attn_x8, attn_x8_workspace,  # noqa: E402
                                    kv_append_x8, kv_cache_x8)
from mxfp8_moe_decode_gb300 import workloads as W  # noqa: E402

PAGE = 64


class DecoderLayer:
    """Weights, cache and buffers of one layer for up to 48 rows a step."""

    def __init__(self, moe: MoeDecode, heads: int, kv_heads: int, head_dim: int, pages: int,
                 window: int = 0, sinks: int = 0, seed: int = 0):
        dev, h = moe.device, moe.hidden
        g = torch.Generator(device=dev).manual_seed(seed)

        def draw(*shape, std):
            return (std * torch.randn(*shape, generator=g, device=dev)).bfloat16()

        self.moe, self.heads, self.kv_heads, self.d = moe, heads, kv_heads, head_dim
        self.window, self.sinks = window, sinks
        self.norm_w = 1 + draw(h, std=0.1)
        self.w_qkv = draw(h, (heads + 2 * kv_heads) * head_dim, std=h ** -0.5)
        self.w_o = draw(heads * head_dim, h, std=(heads * head_dim) ** -0.5)
        self.blocks, self.codes = kv_cache_x8(pages, kv_heads, head_dim, dev)
        self.workspace = attn_x8_workspace(dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def step(self, x, residual, table, had, cu_q=None, max_q=1):
        """One step of x [M, H] (the layer below's output) on the residual
        stream [M, H]: the sequences have `had` tokens in the cache, and their
        new rows are x's (one each, or by cu_q). Returns (the FFN's output, the
        residual stream that it is to be added to, the attention's rows)."""
        m = x.shape[0]
        normed = torch.empty_like(x)
        residual, _, _, _ = add_norm_x8(x, residual, self.norm_w, normed=normed)
        qkv = (normed @ self.w_qkv).view(m, -1, self.d)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        kv_append_x8(self.blocks, self.codes, k, v, table, had, cu_q=cu_q, status=self.status)
        new = 1 if cu_q is None else cu_q.diff()
        attn, _ = attn_x8(q, self.blocks, self.codes, table, had + new, cu_q=cu_q, max_q=max_q,
                          window=self.window, sinks=self.sinks, workspace=self.workspace,
                          status=self.status)
        residual = residual + attn.view(m, -1) @ self.w_o
        return self.moe.step(residual), residual, attn


def small_moe(device="cuda:0") -> MoeDecode:
    """The tiny workload's MoE layer (hidden 1024, 64 experts, top 4)."""
    wl = W.WORKLOADS["tiny_m1"]
    d = wl.dims
    ri = W.router_inputs(wl)
    weights = {k: ri[k].to(device) for k in ("norm_w", "gate_w", "bias")}
    weights.update(W.expert_weights(wl, device=device))
    return MoeDecode(d.hidden, d.experts, d.topk, d.inter, weights, max_tokens=48)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    moe = small_moe(dev)
    seqs, prompt = 4, 100
    per_seq = -(-(prompt + a.steps + 1) // PAGE)
    layer = DecoderLayer(moe, heads=10, kv_heads=2, head_dim=128, pages=seqs * per_seq, window=96, sinks=4)
    table = torch.randperm(seqs * per_seq, device=dev).to(torch.int32).view(seqs, per_seq)
    had = torch.zeros(seqs, dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(1)

    def rows(m):
        return torch.randn(m, moe.hidden, generator=g, device=dev).bfloat16()

    # the prompts, 12 tokens of each sequence at a time (48 rows a step)
    for at in range(0, prompt, 12):
        n = min(12, prompt - at)
        cu = torch.arange(0, seqs * n + 1, n, dtype=torch.int32, device=dev)
        layer.step(rows(seqs * n), rows(seqs * n), table, had, cu_q=cu, max_q=n)
        had += n

    # token by token: the step captured once, then replayed as the cache grows
    x, residual = rows(seqs), rows(seqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x, residual, table, had)  # the same tokens again later: nothing changes
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, res, _ = layer.step(x, residual, table, had)
        had += 1
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        graph.replay()
        x.copy_(out)
        residual.copy_(res)
    end.record()
    torch.cuda.synchronize()
    assert layer.status.item() == 0 and moe.status() == 0
    assert torch.isfinite(out).all()
    print(f"{seqs} sequences, {prompt} + {a.steps} tokens: {1e3 * start.elapsed_time(end) / a.steps:.1f} us a step")


if __name__ == "__main__":
    main()
