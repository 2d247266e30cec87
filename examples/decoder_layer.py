#!/usr/bin/env python3
"""One decoder layer of MoE serving on one GPU, from the library's operators:

    projections -> moe_kv_append -> moe_kv_attention -> projection -> moe_ffn

A ragged batch of prompts goes through the layer once, then decode steps follow,
one token for each sequence, as one captured CUDA graph that is replayed: the
sequence lengths live on the device and grow there, and nothing is allocated.

    python examples/decoder_layer.py [--steps 16] [--prompts 300,77,1200]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_grouped_expert_x128_gb300 as moe  # noqa: E402


def normed(x):
    """Rows scaled to a mean square of 1."""
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Layer:
    """Random weights of a small layer, its cache, and its workspaces."""

    def __init__(self, batch, max_len, hidden=512, q_heads=8, kv_heads=2, dim=128, page=64, experts=8, inner=256, top_k=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.q_heads, self.kv_heads, self.dim, self.experts, self.top_k = hidden, q_heads, kv_heads, dim, experts, top_k

        def normal(*shape, fan):
            return (torch.randn(shape, generator=g, device="cuda") / math.sqrt(fan)).bfloat16()

        self.qkv = normal(hidden, (q_heads + 2 * kv_heads) * dim, fan=hidden)
        self.out = normal(q_heads * dim, hidden, fan=q_heads * dim)
        self.router = normal(hidden, experts, fan=hidden)
        w13, w2 = normal(experts, 2 * inner, hidden, fan=hidden), normal(experts, hidden, inner, fan=inner)
        self.w13, self.w13_s = torch.empty_like(w13, dtype=torch.uint8), torch.empty((experts, 2 * inner // 128, hidden // 128), device="cuda")
        self.w2, self.w2_s = torch.empty_like(w2, dtype=torch.uint8), torch.empty((experts, hidden // 128, inner // 128), device="cuda")
        moe.moe_quant_weight_fp8(w13, self.w13, self.w13_s)
        moe.moe_quant_weight_fp8(w2, self.w2, self.w2_s)
        angle = torch.arange(max_len, device="cuda")[:, None] * 10000.0 ** (-torch.arange(dim // 2, device="cuda") / (dim // 2))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        # the paged cache: every sequence has its pages from the start
        per = -(-max_len // page)
        self.table = torch.randperm(batch * per, generator=g, device="cuda").to(torch.int32).view(batch, per)
        shape = (batch * per, kv_heads, page, dim)
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.ones(shape[:2], device="cuda") for _ in range(2))
        self.kv_len = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.err = moe.new_error_word()
        self.kv_ws = self.ffn_ws = None

    def cache(self):
        return self.k, self.v, self.ks, self.vs, self.table

    def forward(self, x, cu, max_q):
        """x [tokens, hidden] bf16, rows of sequence b at cu[b] ..; the sequences' lengths already count them."""
        T = x.shape[0]
        rows = (normed(x) @ self.qkv).view(T, -1, self.dim)
        q, k, v = rows.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        turned = torch.empty((T, self.q_heads, self.dim), dtype=x.dtype, device=x.device)
        moe.moe_kv_append(k, v, *self.cache(), cu, self.kv_len, cos_sin=self.cos_sin, q=q, q_out=turned, err=self.err)
        attended = torch.empty_like(turned)
        scale = 1.0 / math.sqrt(self.dim)
        if self.kv_ws is None:
            self.kv_ws = moe.alloc_kv_workspace(moe.make_kv_attention_desc(turned, *self.cache(), cu, self.kv_len, attended, scale))
        moe.moe_kv_attention(turned, *self.cache(), cu, self.kv_len, attended, self.kv_ws, scale, max_q=max_q, err=self.err)
        x = x + attended.view(T, -1) @ self.out
        z = normed(x)
        weight, ids = torch.softmax((z @ self.router).float(), -1).topk(self.top_k)
        weight = weight / weight.sum(-1, keepdim=True)
        y = torch.empty_like(x)
        d = moe.make_ffn_desc(z, ids.to(torch.int32), weight, self.w13, self.w13_s, self.w2, self.w2_s, y, 0, self.experts,
                              moe.MOE_LAYOUT_MASKED, max_m=-(-T // 128) * 128, err=self.err)
        if self.ffn_ws is None or self.ffn_ws.numel() < moe.moe_ffn_workspace_size(d):
            self.ffn_ws = moe.alloc_workspace(d)
        moe.moe_ffn(d, self.ffn_ws)
        self.last = turned, attended
        return x + y


def run(prompts, steps, seed=0):
    """Prompts of the given lengths and `steps` decode steps; returns the layer and each step's output."""
    batch = len(prompts)
    layer = Layer(batch, max(prompts) + steps, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn((sum(prompts), layer.hidden), generator=g, device="cuda").bfloat16()
    cu = torch.tensor([sum(prompts[:b]) for b in range(batch + 1)], dtype=torch.int32, device="cuda")
    layer.kv_len.copy_(cu[1:] - cu[:-1])
    y = layer.forward(x, cu, max(prompts))
    outputs = [y]
    token = y[cu[1:].long() - 1].clone()                     # each sequence goes on from its last token
    ones = torch.arange(batch + 1, dtype=torch.int32, device="cuda")

    def step():
        layer.kv_len.add_(1)
        token.copy_(layer.forward(token, ones, 1))

    if steps:
        start = token.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()                                           # a first step outside the graph brings workspaces and kernels up
        torch.cuda.current_stream().wait_stream(side)
        layer.kv_len.sub_(1)                                 # and is taken back: its token is written again
        token.copy_(start)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for _ in range(steps):
            graph.replay()
            outputs.append(token.clone())
    return layer, outputs


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--prompts", default="300,77,1200")
    a = ap.parse_args()
    layer, outputs = run([int(n) for n in a.prompts.split(",")], a.steps)
    status, _ = moe.moe_read_device_status(layer.err)
    assert status == moe.MOE_OK, moe.moe_status_string(status)
    print(f"{outputs[0].shape[0]} prompt tokens, then {len(outputs) - 1} steps of {layer.kv_len.numel()} tokens; lengths now "
          f"{layer.kv_len.tolist()}; last output rms {outputs[-1].float().square().mean().sqrt().item():.4f}")


if __name__ == "__main__":
    main()
