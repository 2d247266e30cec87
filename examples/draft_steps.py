#!/usr/bin/env python3
"""Serving with drafted tokens on one GPU: what each step works on is decided there too.

    moe_kv_pages -> projections -> moe_kv_append -> moe_kv_attention -> moe_gate ->
    moe_route -> moe_ffn -> head -> moe_verify_drafts -> drafts for the next step

A ragged batch of prompts goes through one decoder layer, then steps of one standing
token and a few drafts for each sequence follow as a captured CUDA graph: rejected
drafts leave the cache, pages come from a pool and go back to it, and the host only
replays.  Lengths and the pool's count change places between two buffers from step to
step, so the graph holds two steps.

    python examples/draft_steps.py [--steps 16] [--prompts 300,77,1200] [--drafts 3]
"""
import argparse
import math
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]

import fp8_grouped_expert_x128_gb300 as moe  # noqa: E402
from decoder_layer import Layer, normed  # noqa: E402


class Server(Layer):
    """The layer with a token embedding (also the head's weights), a draft model that is the head without
    the layer, and the pool of its cache's pages."""

    def __init__(self, batch, max_len, drafts, steps, vocab=512, seed=0, **sizes):
        super().__init__(batch, max_len, seed=seed, **sizes)
        g = torch.Generator(device="cuda").manual_seed(seed + 100)
        self.batch, self.drafts, self.vocab, self.page = batch, drafts, vocab, self.k.shape[2]
        self.embedding = (torch.randn((vocab, self.hidden), generator=g, device="cuda") * 0.3).bfloat16()
        self.gate = self.router.t().contiguous()
        i32 = {"dtype": torch.int32, "device": "cuda"}
        self.bias = 0.05 * torch.randn(self.experts, generator=g, device="cuda")
        self.free = self.table.flatten().clone()                  # every page is free at first
        self.table = torch.full_like(self.table, -1)
        self.lengths = [torch.zeros(batch, **i32) for _ in range(2)]
        self.counts = [torch.tensor([self.free.numel()], **i32), torch.zeros(1, **i32)]
        self.keep = torch.zeros(batch, **i32)
        self.accepted = torch.zeros(batch, **i32)
        self.emitted = torch.full((batch, drafts + 1), -1, **i32)
        self.n_new = torch.full((batch,), drafts + 1, **i32)
        rows = batch * (drafts + 1)
        self.tokens = torch.zeros(rows, **i32)
        self.draft_probs = torch.zeros((rows, vocab), device="cuda")
        # every step's random numbers: tests of drafts, next tokens, drafts
        self.u = torch.rand((steps + 1, 2 * rows + batch), generator=g, device="cuda")
        self.step_no = torch.zeros(1, dtype=torch.int64, device="cuda")

    def head(self, x):
        return torch.softmax(0.04 * (normed(x) @ self.embedding.t()).float(), -1)

    def layer(self, x, cu, max_q, kv_len):
        """x [rows, hidden]; rows behind the last sequence's are routed nowhere."""
        T = x.shape[0]
        q, k, v = (normed(x) @ self.qkv).view(T, -1, self.dim).split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        turned = torch.zeros((T, self.q_heads, self.dim), dtype=x.dtype, device=x.device)
        moe.moe_kv_append(k, v, *self.cache(), cu, kv_len, cos_sin=self.cos_sin, q=q, q_out=turned, err=self.err)
        attended = torch.zeros_like(turned)
        scale = 1.0 / math.sqrt(self.dim)
        if self.kv_ws is None:
            self.kv_ws = moe.alloc_kv_workspace(moe.make_kv_attention_desc(turned, *self.cache(), cu, kv_len, attended, scale))
        moe.moe_kv_attention(turned, *self.cache(), cu, kv_len, attended, self.kv_ws, scale, max_q=max_q, err=self.err)
        x = x + attended.view(T, -1) @ self.out
        z = normed(x)
        logits = moe.moe_gate(z, self.gate, torch.empty((T, self.experts), device="cuda"), err=self.err)
        ids = torch.empty((T, self.top_k), dtype=torch.int32, device="cuda")
        weights = torch.empty((T, self.top_k), device="cuda")
        moe.moe_route(logits, ids, weights, bias=self.bias, n_group=4, topk_group=2, flags=moe.MOE_ROUTE_RENORM, n_tokens=cu[-1:])
        y = torch.empty_like(x)
        d = moe.make_ffn_desc(z, ids, weights, self.w13, self.w13_s, self.w2, self.w2_s, y, 0, self.experts, moe.MOE_LAYOUT_MASKED,
                              max_m=-(-T // 128) * 128, err=self.err)
        if self.ffn_ws is None or self.ffn_ws.numel() < moe.moe_ffn_workspace_size(d):
            self.ffn_ws = moe.alloc_workspace(d)
        moe.moe_ffn(d, self.ffn_ws)
        self.routed = logits, ids, weights
        return x + y

    def step(self, turn, tokens, n_new, max_q, n_draft=None):
        """One step: `turn` says which of the two length buffers holds the lengths before it."""
        before, after = self.lengths[turn], self.lengths[1 - turn]
        T, B, K = tokens.numel(), self.batch, self.drafts
        i32 = {"dtype": torch.int32, "device": "cuda"}
        cu, seqs, positions = torch.empty(B + 1, **i32), torch.empty(T, **i32), torch.empty(T, **i32)
        moe.moe_kv_pages(before, n_new, self.table, self.free, self.counts[turn], self.page, after, cu, self.counts[1 - turn],
                         kv_keep=self.keep, seqs=seqs, positions=positions, err=self.err)
        x = self.layer(self.embedding[tokens.long()], cu, max_q, after)
        probs = self.head(x)
        u = self.u.index_select(0, self.step_no)[0]
        rows = B * (K + 1)
        u_accept = torch.zeros(T, device="cuda") if n_draft is not None else u[:rows]
        moe.moe_verify_drafts(probs, tokens, cu, u_accept, u[rows: rows + B].contiguous(), self.accepted, self.emitted,
                              draft_probs=None if n_draft is not None else self.draft_probs, n_draft=n_draft, kv_len=after, kv_keep=self.keep,
                              err=self.err)
        self.seen = {"probs": probs, "tokens": tokens, "cu": cu, "seqs": seqs, "positions": positions}
        # the next step's rows: the token that stands last, and drafts drawn one after another
        token = self.emitted.gather(1, self.accepted.long()[:, None])[:, 0]
        draws = u[rows + B:].view(B, K + 1)
        grid = self.tokens.view(B, K + 1)
        dist = self.draft_probs.view(B, K + 1, self.vocab)
        grid[:, 0] = token
        for i in range(K):
            q = self.head(self.embedding[token.clamp(min=0).long()])
            dist[:, i] = q
            sums = q.cumsum(-1)
            token = torch.searchsorted(sums, draws[:, i: i + 1] * sums[:, -1:], right=True)[:, 0].clamp(max=self.vocab - 1).to(torch.int32)
            grid[:, i + 1] = token
        self.step_no += 1


def run(prompts, steps, drafts=3, seed=0, graph=True, watch=None, **sizes):
    """Prompts of the given lengths, then an even number of steps; returns the server and, for each
    step (the prompts' first), how many drafts were taken and the tokens that came out."""
    batch = len(prompts)
    server = Server(batch, max(prompts) + (steps + 1) * (drafts + 1), drafts, steps, seed=seed, **sizes)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    history = []

    def note():
        history.append((server.accepted.tolist(), server.emitted.tolist()))
        if watch is not None:
            watch(server)

    prompt = torch.randint(server.vocab, (sum(prompts),), generator=g, device="cuda").to(torch.int32)
    server.step(0, prompt, torch.tensor(prompts, **i32), max(prompts), n_draft=torch.zeros(batch, **i32))
    note()
    if not graph:
        for i in range(steps):
            server.step(1 - i % 2, server.tokens, server.n_new, drafts + 1)
            note()
        return server, history
    # a first pair outside the graph brings kernels and workspaces up, on a copy of what it changes
    kept = {n: getattr(server, n).clone() for n in ("tokens", "draft_probs", "keep", "accepted", "emitted", "step_no", "table", "free", "k", "v", "ks", "vs")}
    pairs = [t.clone() for t in server.lengths + server.counts]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for turn in (1, 0):
            server.step(turn, server.tokens, server.n_new, drafts + 1)
    torch.cuda.current_stream().wait_stream(side)
    for n, t in kept.items():
        getattr(server, n).copy_(t)
    for t, was in zip(server.lengths + server.counts, pairs):
        t.copy_(was)
    graphs = []
    for turn in (1, 0):
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            server.step(turn, server.tokens, server.n_new, drafts + 1)
        graphs.append((captured, server.seen, server.routed))
    for i in range(steps):
        captured, server.seen, server.routed = graphs[i % 2]
        captured.replay()
        note()
    return server, history


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--prompts", default="300,77,1200")
    ap.add_argument("--drafts", type=int, default=3)
    a = ap.parse_args()
    server, history = run([int(n) for n in a.prompts.split(",")], a.steps, a.drafts)
    status, _ = moe.moe_read_device_status(server.err)
    assert status == moe.MOE_OK, moe.moe_status_string(status)
    taken = sum(sum(accepted) for accepted, _ in history[1:])
    print(f"{a.steps} steps of {server.batch} sequences with {a.drafts} drafts each: {taken} of {a.steps * a.drafts * server.batch} drafts taken, "
          f"{taken + a.steps * server.batch} tokens; lengths now {server.keep.tolist()}, {server.counts[1 - a.steps % 2].item()} of "
          f"{server.free.numel()} pages free")


if __name__ == "__main__":
    main()
