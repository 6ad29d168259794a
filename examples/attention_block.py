#!/usr/bin/env python
"""A decoder layer's attention block as a server runs it: W4A16 qkv product,
rotary positions with the cache append, attention over the blocked cache,
W4A16 o product.  A step takes any mix of prompt chunks and single decoded
tokens; its plan (rows, slots, new blocks) is made on the GPU from the request
lengths, once per step, and serves every layer.

  python examples/attention_block.py [--steps 8] [--cache bf16|int8|e4m3]

prefills four ragged prompts in one step, then decodes a token per request and
step from a captured CUDA graph, and prints the time per decode step.  With
--cache int8 or e4m3 keys and values lie in 8 bits: the append quantises them
and the attention reads the codes; the rest of the program is the same.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_int4_group_gb300 as q4  # noqa: E402


class Server:
    """The requests' state on the device: lengths, block table, free blocks,
    and how many requests the last step could not serve."""

    def __init__(self, requests: int, blocks: int, block_size: int, width: int):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.block_size = block_size
        self.length = torch.zeros(requests, **i32)
        self.table = torch.full((requests, width), -1, **i32)
        self.free_blocks = torch.arange(blocks, **i32)
        self.free_count = torch.full((1,), blocks, **i32)
        self.refused = torch.zeros(1, **i32)

    def plan(self, fresh: torch.Tensor, T: int, out: q4.CachePlan | None = None) -> q4.CachePlan:
        """The step's plan; the state moves on to the lengths after the step.
        A request that was not served (kv_len 0: no blocks left, or no room in
        the table or among the T rows) keeps its length, and its blocks, and
        goes on from there in a later step."""
        p = q4.cache_plan(self.length, fresh, self.table, self.free_blocks, self.free_count,
                          self.block_size, T, out=out)
        self.length.copy_(torch.where(p.kv_len > 0, p.kv_len, self.length))
        self.free_count.copy_(p.counts[2:3])
        self.refused.copy_(p.counts[3:4])
        return p


class AttentionBlock:
    def __init__(self, hidden: int, heads: int, kv_heads: int, head_dim: int, max_fresh: int,
                 blocks: int, block_size: int = 16, dtype=torch.bfloat16, seed: int = 0, code=None):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            return q4.QWeight.from_float(torch.randn((n, k), generator=g, device="cuda") * k ** -0.5)

        self.heads, self.max_fresh = heads, max_fresh
        self.qkv = weight((heads + 2 * kv_heads) * head_dim, hidden)
        self.o = weight(hidden, heads * head_dim)
        if code is None:
            self.cache = q4.KVCache.empty(blocks, kv_heads, block_size, head_dim, dtype)
        else:
            self.cache = q4.KVCache8.empty(blocks, kv_heads, block_size, head_dim, code, dtype)
        self.freq, self.factor = q4.rope_frequencies(head_dim)
        self.ws = q4.attention_workspace(max_fresh, heads, kv_heads, head_dim, eight_bit=code is not None)
        self.products_ws: dict[int, torch.Tensor] = {}

    def _product(self, x: torch.Tensor, w: q4.QWeight) -> torch.Tensor:
        M = x.shape[0]
        small = M <= q4.GEMV_MAX_M
        if M not in self.products_ws:  # one per row count, zero-filled once, kept
            size = q4.workspace if small else q4.gemm_workspace
            self.products_ws[M] = max((size(M, v.N, v.K) for v in (self.qkv, self.o)),
                                      key=lambda t: 0 if t is None else t.numel())
        return (q4.gemv if small else q4.gemm)(x, w, ws=self.products_ws[M])

    def __call__(self, x: torch.Tensor, server: Server, plan: q4.CachePlan) -> torch.Tensor:
        """x [T][hidden] -> [T][hidden], every token attending to its request's cache."""
        qkv = self._product(x, self.qkv)
        q = q4.rope_append(qkv, self.cache, plan.position, plan.slot, self.freq, self.heads, factor=self.factor)
        o = q4.attention(q, self.cache, server.table, plan.q_start, plan.kv_len, self.max_fresh, ws=self.ws)
        return self._product(o.flatten(1), self.o)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--cache", choices=["bf16", "int8", "e4m3"], default="bf16")
    args = ap.parse_args()
    steps, code = args.steps, {"bf16": None, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[args.cache]
    hidden, prompts = 8192, [700, 33, 1, 256]
    server = Server(len(prompts), 512, 16, 256)
    block = AttentionBlock(hidden, 64, 8, 128, max(prompts), 512, code=code)
    x = torch.randn(sum(prompts), hidden, device="cuda").bfloat16()
    fresh = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    y = block(x, server, server.plan(fresh, len(x)))

    B = len(prompts)
    block.max_fresh = 1
    x, one = x[:B].clone(), torch.ones(B, dtype=torch.int32, device="cuda")
    out = q4.CachePlan.empty(B, B)
    state = (server.length, server.free_count, server.refused)
    saved = [t.clone() for t in state]
    y = block(x, server, server.plan(one, B, out))  # first use outside the graph: workspaces
    for t, s in zip(state, saved):
        t.copy_(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(x, server, server.plan(one, B, out))
    t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    t0.record()
    for _ in range(steps):
        graph.replay()
    t1.record()
    assert q4.check() == q4.OK and torch.isfinite(y).all()
    print(f"lengths {server.length.tolist()}, free blocks {server.free_count.item()}, "
          f"not served in the last step {server.refused.item()}, "
          f"{t0.elapsed_time(t1) / steps * 1e3:.1f} us per decode step of {B} requests")


if __name__ == "__main__":
    main()
