"""Serving one MoE decoder layer token by token with the library's kernels.

A step takes one new token of each running sequence through the layer:

    x += attention(rms_norm(x));  x += experts(rms_norm(x))

Keys and values go into a paged cache (PagedKVCache.append, which also rotates
queries and keys), the new tokens attend to their sequences over the cache
(PagedKVCache.attend), the router picks their experts (moe_route_topk) and the
experts run on 4-bit weights (W4Experts).  Norms and projections are plain
torch.  Pages are handed out as sequences grow.

    python examples/decode_step.py [--seqs 8] [--steps 64] [--cache bf16|e4m3] [--graph]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import top_routing_dispatch_gb300 as M  # noqa: E402


def rms_norm(x, eps=1e-6):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + eps)).to(x.dtype)


class DecoderLayer:
    """Weights (random, from `seed`), cache and buffers of one layer for up to
    `seqs` sequences of up to `max_len` tokens."""

    def __init__(self, seqs, max_len, hidden=1024, q_heads=8, kv_heads=2, head_dim=128,
                 intermediate=512, experts=16, top_k=4, group=64, page=16, cache="bf16", seed=0):
        dev, bf = torch.device("cuda"), torch.bfloat16
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
        self.heads, self.dim = (q_heads, kv_heads, kv_heads), head_dim
        width = head_dim * sum(self.heads)
        self.w_qkv = (rand(hidden, width) / hidden ** 0.5).to(bf)
        self.w_out = (rand(q_heads * head_dim, hidden) / (q_heads * head_dim) ** 0.5).to(bf)
        self.w_gate = (rand(hidden, experts) * 0.05).to(bf)
        w13 = (rand(experts, hidden, 2 * intermediate) / hidden ** 0.5).to(bf)
        w2 = (rand(experts, intermediate, hidden) / intermediate ** 0.5).to(bf)
        self.codes = M.quantize_weights_w4(w13, w2, group)  # kept for inspection only
        self.experts = M.W4Experts(*self.codes, K=top_k, max_tokens=seqs)
        self.route = M.make_desc(seqs, hidden, intermediate, experts, top_k, bf, True)

        pages_per_seq = -(-max_len // page)
        pool = seqs * pages_per_seq
        kind = torch.float8_e4m3fn if cache == "e4m3" else bf
        kv = [torch.empty((pool, kv_heads, page, head_dim), device=dev, dtype=kind) for _ in range(2)]
        scale = {}
        if kind is not bf:  # about six deviations of a unit-variance head fit
            scale = {n: torch.full((kv_heads,), 6.0 / 448.0, device=dev) for n in ("k_scale", "v_scale")}
        self.page, self.free = page, list(range(pool))
        self.table = torch.full((seqs, pages_per_seq), -1, dtype=torch.int32, device=dev)
        self.cache = M.PagedKVCache(*kv, self.table, q_heads, rope=M.rope_table(max_len, head_dim),
                                    **scale)
        self.seq_ids = torch.arange(seqs, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device=dev)
        self.host_lens = [0] * seqs
        i32, f32 = torch.int32, torch.float32
        self.idx = torch.empty((seqs, top_k), dtype=i32, device=dev)
        self.weights = torch.empty((seqs, top_k), dtype=f32, device=dev)
        self.logits = torch.empty((seqs, experts), dtype=f32, device=dev)

    def grow(self):
        """The host's part of a step: a page for every sequence that starts one."""
        for s, n in enumerate(self.host_lens):
            if n % self.page == 0:
                self.table[s, n // self.page] = self.free.pop()
            self.host_lens[s] = n + 1

    def step(self, x):
        """One new token of every sequence: x (seqs, hidden) bf16 -> the same."""
        positions = self.lens.clone()
        self.lens += 1
        qkv = rms_norm(x) @ self.w_qkv
        q, k, v = (t.unflatten(1, (-1, self.dim))
                   for t in qkv.split([h * self.dim for h in self.heads], 1))
        q = self.cache.append(q, k, v, self.seq_ids, positions)
        a = self.cache.attend(q, self.lens)
        x = x + a.flatten(1) @ self.w_out
        h = rms_norm(x)
        M.moe_route_topk(self.route, h, self.w_gate, None, self.idx, self.weights, self.logits)
        return x + self.experts(h, self.idx, self.weights)

    def check(self):
        self.cache.check()
        self.experts.check()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--graph", action="store_true", help="capture the step in a CUDA graph")
    a = ap.parse_args()
    layer = DecoderLayer(a.seqs, a.steps + 3, cache=a.cache)
    x = torch.randn((a.seqs, layer.w_qkv.shape[0]), device="cuda").to(torch.bfloat16)
    step = lambda: layer.step(x)  # noqa: E731
    layer.grow()
    y = step()  # loads the kernels
    if a.graph:
        graph = torch.cuda.CUDAGraph()
        layer.grow()
        with torch.cuda.graph(graph):
            y = layer.step(x)
        graph.replay()  # capturing ran nothing
        step = graph.replay
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        layer.grow()
        y = step() if not a.graph else (step(), y)[1]
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    layer.check()
    print(f"{a.seqs} sequences, {a.steps} steps: {1e6 * t / a.steps:.1f} us a step, "
          f"|y| = {float(y.float().norm()):.4f}")


if __name__ == "__main__":
    main()
