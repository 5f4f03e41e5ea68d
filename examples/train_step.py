"""Training a small stack of MoE blocks with the library's kernels.

Each block adds the experts of its normalised input to the residual stream:

    s += f;  f = experts(norm(s))

(MoEBlock: LayerNorm with the residual added on the way, router, dispatch,
experts, combine).  A step runs the stack, takes the gradient of a squared error
against a fixed target through all blocks, clips the gradients by their global
norm (GradNorm) and updates every parameter (AdamW), optionally as one CUDA
graph.

    python examples/train_step.py [--blocks 2] [--tokens 256] [--steps 20] [--state f32|e4m3] [--graph]
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


class Stack:
    """Blocks with random weights (from `seed`), their optimizer and a target."""

    def __init__(self, blocks, tokens, hidden=256, intermediate=128, experts=8, top_k=2,
                 state="f32", lr=1e-3, max_norm=1.0, seed=0):
        dev, bf = torch.device("cuda"), torch.bfloat16
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
        desc = M.make_desc(tokens, hidden, intermediate, experts, top_k, bf, True)
        self.blocks = []
        for _ in range(blocks):
            norm = M.LayerNorm(torch.ones(hidden, device=dev), torch.zeros(hidden, device=dev), dtype=bf)
            self.blocks.append(M.MoEBlock(
                desc, norm, (rand(hidden, experts) * 0.05).to(bf), torch.zeros(experts, device=dev),
                (rand(experts, hidden, 2 * intermediate) / hidden ** 0.5).to(bf),
                (rand(experts, intermediate, hidden) / intermediate ** 0.5).to(bf)))
        self.params = [p for b in self.blocks for p in b.params]
        self.grads = [p for b in self.blocks for p in b.grads]
        # matrices decay, norms and biases do not
        decay = [0.1 if p.dim() > 1 else 0.0 for p in self.params]
        self.optimizer = M.AdamW(
            self.params, self.grads, lr=lr, weight_decay=decay, masters=True,
            state=torch.float8_e4m3fn if state == "e4m3" else torch.float32)
        self.norm, self.max_norm = M.GradNorm(self.grads), max_norm
        self.x, self.target = rand(tokens, hidden).to(bf), rand(tokens, hidden)

    def forward(self):
        """The residual stream behind the last block, float32."""
        f, s = self.blocks[0].forward(self.x)
        for b in self.blocks[1:]:
            f, s = b.forward(f, s)
        return f.float() + s.float()

    def backward(self, dy):
        """Fills the gradients for dy; returns that of x."""
        df = ds = dy.to(torch.bfloat16)
        for b in reversed(self.blocks):
            df = ds = b.backward(df, ds)
        return df

    def step(self):
        """One update; returns (loss, norm of the gradients), on the device."""
        e = self.forward() - self.target
        self.backward(e / e.numel())
        norm, factor = self.norm(self.max_norm)
        self.optimizer.step(grad_scale=factor)
        return e.square().mean() / 2, norm

    def check(self):
        for b in self.blocks:
            b.check()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--state", choices=("f32", "e4m3"), default="f32")
    ap.add_argument("--graph", action="store_true", help="capture the step in a CUDA graph")
    a = ap.parse_args()
    stack = Stack(a.blocks, a.tokens, state=a.state)
    step = stack.step
    out = step()  # loads the kernels
    if a.graph:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = stack.step()
        step = lambda: (graph.replay(), out)[1]  # noqa: E731
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        out = step()
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    stack.check()
    print(f"{a.blocks} blocks, {a.tokens} tokens, {stack.optimizer.steps} steps: "
          f"{1e6 * t / a.steps:.1f} us a step, loss {float(out[0]):.4f}, "
          f"|gradient| {float(out[1]):.3e}")


if __name__ == "__main__":
    main()
