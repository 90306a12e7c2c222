"""Decoding through a mixture of SwiGLU experts, with its experts in bf16 and in 4 bits.

    python examples/serve_moe.py [--tokens 8] [--experts 64] [--top-k 8] [--dim 2048] [--hidden 1408] [--steps 50]

Builds SwiGLUMoE from separate blocks as a checkpoint has them, takes a prompt
through it, captures one decoding step of `tokens` sequences in a HIP graph, and
prints the time of a step and how far the 4-bit experts' output is from the bf16
ones'. Random weights.
"""

import argparse
import os
import sys
from types import SimpleNamespace

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import backward_gate_up_amd as mlp  # noqa: E402


def step_of(block, x):
    """A graph of one step on x, and its output."""
    block(x)  # allocations and first-call work outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(x)
    return graph, y


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("tokens", 8), ("experts", 64), ("top-k", 8), ("dim", 2048), ("hidden", 1408), ("steps", 50)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    torch.manual_seed(0)
    kw = {"device": "cuda", "dtype": torch.bfloat16}
    cfg = SimpleNamespace(hidden_size=a.dim, intermediate_size=a.hidden)
    with torch.no_grad():
        experts = [mlp.SwiGLUMLP(cfg).to(**kw) for _ in range(a.experts)]
        router = torch.nn.Linear(a.dim, a.experts, bias=False).to(**kw)
        block = mlp.SwiGLUMoE.from_experts(router, experts, a.top_k)
        prompt = torch.randn(1, 100, a.dim, **kw)
        weights, ids = mlp.moe_route(prompt[0], router.weight, a.top_k)
        load = torch.bincount(ids.flatten().long(), minlength=a.experts)
        print(f"prompt of {prompt.shape[1]} tokens: {int((load > 0).sum())} of {a.experts} experts used, at most {int(load.max())} times")
        y_prompt = block(prompt)
        x = torch.randn(a.tokens, 1, a.dim, **kw)
        out = {}
        for name in ("bf16", "4 bits"):
            if name == "4 bits":
                block.quantize_(group=128)
            graph, y = step_of(block, x)
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            graph.replay()
            begin.record()
            for _ in range(a.steps):
                graph.replay()
            end.record()
            torch.cuda.synchronize()
            out[name] = y.float().clone()
            print(f"{name:7s} {a.tokens} tokens: {1e3 * begin.elapsed_time(end) / a.steps:.1f} us a step")
        far = (out["4 bits"] - out["bf16"]).norm() / out["bf16"].norm()
        far_prompt = (block(prompt).float() - y_prompt.float()).norm() / y_prompt.float().norm()
        print(f"4 bits against bf16: {far:.3f} of the norm, prompt {far_prompt:.3f}")
    return float(far)


if __name__ == "__main__":
    main()
