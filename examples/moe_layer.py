"""The expert half of a decoder layer on quantised weights: a Q4_K projection with the requests' low-rank adapters, a
Q8_0 router, the choice of experts, and the experts' products.

    python examples/moe_layer.py

serves requests with random weights, a prompt chunk and then single tokens of all of them, and prints the time of each
kind of step.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from quantised_gguf_weight_gb300 import qk, synth  # noqa: E402


class MoELayer:
    """One layer's weights: Q4_K rows w_in [width][width] with adapters A [n][rank][width], B [n][width][rank], Q8_0 rows
    w_router [experts][width], and the experts' gate, up and down."""

    def __init__(self, w_in, A, B, scales, w_router, gate, up, down, width, hidden, n_experts, top_k, max_tokens):
        self.w_in, self.A, self.B, self.scales, self.w_router = w_in, A, B, scales, w_router
        self.gate, self.up, self.down = gate, up, down
        self.width, self.hidden, self.n_experts, self.top_k = width, hidden, n_experts, top_k
        self.workspace = qk.moe_ffn_workspace(max_tokens, top_k, n_experts, width, hidden)

    def project(self, x, adapters):
        """The adapted projection of rows x [T][width] fp32; adapters [T] int32, -1: none."""
        few = x.shape[0] <= qk.MAX_BATCH
        y = (qk.qmatvec_q4_k if few else qk.qgemm_q4_k)(self.w_in, 0, self.width, self.width, x)
        return qk.lora(x, y, self.A, self.B, adapters, scales=self.scales, out=y)

    def route(self, h):
        few = h.shape[0] <= qk.MAX_BATCH
        logits = (qk.qmatvec_q8_0 if few else qk.qgemm_q8_0)(self.w_router, 0, self.n_experts, self.width, h)
        return (logits, *qk.moe_route(logits, self.top_k))

    def experts(self, h, ids, weights):
        return qk.moe_ffn(h, ids, weights, self.gate, self.up, self.down, self.n_experts, self.hidden, workspace=self.workspace)

    def step(self, x, adapters):
        h = self.project(x, adapters)
        _, ids, weights = self.route(h)
        return h + self.experts(h, ids, weights)


def random_layer(width=1024, hidden=512, n_experts=32, top_k=4, n_adapters=6, rank=16, max_tokens=512, seed=1):
    """A layer with random weights."""
    def rows(fmt, n, k, i):
        return torch.from_numpy(synth.weights(fmt, n, k, seed + i)).cuda()

    g = torch.Generator().manual_seed(seed)
    A = (torch.randn(n_adapters, rank, width, generator=g) * width ** -0.5).half().cuda()
    B = (torch.randn(n_adapters, width, rank, generator=g) * rank ** -0.5).half().cuda()
    gate, up = (qk.ExpertWeights("q4_k", rows("q4_k", n_experts * hidden, width, i)) for i in (1, 2))
    down = qk.ExpertWeights("q6_k", rows("q6_k", n_experts * width, hidden, 3))
    return MoELayer(rows("q4_k", width, width, 0), A, B, (0.5 + torch.rand(n_adapters, generator=g)).cuda(),
                    rows("q8_0", n_experts, width, 4), gate, up, down, width, hidden, n_experts, top_k, max_tokens)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--requests", type=int, default=8)
    args = ap.parse_args()
    layer = random_layer(max_tokens=max(args.prompt, args.requests))
    g = torch.Generator().manual_seed(2)
    for name, T, adapters in (("a prompt of", args.prompt, torch.zeros(args.prompt)),
                              ("single tokens of", args.requests, torch.arange(args.requests) % 7 - 1)):
        x, adapters = torch.randn(T, layer.width, generator=g).cuda(), adapters.int().cuda()
        layer.step(x, adapters)
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        layer.step(x, adapters)
        end.record()
        end.synchronize()
        print(f"{name} {T}: {1e3 * begin.elapsed_time(end):.0f} us")


if __name__ == "__main__":
    main()
