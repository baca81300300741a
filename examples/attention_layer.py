"""The attention half of a decoder layer on quantised weights: Q4_K projections, per-head norm and rotation with the
append to the 4-bit paged cache, attention over it, and the output projection.

    python examples/attention_layer.py

serves two sequences with random weights: a prompt each, in chunks, then single tokens, all sequences in one step.  It
prints the time of each kind of step and compares a token computed alone with the same token computed in a chunk.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from quantised_gguf_weight_gb300 import qk, synth  # noqa: E402


class AttentionLayer:
    """One layer's weights and cache.  w_qkv holds the Q4_K rows of all query heads, key heads and value heads, w_out
    `width` rows of all query heads' channels."""

    def __init__(self, w_qkv, w_out, width, n_q, n_kv, head_dim, n_pages, page_tokens, table, q_norm=None, k_norm=None,
                 window=0):
        self.w_qkv, self.w_out, self.width = w_qkv, w_out, width
        self.n_q, self.n_kv, self.D, self.page_tokens = n_q, n_kv, head_dim, page_tokens
        self.table, self.q_norm, self.k_norm, self.window = table, q_norm, k_norm, window
        self.cache = qk.kv_cache_q4(n_pages, n_kv, page_tokens, head_dim)
        self.workspace = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")      # zeroed once, kept

    def _matmul(self, w, rows, K, x):
        if x.shape[0] <= qk.MAX_BATCH:
            return qk.qmatvec_q4_k(w, 0, rows, K, x)
        return qk.qgemm_q4_k(w, 0, rows, K, x)

    def step(self, x, positions, slots, page_table, lens, q_start=None, max_q=1, max_len=0):
        """x [T][width] fp32: the new tokens of all sequences, sequence b's at rows q_start[b]..q_start[b+1] (None: max_q
        each), stored at `slots`; lens count them."""
        q_rows, kv_rows = self.n_q * self.D, self.n_kv * self.D
        qkv = self._matmul(self.w_qkv, q_rows + 2 * kv_rows, self.width, x)
        q, k, v = qkv.split([q_rows, kv_rows, kv_rows], 1)
        q = qk.kv_append_q4(self.cache, q, k, v, positions, slots, self.table, q_weight=self.q_norm,
                            k_weight=self.k_norm, q_out=q)
        mixed = qk.attn_q4(self.cache, q, page_table, lens, q_start=q_start, max_q=max_q, max_len=max_len,
                           window=self.window, workspace=self.workspace)
        return self._matmul(self.w_out, self.width, q_rows, mixed)


class Pages:
    """Which pages a batch of sequences has, on the host: the arguments of a step."""

    def __init__(self, n_pages, page_tokens, batch, max_len):
        self.free, self.page_tokens = list(range(n_pages)), page_tokens
        self.table = torch.full((batch, -(-max_len // page_tokens)), -1, dtype=torch.int32)
        self.lens = [0] * batch

    def extend(self, new):
        """new[b] more tokens for sequence b: the step's arguments but x."""
        positions, slots, starts = [], [], [0]
        for b, n in enumerate(new):
            for pos in range(self.lens[b], self.lens[b] + n):
                page, at = divmod(pos, self.page_tokens)
                if at == 0:
                    self.table[b, page] = self.free.pop()
                positions.append(pos)
                slots.append(int(self.table[b, page]) * self.page_tokens + at)
            self.lens[b] += n
            starts.append(starts[-1] + n)
        return dict(positions=torch.tensor(positions, dtype=torch.int32).cuda(), slots=torch.tensor(slots).cuda(),
                    page_table=self.table.cuda(), lens=torch.tensor(self.lens, dtype=torch.int32).cuda(),
                    q_start=torch.tensor(starts, dtype=torch.int32).cuda(), max_q=max(new), max_len=max(self.lens))


def random_layer(width=1024, n_q=8, n_kv=2, head_dim=128, n_pages=64, page_tokens=32, max_len=4096, seed=1):
    """A layer with random weights and head norms."""
    rows = (n_q + 2 * n_kv) * head_dim
    w = [torch.from_numpy(synth.weights("q4_k", n, k, seed + i)).cuda()
         for i, (n, k) in enumerate([(rows, width), (width, n_q * head_dim)])]
    g = torch.Generator().manual_seed(seed)
    norms = [(1 + 0.1 * torch.randn(head_dim, generator=g)).cuda() for _ in range(2)]
    table = qk.rope_table(max_len, head_dim, base=500000.0)
    return AttentionLayer(w[0], w[1], width, n_q, n_kv, head_dim, n_pages, page_tokens, table, *norms)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--chunk", type=int, default=128)
    ap.add_argument("--tokens", type=int, default=16)
    args = ap.parse_args()
    layer = random_layer()
    g = torch.Generator().manual_seed(2)
    batch = 2
    length = args.prompt + args.tokens
    x = torch.randn(batch, length, layer.width, generator=g).cuda()
    pages = Pages(layer.cache.shape[0], layer.page_tokens, batch, length)

    def step(n):
        at = pages.lens[0]
        rows = x[:, at:at + n].reshape(batch * n, -1).contiguous()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        arguments = pages.extend([n] * batch)
        begin.record()
        y = layer.step(rows, **arguments)
        end.record()
        end.synchronize()
        return y.reshape(batch, n, -1), begin.elapsed_time(end)

    while pages.lens[0] < args.prompt:
        n = min(args.chunk, args.prompt - pages.lens[0])
        y, ms = step(n)
        print(f"{batch} chunks of {n} tokens to {pages.lens[0]}: {1e3 * ms:.0f} us")
    for _ in range(args.tokens):
        y, ms = step(1)
    print(f"{batch} single tokens at {pages.lens[0]}: {1e3 * ms:.0f} us")
    # the last token again, as the end of one chunk that holds the whole sequence
    pages.free = list(range(layer.cache.shape[0]))
    pages.lens = [0] * batch
    again, _ = step(length)
    off = (again[:, -1] - y[:, -1]).norm() / y[:, -1].norm()
    print(f"the last token in one chunk of {length}: {off:.1e} off (its projections take bf16 inputs, and a key that "
          "they move over a rounding edge is another 4-bit value)")
    assert qk.device_error() == 0


if __name__ == "__main__":
    main()
