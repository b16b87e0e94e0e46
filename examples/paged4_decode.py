"""A decode loop over a paged 4-bit cache that is kept to a budget.

The library's calls as one layer of a serving program makes them, for a batch
of sequences: the prompts are appended in one call; the attention weights that
their last queries give decide which tokens stay; then every step appends a
token to each sequence, attends over the cache and adds the step's weights to
its tokens', and when a sequence has outgrown the budget by a slack, the tokens
of the least weight go.

    python examples/paged4_decode.py [--tokens 32768] [--budget 4096] [--steps 128]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import top_block_selection_gb300 as tbs  # noqa: E402


class Layer:
    """Cache, weights and angles of one attention layer of B sequences."""

    def __init__(self, B: int, capacity: int, positions: int, Hq: int, Hkv: int, D: int, block: int = 64,
                 device="cuda", base: float = 10000.0):
        blocks = -(-capacity // block)
        self.Hq, self.Hkv, self.D, self.block = Hq, Hkv, D, block
        self.longest = 0  # tokens of the longest sequence, known on the host
        self.k = torch.empty((B * blocks, Hkv, block, D // 2), dtype=torch.uint8, device=device)
        self.v = torch.empty_like(self.k)
        self.k_scale = torch.empty((B * blocks, Hkv, block), dtype=torch.bfloat16, device=device)
        self.v_scale = torch.empty_like(self.k_scale)
        self.weights = torch.zeros((B * blocks, Hkv, block), device=device)
        self.table = torch.randperm(B * blocks, device=device).to(torch.int32).view(B, blocks)  # pages in any order
        self.lens = torch.zeros(B, dtype=torch.int32, device=device)
        self.offset = torch.zeros(B, dtype=torch.int32, device=device)  # tokens that went
        angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] \
            * base ** (-torch.arange(D // 2, device=device, dtype=torch.float64) / (D // 2))
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def cache(self):
        return self.k, self.v, self.k_scale, self.v_scale, self.table, self.lens

    def append(self, q, k, v):
        """q [B, n, Hq, D], k and v [B, n, Hkv, D] of the next n tokens; returns the rotated q."""
        self.longest += k.shape[1]
        self.lens += k.shape[1]
        return tbs.qsa_kv4_append(k, v, *self.cache(), cos=self.cos, sin=self.sin, offset=self.offset, q=q)

    def attend(self, q, decay: float = 1.0):
        """Attention of the newest rows q [B, n, Hq, D]; their weights are added to the cached tokens'."""
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
        out = tbs.qsa_kv4_attend(q, *self.cache(), lse=lse)
        tbs.qsa_kv4_weights(q, lse, *self.cache(), self.weights, decay=decay)
        return out

    def keep(self, budget: int, sink: int, recent: int):
        """Down to `budget` tokens a sequence and KV head."""
        self.lens = tbs.qsa_kv4_evict(*self.cache(), self.weights, budget, sink, recent, offset=self.offset)
        self.longest = min(self.longest, budget)


def decode(B: int, tokens: int, steps: int, budget: int, slack: int, Hq: int = 32, Hkv: int = 8, D: int = 128,
           block: int = 64, seed: int = 0, sink: int = 4, last: int = 32):
    """Runs the loop on random projections; returns the layer, and the last step's rotated queries and output."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def project(n):
        x = torch.randn((B, n, Hq + 2 * Hkv, D), generator=g, device="cuda").bfloat16()
        return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]

    layer = Layer(B, max(tokens, budget + slack) + 1, tokens + steps, Hq, Hkv, D, block)
    q = layer.append(*project(tokens))
    layer.attend(q[:, -min(last, tokens):], decay=0.0)  # every token's weight begins here
    recent = budget // 4
    layer.keep(budget, sink, recent)
    for _ in range(steps):
        q = layer.append(*project(1))
        out = layer.attend(q)
        if layer.longest >= budget + slack:
            layer.keep(budget, sink, recent)
    return layer, q, out


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--tokens", type=int, default=32768)
    p.add_argument("--budget", type=int, default=4096)
    p.add_argument("--steps", type=int, default=128)
    a = p.parse_args()
    layer, q, _ = decode(a.batch, a.tokens, a.steps, a.budget, slack=64)
    torch.cuda.synchronize()

    def timed(fn, n=50):
        fn()
        start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(n):
            fn()
        stop.record()
        stop.synchronize()
        return start.elapsed_time(stop) / n * 1e3

    print(f"{a.batch} sequences of {a.tokens} tokens kept to {a.budget}: {layer.lens.tolist()} tokens, "
          f"{layer.offset.tolist()} gone; attention and weights of a step {timed(lambda: layer.attend(q)):.1f} us")
    status, bits = tbs.qsa_device_status()
    assert status == 0, (status, bits)


if __name__ == "__main__":
    main()
