"""A decode loop with block selection over a paged 8-bit cache.

The library's calls as one layer of a serving program makes them, for one
sequence: the prompt's keys and values are appended in one call, then every
step appends a token (rotating its query on the way), scores the cache's
blocks against the query's heads, one KV head to a batch of the selection,
selects the best k of each KV head, and attends over them.

    python examples/paged_decode.py [--tokens 131072] [--steps 32] [--k 64]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import top_block_selection_gb300 as tbs  # noqa: E402


class Layer:
    """Cache, block keys and angles of one attention layer of one sequence."""

    def __init__(self, capacity: int, Hq: int, Hkv: int, D: int, block: int = 64, device="cuda", base: float = 10000.0):
        blocks = -(-capacity // block)
        self.Hq, self.Hkv, self.D, self.block, self.tokens = Hq, Hkv, D, block, 0
        self.k = torch.empty((blocks, Hkv, block, D), dtype=torch.float8_e4m3fn, device=device)
        self.v = torch.empty_like(self.k)
        self.k_scale = torch.empty((blocks, Hkv), device=device)
        self.v_scale = torch.empty_like(self.k_scale)
        self.table = torch.randperm(blocks, device=device).to(torch.int32)[None]  # pages in any order
        self.kb = torch.zeros((1, Hkv, blocks, D), dtype=torch.float16, device=device)
        self.lens = torch.zeros(1, dtype=torch.int32, device=device)
        angle = torch.arange(capacity, device=device, dtype=torch.float64)[:, None] \
            * base ** (-torch.arange(D // 2, device=device, dtype=torch.float64) / (D // 2))
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def cache(self):
        return self.k, self.v, self.k_scale, self.v_scale, self.table, self.lens

    def append(self, q, k, v):
        """q [1, n, Hq, D], k and v [1, n, Hkv, D] of the next n tokens; returns the rotated q."""
        self.tokens += k.shape[1]
        self.lens += k.shape[1]
        return tbs.qsa_kv_append(k, v, *self.cache(), cos=self.cos, sin=self.sin, q=q, kb=self.kb)

    def select(self, q, k: int):
        """The k best blocks of each KV head for rotated queries q [1, n, Hq, D]: ids [1, Hkv, n, k]."""
        n = q.shape[1]
        per_head = q.reshape(n, self.Hkv, self.Hq // self.Hkv, self.D).transpose(0, 1).contiguous()
        _, ids = tbs.qsa_score_select_batched(per_head, self.kb[0], self.tokens, k, self.block)
        return ids[None]

    def attend(self, q, ids=None):
        return tbs.qsa_kv_attend(q, *self.cache(), ids=ids)


def decode(tokens: int, steps: int, k: int, Hq: int = 32, Hkv: int = 4, D: int = 128, block: int = 64, seed: int = 0):
    """Runs the loop on random projections; returns the layer and the last
    step's (rotated query, ids, output)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def project(n):
        x = torch.randn((1, n, Hq + 2 * Hkv, D), generator=g, device="cuda").half()
        return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]

    layer = Layer(tokens + steps, Hq, Hkv, D, block)
    layer.append(*project(tokens))
    for _ in range(steps):
        q = layer.append(*project(1))
        ids = layer.select(q, k)
        out = layer.attend(q, ids)
    return layer, (q, ids, out)


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=131072)
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--k", type=int, default=64)
    a = p.parse_args()
    layer, (q, ids, out) = decode(a.tokens, a.steps, a.k)
    dense = layer.attend(q)
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

    x = torch.cosine_similarity(out.float().flatten(), dense.float().flatten(), 0)
    print(f"{layer.tokens} tokens, {ids.shape[-1]} of {-(-layer.tokens // layer.block)} blocks: "
          f"select {timed(lambda: layer.select(q, a.k)):.1f} us, attend {timed(lambda: layer.attend(q, ids)):.1f} us "
          f"(every block: {timed(lambda: layer.attend(q)):.1f} us); cosine with attention over every block {x:.4f}")
    status, bits = tbs.qsa_device_status()
    assert status == 0, (status, bits)


if __name__ == "__main__":
    main()
