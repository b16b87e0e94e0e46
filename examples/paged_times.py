"""Times of attention over the paged 8-bit cache that the decode example does not
show: chunks of prompts over the whole cache, and decode batches of mixed
lengths.

Caches of random codes; each line is the median of seven runs of some calls in
a stream, by CUDA events, after warm-up. The prompts' caches fit the L2 cache
(their time is arithmetic); the batches' larger ones do not.

    python examples/paged_times.py [prompts] [batches]
"""
from __future__ import annotations

import os
import statistics
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import top_block_selection_gb300 as tbs  # noqa: E402

F16, BF16 = torch.float16, torch.bfloat16

# n queries at the end of `tokens` cached tokens, for each of B sequences
PROMPTS = [  # (B, n, tokens, Hq, Hkv, D, dtype)
    (1, 4096, 4096, 32, 8, 128, F16), (1, 4096, 4096, 32, 8, 128, BF16),
    (1, 4096, 32768, 32, 8, 128, F16), (1, 4096, 32768, 32, 8, 128, BF16),
    (1, 2048, 32768, 32, 8, 64, F16), (1, 2048, 32768, 32, 8, 64, BF16),
    (1, 128, 8192, 32, 8, 128, F16), (8, 64, 4096, 32, 8, 128, BF16),
]
BATCHES = [  # (what, tokens of each sequence, n, Hq, Hkv, D, dtype)
    ("32 of 100 and 32 of 16,384", [100] * 32 + [16384] * 32, 1, 32, 8, 128, BF16),
    ("one of 131,072 and 63 of 200", [131072] + [200] * 63, 1, 32, 8, 128, BF16),
    ("64 of 1,000 to 16,384", [1000 + 244 * i for i in range(64)], 1, 32, 8, 128, BF16),
    ("256 of 500", [500] * 256, 1, 32, 8, 128, BF16),
    ("256 of 64 to 829, D 64", [64 + 3 * i for i in range(256)], 1, 32, 8, 64, F16),
    ("1,000 of 50 and 24 of 2,000", [50] * 1000 + [2000] * 24, 1, 16, 2, 128, BF16),
    ("8 of 300 and 8 of 8,000, 4 queries", [300] * 8 + [8000] * 8, 4, 32, 8, 128, F16),
]


def cache(lens, Hkv, D, block=64):
    need = [-(-x // block) for x in lens]
    shape = (sum(need), Hkv, block, D)
    k, v = (torch.randint(0, 0x58, shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    scale = torch.full(shape[:2], 2.0 ** -4, device="cuda")
    order = torch.randperm(shape[0], device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return k, v, scale, scale.clone(), table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def time_us(lens, n, Hq, Hkv, D, dtype, calls=5):
    c = cache(lens, Hkv, D)
    q = torch.randn((len(lens), n, Hq, D), device="cuda").to(dtype)
    out = torch.empty_like(q)
    for _ in range(5):
        tbs.qsa_kv_attend(q, *c, out=out)
    times = []
    for _ in range(7):
        start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(calls):
            tbs.qsa_kv_attend(q, *c, out=out)
        stop.record()
        stop.synchronize()
        times.append(start.elapsed_time(stop) / calls * 1e3)
    return statistics.median(times)


def main():
    which = sys.argv[1:] or ["prompts", "batches"]
    if "prompts" in which:
        for B, n, tokens, Hq, Hkv, D, dtype in PROMPTS:
            us = time_us([tokens] * B, n, Hq, Hkv, D, dtype)
            flops = 4 * B * Hq * D * sum(tokens - n + j + 1 for j in range(n))
            print(f"{B} x {n} queries over {tokens} tokens, {Hq} heads on {Hkv}, D {D}, {str(dtype)[6:]}: {us:.1f} us, "
                  f"{flops / us * 1e-6:.0f} TFLOP/s", flush=True)
    if "batches" in which:
        for what, lens, n, Hq, Hkv, D, dtype in BATCHES:
            us = time_us(lens, n, Hq, Hkv, D, dtype)
            print(f"{what}: {us:.1f} us, {sum(lens) * Hkv * D * 2 / us * 1e-6:.2f} TB/s", flush=True)
    status, bits = tbs.qsa_device_status()
    assert status == 0, (status, bits)


if __name__ == "__main__":
    main()
