"""Inputs of the 4-bit cache's tests: small caches with scattered pages; slots
that hold no token have codes of every kind and NaN scales and weights, so that
a stray read shows."""
import numpy as np

from kv_cases import angles, as_bf16, as_f16, blocks_of, ROUND  # noqa: F401
from oracle import kv4_oracle as ko


def make_cache(lens, Hkv, block, D, seed=0, max_blocks=None, n_new=None, filled=True, spread=1.0):
    """A cache for sequences of these lengths; filled: random codes, and scales
    spread by 2^(spread N(0, 1)), up to each length. w: weights of its tokens."""
    rng = np.random.default_rng(seed)
    need = [-(-max(n, 0) // block) for n in lens]
    max_blocks = max(max(need), 1) if max_blocks is None else max_blocks
    pages = sum(need) + 2
    order = rng.permutation(pages)
    table = np.full((len(lens), max_blocks), -7, np.int32)
    c = dict(k=rng.integers(0, 256, (pages, Hkv, block, D // 2), dtype=np.uint8),
             v=rng.integers(0, 256, (pages, Hkv, block, D // 2), dtype=np.uint8),
             k_scale=np.full((pages, Hkv, block), np.nan, np.float32),
             v_scale=np.full((pages, Hkv, block), np.nan, np.float32), table=table, lens=np.array(lens, np.int32),
             n_new=None if n_new is None else np.array(n_new, np.int32),
             w=np.full((pages, Hkv, block), np.nan, np.float32))
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
        for i in range(m if filled else 0):
            held = min(block, lens[b] - i * block)
            for name in ("k_scale", "v_scale"):
                c[name][table[b, i], :, :held] = as_bf16(0.3 * 2.0 ** (spread * rng.standard_normal((Hkv, held))))
            c["w"][table[b, i], :, :held] = np.exp(2 * rng.standard_normal((Hkv, held)))
    return c


def copy_cache(c):
    return {k: None if v is None else v.copy() for k, v in c.items()}


def roomy(c, rows):
    """Page tables with room (of pages that there are not) for 10 x 2^20 rows x tokens:
    calls over these take the form of many rows."""
    block = c["k"].shape[2]
    blocks = -(-(10 << 20) // (rows * block))
    t = np.full((c["table"].shape[0], max(blocks, c["table"].shape[1])), -7, np.int32)
    t[:, :c["table"].shape[1]] = c["table"]
    c["table"] = t
    return c
