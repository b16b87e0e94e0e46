"""Inputs of the paged-cache tests: small caches with scattered pages, spare
pages and slots filled with NaN codes, so that a stray read shows."""
import numpy as np

from oracle import kv_oracle as ko


def as_f16(x):
    return x.astype(np.float16).astype(np.float32)


def as_bf16(x):
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


ROUND = {"f16": as_f16, "bf16": as_bf16}


def make_cache(lens, Hkv, block, D, seed=0, max_blocks=None, n_new=None, filled=True, spread=1.0):
    """A cache for sequences of these lengths; filled: random codes and scales
    up to each length. Every other slot holds the NaN code, every other scale NaN."""
    rng = np.random.default_rng(seed)
    need = [-(-max(n, 0) // block) for n in lens]
    max_blocks = max(max(need), 1) if max_blocks is None else max_blocks
    pages = sum(need) + 2
    order = rng.permutation(pages)
    table = np.full((len(lens), max_blocks), -7, np.int32)
    c = dict(k=np.full((pages, Hkv, block, D), 0x7F, np.uint8), v=np.full((pages, Hkv, block, D), 0xFF, np.uint8),
             k_scale=np.full((pages, Hkv), np.nan, np.float32), v_scale=np.full((pages, Hkv), np.nan, np.float32),
             table=table, lens=np.array(lens, np.int32),
             n_new=None if n_new is None else np.array(n_new, np.int32))
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
        if not filled:
            continue
        for i in range(m):
            held = min(block, lens[b] - i * block)
            for name in ("k", "v"):
                x = rng.standard_normal((Hkv, held, D)) * 2.0 ** (spread * rng.standard_normal((Hkv, 1, 1)))
                for h in range(Hkv):
                    s = ko.scale_of(np.abs(x[h]).max())
                    c[name][table[b, i], h, :held] = ko.encode(x[h] / s)
                    c[name + "_scale"][table[b, i], h] = s
    return c


def make_long_cache(lens, Hkv, block, D, seed=0):
    """As make_cache, of random codes below 16 in magnitude (quick to make)."""
    rng = np.random.default_rng(seed)
    c = make_cache(lens, Hkv, block, D, seed=seed, filled=False)
    for b, length in enumerate(lens):
        for i in range(-(-length // block)):
            held, page = min(block, length - i * block), c["table"][b, i]
            for name in ("k", "v"):
                x = rng.integers(0, 0x58, (Hkv, held, D), dtype=np.uint8)
                c[name][page, :, :held] = x | (rng.integers(0, 2, x.shape, dtype=np.uint8) << 7)
                c[name + "_scale"][page] = 2.0 ** rng.integers(-4, -1, Hkv)
    return c


def angles(positions, rot, base=10000.0):
    f = base ** (-np.arange(rot // 2) / (rot // 2))
    a = np.arange(positions)[:, None] * f
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def copy_cache(c):
    return {k: None if v is None else v.copy() for k, v in c.items()}


def blocks_of(rng, cache, n, lists, k, block):
    """Random distinct blocks per row of each sequence, -1 after them (and one
    -1 between them where there is room)."""
    B = len(cache["lens"])
    ids = np.full((B, lists, n, k), -1, np.int32)
    for b in range(B):
        nb = -(-int(cache["lens"][b]) // block)
        for s in range(lists):
            for j in range(n):
                pick = rng.permutation(nb)[:k]
                ids[b, s, j, :len(pick)] = pick
                if len(pick) > 2 and rng.random() < 0.3:
                    ids[b, s, j, 1] = -1
    return ids
