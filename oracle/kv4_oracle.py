"""CPU oracle of the paged 4-bit cache: append, read, attention, the weight
that cached tokens gather, and eviction by it. Plain numpy, written from the
definitions; shares no code with the GPU path.

A cache here is a dict of numpy arrays: k, v uint8 [pages, Hkv, block, D / 2]
(element 2 i in the low half of byte i); k_scale, v_scale f32 holding bf16
values [pages, Hkv, block]; table int32 [B, max_blocks]; lens int32 [B]; n_new
int32 [B] or None.
"""
from __future__ import annotations

import numpy as np

from .kv_oracle import rotate_f32

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
S_MIN = 2.0 ** -100


def decode(codes):
    """Values of packed bytes [..., D / 2] -> [..., D]."""
    n = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    return np.where(n & 8, -1.0, 1.0) * E2M1[n & 7]


def encode(x):
    """Packed nearest codes of x [..., D], ties to the even code, beyond 6 to 6
    (searched among the eight magnitudes); NaN to 0."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 6.0)
    hi = np.clip(np.searchsorted(E2M1, a), 1, 7)
    lo = hi - 1
    down, up = a - E2M1[lo], E2M1[hi] - a
    n = np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))
    n = np.where(np.isnan(x), 0, n | np.where(np.signbit(x), 8, 0)).astype(np.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def scale_of(amax: float) -> float:
    """The smallest bf16 s >= 2^-100 with amax <= 6 s."""
    amax = min(float(amax), float(np.finfo(np.float32).max))
    if amax <= 6 * S_MIN:
        return S_MIN
    e = int(np.floor(np.log2(amax / 6))) - 1
    while True:  # 128 .. 255 times 2^(e - 7)
        for m in range(128, 256):
            s = m * 2.0 ** (e - 7)
            if amax <= 6 * s:
                return s
        e += 1


def stored(x):
    """(packed codes, scale) of one token's f32 x [D]; NaN anywhere: scale NaN, codes 0."""
    if np.isnan(x).any():
        return np.zeros(len(x) // 2, np.uint8), np.nan
    s = scale_of(np.abs(x).max())
    return encode(x.astype(np.float64) / s), s


def rows_of(cache, b, n):
    """(row, slot) of the rows of sequence b that exist."""
    length = int(cache["lens"][b])
    m = n if cache["n_new"] is None else int(cache["n_new"][b])
    return [(j, length - m + j) for j in range(min(m, n)) if length - m + j >= 0]


def place(cache, b, slot):
    block = cache["k"].shape[2]
    return int(cache["table"][b, slot // block]), slot % block


def append(cache, k, v, cos=None, sin=None, interleaved=False, q=None, kb=None, offset=None):
    """Updates the cache in place from f32 k, v [B, n, Hkv, D]; kb f64 [B, Hkv,
    max_blocks, D] receives the unrounded means. Returns the rotated f32 q."""
    B, n, Hkv, D = k.shape
    block = cache["k"].shape[2]
    q_out = None if q is None else np.zeros_like(q, dtype=np.float32)
    for b in range(B):
        ahead = 0 if offset is None else int(offset[b])
        touched = set()
        for j, slot in rows_of(cache, b, n):
            key, query = k[b, j].astype(np.float32), None if q is None else q[b, j].astype(np.float32)
            if cos is not None:
                key = rotate_f32(key, cos[slot + ahead], sin[slot + ahead], interleaved)
                query = None if q is None else rotate_f32(query, cos[slot + ahead], sin[slot + ahead], interleaved)
            if q is not None:
                q_out[b, j] = query
            page, off = place(cache, b, slot)
            touched.add(slot // block)
            for h in range(Hkv):
                for name, x in (("k", key[h]), ("v", v[b, j, h].astype(np.float32))):
                    cache[name][page, h, off], cache[name + "_scale"][page, h, off] = stored(x)
        if kb is not None:
            for blk in touched:
                held = min(block, int(cache["lens"][b]) - blk * block)
                page = int(cache["table"][b, blk])
                x = decode(cache["k"][page, :, :held]) * cache["k_scale"][page, :, :held].astype(np.float64)[..., None]
                kb[b, :, blk] = x.mean(1)
    return q_out


def read(cache, n):
    """(k, v) f64 [B, n, Hkv, D] of the call's rows, zero where there is none."""
    B, Hkv, D = len(cache["lens"]), cache["k"].shape[1], 2 * cache["k"].shape[3]
    out = np.zeros((2, B, n, Hkv, D))
    for b in range(B):
        for j, slot in rows_of(cache, b, n):
            page, off = place(cache, b, slot)
            for i, name in enumerate(("k", "v")):
                out[i, b, j] = decode(cache[name][page, :, off]) * cache[name + "_scale"][page, :, off, None]
    return out


def seen_slots(cache, b, slot, ids=None):
    """Slots that the row at `slot` sees, in order (with a list, as often as it names their block)."""
    block = cache["k"].shape[2]
    blocks = range(slot // block + 1) if ids is None else [int(i) for i in ids if i >= 0]
    return np.array([i * block + o for i in blocks for o in range(block) if i * block + o <= slot], np.int64)


def gathered(cache, b, h, slots, name):
    """(codes [T, D], scales [T]) f64."""
    block = cache["k"].shape[2]
    page = cache["table"][b, slots // block]
    return decode(cache[name][page, h, slots % block]), cache[name + "_scale"][page, h, slots % block].astype(np.float64)


def attend(cache, q, scale, ids=None, terms=3):
    """q [B, n, Hq, D] -> (out, lse, bound); ids [B, lists, n, k] or None.

    `bound` is the first-order error of the GPU path before the rounding of its
    result, from its number formats, as of the 8-bit cache: a probability times
    its value scale off by at most 2^-12 (three terms) or 2^-9 (two) of itself, or
    2^-22 or 2^-19 of the row's largest; a score (fp32 sums of exact products, a
    query's elements to 2^-25 or 2^-21 of the row's largest) by (D + 8) 2^-23 sum|q k|
    + 2^-25 (2^-21) max|q| sum|k|; exp2 and the scaling of its argument by 2^-21 (1 + |x|)."""
    B, n, Hq, D = q.shape
    R = Hq // cache["k"].shape[1]
    out, lse, bound = np.zeros(q.shape), np.full(q.shape[:3], -np.inf), np.zeros(q.shape)
    for b in range(B):
        for j, slot in rows_of(cache, b, n):
            for hq in range(Hq):
                h = hq // R
                slots = seen_slots(cache, b, slot, None if ids is None else ids[b, h if ids.shape[1] > 1 else 0, j])
                if not len(slots):
                    continue
                kc, ks = gathered(cache, b, h, slots, "k")
                vc, vs = gathered(cache, b, h, slots, "v")
                kk, vv, x1 = kc * ks[:, None], vc * vs[:, None], q[b, j, hq].astype(np.float64)
                x = scale * (kk @ x1)
                m = x.max()
                p = np.exp(x - m)
                total = p.sum()
                o = p @ vv / total
                dx = abs(scale) * ((D + 8) * 2.0 ** -23 * (np.abs(kk) @ np.abs(x1))
                                   + (2.0 ** -25 if terms == 3 else 2.0 ** -21) * np.abs(x1).max() * np.abs(kk).sum(1)) \
                    + 2.0 ** -21 * (1 + np.abs(x - m) + np.abs(x))
                rel = (2.0 ** -12 if terms == 3 else 2.0 ** -9) + 2 * dx
                out[b, j, hq], lse[b, j, hq] = o, m + np.log(total)
                bound[b, j, hq] = ((p * rel)[:, None] * np.abs(vv)).sum(0) / total \
                    + (p * 2 * dx).sum() / total * np.abs(o) \
                    + (2.0 ** -22 if terms == 3 else 2.0 ** -19) * (p * vs).max() * np.abs(vc).sum(0) / total \
                    + (len(slots) + 8) * 2.0 ** -23 * (p @ np.abs(vv)) / total
    return out, lse, bound


def weights(cache, q, lse, w, scale, decay, terms=3):
    """(new weights, bound) f64 [pages, Hkv, block] from w f32. The bound is of the
    GPU path's fp32: an exponent off by (D + 8) 2^-23 |scale| sum|q k| + 2^-25 (2^-21)
    |scale| max|q| sum|k| + 2^-22 (|x| + |lse| + 1), exp2 by 2^-21, a sum of N terms by N 2^-24."""
    B, n, Hq, D = q.shape
    Hkv, block = cache["k"].shape[1:3]
    R = Hq // Hkv
    new, bound = w.astype(np.float64), np.zeros(w.shape)
    for b in range(B):
        length = int(cache["lens"][b])
        m = n if cache["n_new"] is None else int(cache["n_new"][b])
        for h in range(Hkv):
            slots = np.arange(length)
            page, off = cache["table"][b, slots // block], slots % block
            kc, ks = gathered(cache, b, h, slots, "k")
            kk = kc * ks[:, None]
            total = np.where((slots < length - m) & (decay != 0), np.where(slots < length - m, new[page, h, off], 0) * decay, 0.0) \
                if decay != 0 else np.zeros(length)
            err = 2.0 ** -24 * np.abs(total)
            for j, slot in rows_of(cache, b, n):
                for i in range(R):
                    l = float(lse[b, j, h * R + i])
                    if l == -np.inf:
                        continue
                    x1 = q[b, j, h * R + i].astype(np.float64)
                    y = scale * (kk @ x1)
                    p = np.where(slots <= slot, np.exp(y - l), 0.0)
                    dx = abs(scale) * ((D + 8) * 2.0 ** -23 * (np.abs(kk) @ np.abs(x1))
                                       + (2.0 ** -25 if terms == 3 else 2.0 ** -21) * np.abs(x1).max() * np.abs(kk).sum(1)) \
                        + 2.0 ** -22 * (np.abs(y) + abs(l) + 1) + 2.0 ** -21
                    total = total + p
                    err = err + 2 * p * dx
            new[page, h, off] = total
            bound[page, h, off] = err + (len(rows_of(cache, b, n)) * R + 2) * 2.0 ** -24 * np.abs(total)
    return new, bound


def evict(cache, w, budget, sink, recent):
    """Updates the cache and w in place; returns (new lens, tokens that went)."""
    block, Hkv = cache["k"].shape[2], cache["k"].shape[1]
    lens = np.array(cache["lens"])
    for b, length in enumerate(lens):
        if length <= budget:
            continue
        for h in range(Hkv):
            slots = np.arange(length)
            page, off = cache["table"][b, slots // block], slots % block
            middle = list(range(sink, length - recent))
            key = lambda t: np.inf if np.isnan(w[page[t], h, off[t]]) else w[page[t], h, off[t]]  # noqa: E731
            nan = {t for t in middle if np.isnan(w[page[t], h, off[t]])}
            order = sorted(middle, key=lambda t: (t not in nan, -key(t) if t not in nan else 0, t))
            kept = sorted(list(range(sink)) + order[:budget - sink - recent] + list(range(length - recent, length)))
            held = [(cache["k"][page[t], h, off[t]].copy(), cache["v"][page[t], h, off[t]].copy(),
                     cache["k_scale"][page[t], h, off[t]], cache["v_scale"][page[t], h, off[t]], w[page[t], h, off[t]])
                    for t in kept]
            for t, (ck, cv, sk, sv, x) in enumerate(held):
                cache["k"][page[t], h, off[t]], cache["v"][page[t], h, off[t]] = ck, cv
                cache["k_scale"][page[t], h, off[t]], cache["v_scale"][page[t], h, off[t]] = sk, sv
                w[page[t], h, off[t]] = x
    now = np.minimum(lens, budget)
    return now, lens - now
