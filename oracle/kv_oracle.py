"""CPU oracle of the paged 8-bit cache: the append (rotation, scales, e4m3
codes, block keys) and attention over it. Plain numpy, written from the
definitions; shares no code with the GPU path.

A cache here is a dict of numpy arrays: k, v uint8 codes
[pages, Hkv, block, D]; k_scale, v_scale f32 [pages, Hkv]; table int32
[B, max_blocks]; lens int32 [B]; n_new int32 [B] or None.
"""
from __future__ import annotations

import numpy as np

E_MIN = -100


def _decode_table() -> np.ndarray:
    """The 256 values of e4m3: sign, 4 exponent bits (bias 7), 3 fraction
    bits; exponent 0 is subnormal; 0x7F and 0xFF are NaN; no infinities."""
    t = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = np.nan if (c & 0x7F) == 0x7F else (f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10))
        t[c] = -x if c & 0x80 else x
    return t


E4M3 = _decode_table()


def decode(codes):
    return E4M3[codes]


def encode(x):
    """Nearest e4m3 code, ties to the even code, beyond 448 to 448, NaN to NaN
    (searched among the 127 non-negative finite values)."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    grid = E4M3[:127]
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    down, up = a - grid[lo], grid[hi] - a
    code = np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isnan(x), 0x7F, code)
    return (code | np.where(np.signbit(x) & ~np.isnan(x), 0x80, 0)).astype(np.uint8)


def scale_of(amax: float) -> float:
    """The smallest power of two s >= 2^-100 with amax <= 448 s."""
    amax = min(float(amax), float(np.finfo(np.float32).max))
    e = E_MIN
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rotate_f32(x, cos, sin, interleaved):
    """x f32 [..., D] by cos, sin f32 [rot / 2]: fp32, each product and sum
    rounded."""
    rot = 2 * cos.shape[-1]
    y = np.array(x, np.float32)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., a] = (x[..., a] * cos).astype(np.float32) - (x[..., b] * sin).astype(np.float32)
    y[..., b] = (x[..., b] * cos).astype(np.float32) + (x[..., a] * sin).astype(np.float32)
    return y


def append(cache, k, v, cos=None, sin=None, interleaved=False, q=None, kb=None):
    """Updates the cache (and kb f16 [B, Hkv, max_blocks, D]) in place from
    f32 k, v [B, n, Hkv, D]; returns the rotated f32 q (zero where a row does
    not exist)."""
    B, n, Hkv, D = k.shape
    block = cache["k"].shape[2]
    q_out = None if q is None else np.zeros_like(q, dtype=np.float32)
    for b in range(B):
        length = int(cache["lens"][b])
        m = n if cache["n_new"] is None else int(cache["n_new"][b])
        new = {}  # position -> (key, value)
        for j in range(m):
            p = length - m + j
            if p < 0:
                continue
            key = k[b, j].astype(np.float32)
            if cos is not None:
                key = rotate_f32(key, cos[p], sin[p], interleaved)
            new[p] = (key, v[b, j].astype(np.float32))
            if q is not None:
                row = q[b, j].astype(np.float32)
                q_out[b, j] = row if cos is None else rotate_f32(row, cos[p], sin[p], interleaved)
        for blk in sorted({p // block for p in new}):
            page = int(cache["table"][b, blk])
            here = sorted(p for p in new if p // block == blk)
            n_old = here[0] - blk * block
            for h in range(Hkv):
                for which, name in ((0, "k"), (1, "v")):
                    x = np.stack([new[p][which][h] for p in here])
                    finite = np.abs(x[~np.isnan(x)])
                    s = scale_of(finite.max() if finite.size else 0.0)
                    codes, scale = cache[name][page, h], cache[name + "_scale"]
                    if n_old:
                        old = float(scale[page, h])
                        s = max(s, old)
                        if s != old:
                            codes[:n_old] = encode(decode(codes[:n_old]) * (old / s))
                    codes[n_old:n_old + len(here)] = encode(x.astype(np.float64) / s)
                    scale[page, h] = s
                    if which == 0 and kb is not None:
                        held = n_old + len(here)
                        total = decode(codes[:held]).sum(0).astype(np.float32) * np.float32(s)
                        kb[b, h, blk] = (total / np.float32(held)).astype(np.float16)
    return q_out


def seen_tokens(cache, b, j, n, ids=None):
    """(page, offset, position) of what row j of sequence b sees, in order."""
    length = int(cache["lens"][b])
    m = n if cache["n_new"] is None else int(cache["n_new"][b])
    p = length - m + j
    if j >= m or p < 0:
        return []
    block = cache["k"].shape[2]
    blocks = range(p // block + 1) if ids is None else [int(i) for i in ids if i >= 0]
    return [(int(cache["table"][b, i]), o, i * block + o) for i in blocks for o in range(block) if i * block + o <= p]


def attend_row(cache, q, b, j, n, h, scale, ids=None, terms=3):
    """(out [D], lse, bound [D]) in float64 of one query row on KV head h.

    `bound` is the first-order error of the GPU path before the rounding of
    its result, from its number formats: a probability times its value scale is
    off by at most 2^-12 (three terms) or 2^-9 (two) of itself, or 2^-22 or
    2^-19 of the row's largest; a score (fp32 sums of exact products, a query's
    elements to 2^-25 or 2^-21 of the row's largest)
    by (D + 8) 2^-23 sum|q k| + 2^-25 (2^-21) max|q| sum|k|; exp2 and the scaling
    of its argument by 2^-21 (1 + |x|)."""
    seen = seen_tokens(cache, b, j, n, ids)
    D = q.shape[-1]
    if not seen:
        return np.zeros(D), -np.inf, np.zeros(D)
    page, off = np.array([t[0] for t in seen]), np.array([t[1] for t in seen])
    kk = decode(cache["k"][page, h, off]) * cache["k_scale"][page, h].astype(np.float64)[:, None]
    vs = cache["v_scale"][page, h].astype(np.float64)
    code = decode(cache["v"][page, h, off])
    vv = code * vs[:, None]
    q = q.astype(np.float64)
    x = scale * (kk @ q)
    m = np.max(x)
    p = np.exp(x - m)
    total = p.sum()
    out = p @ vv / total
    dx = abs(scale) * ((D + 8) * 2.0 ** -23 * (np.abs(kk) @ np.abs(q))
                       + (2.0 ** -25 if terms == 3 else 2.0 ** -21) * np.abs(q).max() * np.abs(kk).sum(1)) + 2.0 ** -21 * (1 + np.abs(x - m) + np.abs(x))
    rel = (2.0 ** -12 if terms == 3 else 2.0 ** -9) + 2 * dx
    bound = ((p * rel)[:, None] * np.abs(vv)).sum(0) / total + (p * 2 * dx).sum() / total * np.abs(out) \
        + (2.0 ** -22 if terms == 3 else 2.0 ** -19) * (p * vs).max() * np.abs(code).sum(0) / total + (len(seen) + 8) * 2.0 ** -23 * (p @ np.abs(vv)) / total
    return out, m + np.log(total), bound


def attend(cache, q, scale, ids=None, terms=3):
    """q [B, n, Hq, D] -> (out, lse, bound); ids [B, lists, n, k] or None."""
    B, n, Hq, D = q.shape
    Hkv = cache["k"].shape[1]
    R = Hq // Hkv
    out, lse, bound = np.zeros(q.shape), np.zeros(q.shape[:3]), np.zeros(q.shape)
    for b in range(B):
        for j in range(n):
            for hq in range(Hq):
                h = hq // R
                row = None if ids is None else ids[b, h if ids.shape[1] > 1 else 0, j]
                out[b, j, hq], lse[b, j, hq], bound[b, j, hq] = attend_row(cache, q[b, j, hq], b, j, n, h, scale, row,
                                                                               terms)
    return out, lse, bound
