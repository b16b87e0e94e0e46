"""Measured cases of the paged 4-bit cache operators: the append (position
rotation, quantisation, block keys) with the tokens read back, attention over
the whole cached context and over the blocks a selection step chose, the
attention weight that each cached token gathers, and eviction by it.

Where `own` is false, run() computes an operator in elementary torch
operations in 32 bits; where it is true, it calls the library.
"""
import math

import torch

own = False

S_MIN = 2.0 ** -100  # smallest scale of a token
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of a full serving batch, contexts of every length
        dict(name="append_decode_64", op="append", B=64, n=1, Hq=32, Hkv=8, D=128, block=64, lo=1, hi=8191, rot=128,
             style="half", dtype="f16", ragged=False, evicted=0),
        # a prefill chunk of the 4096-query batch, behind 28K tokens that are cached already
        dict(name="append_chunk_4096", op="append", B=1, n=4096, Hq=32, Hkv=8, D=128, block=64, lo=32805, hi=32805,
             rot=128, style="half", dtype="f16", ragged=False, evicted=0),
        # chunks of several requests, different counts of new tokens, half the dimensions rotated, small blocks, behind
        # tokens of which some were evicted
        dict(name="append_ragged_7x333", op="append", B=7, n=333, Hq=12, Hkv=4, D=64, block=32, lo=200, hi=2999, rot=32,
             style="pairs", dtype="bf16", ragged=True, evicted=500),
        # one decoded token over a short context: latency
        dict(name="attend_1x1000", op="attend", B=1, n=1, Hq=8, Hkv=2, D=128, block=64, lo=1000, hi=1000, dtype="f16"),
        # a decode step of a serving batch, contexts of 1K to 16K tokens
        dict(name="attend_decode_64", op="attend", B=64, n=1, Hq=32, Hkv=8, D=128, block=64, lo=1000, hi=16384,
             dtype="bf16"),
        # two long contexts, one token each, 16 query heads on each KV head of 64 dimensions
        dict(name="attend_2x131073_d64", op="attend", B=2, n=1, Hq=64, Hkv=4, D=64, block=64, lo=131073, hi=131073,
             dtype="f16"),
        # a long chunk of a prompt over what is cached of it so far, itself included
        dict(name="attend_chunk_2048", op="attend", B=1, n=2048, Hq=32, Hkv=8, D=128, block=64, lo=32768, hi=32768,
             dtype="bf16"),
        # a decode step of a serving batch, 64 blocks chosen for each KV head of each request
        dict(name="chosen_decode_32", op="chosen", B=32, n=1, Hq=32, Hkv=4, D=128, block=64, lo=8191, hi=32805, k=64,
             per_head=True, dtype="bf16"),
        # a decode step of a serving batch: every cached token's weight grows by what the step gave it
        dict(name="weights_decode_64", op="weights", B=64, n=1, Hq=32, Hkv=8, D=128, block=64, lo=1000, hi=16384,
             decay=1.0, dtype="f16"),
        # the last 64 queries of a prompt say which of its tokens to keep
        dict(name="weights_64_of_32805", op="weights", B=1, n=64, Hq=32, Hkv=8, D=128, block=64, lo=32805, hi=32805,
             decay=0.0, dtype="bf16"),
        # a serving batch back to 4,096 tokens each, after 64 more were decoded
        dict(name="evict_64x4160", op="evict", B=64, n=1, Hq=8, Hkv=8, D=128, block=64, lo=4160, hi=4160, budget=4096,
             sink=4, recent=512, dtype="f16"),
        # a prompt of 128K tokens down to a quarter before decoding
        dict(name="evict_131072_to_32768", op="evict", B=1, n=1, Hq=8, Hkv=8, D=128, block=64, lo=131072, hi=131072,
             budget=32768, sink=64, recent=2048, dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "chosen", "weights", "evict"])
    D = rng.choice([64, 128, 128])
    block = rng.choice([16, 32, 64, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    R = rng.choice([1, 2, 4, 5, 8, 16])
    while Hkv * R > 64:
        R = rng.choice([1, 2, 4, 5, 8])
    case = dict(op=op, Hq=Hkv * R, Hkv=Hkv, D=D, block=block, dtype=rng.choice(["f16", "bf16"]))
    if op == "append":
        n = _log_int(rng, 1, 4096)
        B = _log_int(rng, 1, max(1, min(64, 4096 // n)))
        hi = _log_int(rng, n, max(n, 32768 // B)) + rng.randrange(64)
        lo = max(1, int(hi * rng.uniform(0.05, 1.0)))
        case.update(B=B, n=n, lo=lo, hi=hi, rot=rng.choice([D, D, D // 2]), style=rng.choice(["half", "pairs"]),
                    ragged=rng.random() < 0.5, evicted=rng.choice([0, _log_int(rng, 1, 9999)]))
    elif op == "attend":
        n = rng.choice([1, 1, 1, 2, 4, _log_int(rng, 8, 512)])
        # keys in all: up to those of 64 requests of 8K tokens on 8 heads; keys times rows in all as a chunk's
        B = _log_int(rng, 1, 64 if n < 8 else 4)
        most = min((1 << 22) // (B * Hkv), 131073, (1 << 29) // (B * n * Hkv * R))
        hi = _log_int(rng, max(n, 65), max(n + 65, most))
        case.update(B=B, n=n, lo=max(1, int(hi * rng.uniform(0.05, 1.0))), hi=hi)
    elif op == "chosen":
        n = rng.choice([1, 1, _log_int(rng, 2, 512)])
        B = _log_int(rng, 1, 32) if n == 1 else 1
        k = _log_int(rng, 4, 64)
        # chosen keys in all at most those of 64 queries on 8 KV heads; a cache of at most 4M keys
        while B * n * Hkv * k * block > 64 * 8 * 64 * 64 and n > 1:
            n = max(1, n // 2)
        hi = max(n + block, _log_int(rng, 2000, max(2001, min(131073, (1 << 22) // (B * Hkv)))))
        case.update(B=B, n=n, lo=max(1, int(hi * rng.uniform(0.3, 1.0))) if n == 1 else hi, hi=hi, k=k,
                    per_head=rng.random() < 0.5)
    elif op == "weights":
        n = rng.choice([1, 1, 1, _log_int(rng, 2, 64)])
        B = _log_int(rng, 1, 64 if n == 1 else 4)
        most = min((1 << 22) // (B * Hkv), 131073, (1 << 26) // (B * n * Hkv * R))
        hi = _log_int(rng, max(n, 65), max(n + 65, most))
        case.update(B=B, n=n, lo=max(1, int(hi * rng.uniform(0.05, 1.0))), hi=hi, decay=rng.choice([0.0, 0.98, 1.0]))
    else:
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 200, max(201, min(131072, (1 << 21) // (B * Hkv))))
        budget = max(8, int(hi * rng.choice([0.25, 0.5, 0.9, 0.99])))
        case.update(B=B, n=1, lo=max(1, int(hi * rng.uniform(0.5, 1.0))), hi=hi, budget=budget,
                    sink=min(rng.choice([0, 4, 64]), budget // 4), recent=int(budget * rng.choice([0.0, 0.1, 0.5])))
    return case


def lengths(case):
    """Tokens of each sequence, the new ones included: spread evenly from hi down to lo."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]


def new_counts(case):
    """New tokens of each sequence: all n rows, or in ragged cases from n down to about n / 3, one with none."""
    n, B = case["n"], case["B"]
    if not case.get("ragged"):
        return [n] * B
    return [0 if B > 2 and i == B - 2 else max(1, n - (2 * n // 3) * i // max(1, B - 1)) for i in range(B)]


def work(case):
    B, n, Hq, Hkv, D, block = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "block"))
    L, held = lengths(case), D // 2 + 2  # bytes of a cached key or value
    if case["op"] == "append":
        new = [min(a, b) for a, b in zip(new_counts(case), L)]
        t = sum(new)
        blocks = sum((length - 1) // block - (length - m) // block + 1 for length, m in zip(L, new) if m)
        # a block that was begun earlier has its cached keys read for its block key
        old = sum((length - m) % block for length, m in zip(L, new) if m)
        bytes_ = (t * (2 * Hkv * (2 * D + held) + Hq * D * 4 + case["rot"] * 4) + old * Hkv * held
                  + blocks * Hkv * D * 2 + t * 2 * Hkv * D * 2)
        return {"bytes": bytes_, "flops": t * (Hq + Hkv) * case["rot"] * 3 + t * Hkv * D * 2}
    if case["op"] == "evict":
        # all weights are read; kept tokens behind the first evicted one are read and written
        bytes_ = sum(Hkv * (length * 4 + (case["budget"] - case["sink"]) * (2 * 2 * held + 4))
                     for length in L if length > case["budget"])
        return {"bytes": bytes_ + 12 * B, "flops": 0}
    rows = B * n * Hq * D * 2
    pairs = sum(sum(max(0, length - n + j + 1) for j in range(n)) for length in L)
    if case["op"] == "attend":
        return {"bytes": 2 * sum(L) * Hkv * held + 2 * rows, "flops": 4 * pairs * Hq * D}
    if case["op"] == "weights":
        return {"bytes": sum(L) * Hkv * (held + (8 if case["decay"] else 4)) + rows + B * n * Hq * 4,
                "flops": 2 * pairs * Hq * D}
    k, lists = case["k"], Hkv if case["per_head"] else 1
    nb = [-(-length // block) for length in L]
    read = sum(min(m, n * min(k, m)) for m in nb) * block * Hkv * 2 * held
    pairs = sum(n * min(length, min(k, m) * block) for length, m in zip(L, nb))
    return {"bytes": read + 2 * rows + B * n * k * lists * 4, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ inputs
def _scale_of(top):
    """The smallest bf16 that is at least max|x| / 6 (f32 `top`), and at least S_MIN."""
    s = (top / 6).clamp(min=S_MIN)
    up = ((s.view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32)
    return torch.where(up * 6 < top, (up.view(torch.int32) + 0x10000).view(torch.float32), up)


def _nibbles(y):
    """e2m1 codes, to nearest even, of f32 y."""
    a = y.abs()
    # steps of 1/2 up to 2, of 1 up to 4, of 2 up to 6; round() goes to even
    m = torch.where(a < 2, torch.round(a * 2), torch.where(a < 4, torch.round(a) + 2, (torch.round(a / 2) + 4)))
    return (m.clamp(max=7) + torch.where(torch.signbit(y), 8, 0)).to(torch.uint8)


def _packed(x, s):
    """Bytes of two codes each of x / s, the even element in the low half."""
    c = _nibbles(x / s[..., None])
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _filled_pages(g, pages, Hkv, block, D, dev):
    """Codes and scales of random keys or values, a spread of magnitudes over heads and tokens."""
    codes = torch.empty((pages, Hkv, block, D // 2), dtype=torch.uint8, device=dev)
    scale = torch.empty((pages, Hkv, block), dtype=torch.bfloat16, device=dev)
    step = max(1, (1 << 26) // (Hkv * block * D))
    for i in range(0, pages, step):
        j = min(pages, i + step)
        x = torch.randn((j - i, Hkv, block, D), generator=g, device=dev)
        x *= torch.exp2(torch.randn((j - i, Hkv, block, 1), generator=g, device=dev) * 0.5)
        s = _scale_of(x.abs().amax(-1))
        codes[i:j] = _packed(x, s)
        scale[i:j] = s.to(torch.bfloat16)
    return codes, scale


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, n, Hq, Hkv, D, block = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "block"))
    dt = torch.float16 if case["dtype"] == "f16" else torch.bfloat16
    L = lengths(case)
    max_blocks = -(-max(L) // block)
    need = [-(-length // block) for length in L]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max_blocks), -1, dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    k_cache, k_scale = _filled_pages(g, pages, Hkv, block, D, dev)
    v_cache, v_scale = _filled_pages(g, pages, Hkv, block, D, dev)
    s = dict(case=dict(case), k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale, table=table,
             lens=torch.tensor(L, dtype=torch.int32, device=dev), scale=D ** -0.5)
    s["e2m1"] = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=dev)
    if case["op"] == "append":
        # queries, keys and values as one projection leaves them, side by side
        qkv = torch.randn((B, n, Hq + 2 * Hkv, D), generator=g, device=dev)
        qkv[:, :, Hq:] *= torch.exp2(torch.randn((1, 1, 2 * Hkv, 1), generator=g, device=dev))
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        f = 10000.0 ** (-torch.arange(case["rot"] // 2, dtype=torch.float64, device=dev) / (case["rot"] // 2))
        a = torch.arange(max(L) + case["evicted"], dtype=torch.float64, device=dev)[:, None] * f
        s["cos"], s["sin"] = a.cos().float(), a.sin().float()
        s["new"] = torch.tensor(new_counts(case), dtype=torch.int32, device=dev) if case["ragged"] else None
        s["offset"] = None
        if case["evicted"]:
            s["offset"] = torch.randint(0, case["evicted"] + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        s["q_out"] = torch.zeros((B, n, Hq, D), dtype=dt, device=dev)
        s["kb"] = torch.zeros((B, Hkv, max_blocks, D), dtype=torch.float16, device=dev)
        return s
    if case["op"] == "evict":
        # attention weights as they gather: a few tokens have most of it
        s["weights"] = torch.exp(torch.randn((pages, Hkv, block), generator=g, device=dev) * 2 - 4)
        s["offset"] = torch.zeros(B, dtype=torch.int32, device=dev)
        s["lens_out"] = torch.zeros(B, dtype=torch.int32, device=dev)
        return s
    s["q"] = torch.randn((B, n, Hq, D), generator=g, device=dev).to(dt)
    if case["op"] == "weights":
        s["weights"] = torch.rand((pages, Hkv, block), generator=g, device=dev) * 1e-2
        s["lse"] = torch.logsumexp(_scores(s), -1).reshape(B, Hkv, Hq // Hkv, n).permute(0, 3, 1, 2).reshape(B, n, Hq)
        s["lse"] = s["lse"].contiguous()
    if case["op"] == "chosen":
        # blocks as a selection step lists them: distinct, the part-filled last block first, -1 where there are too few
        lists, k = Hkv if case["per_head"] else 1, case["k"]
        nb = torch.tensor(need, device=dev)
        r = torch.rand((B, lists, n, max_blocks), generator=g, device=dev)
        blk = torch.arange(max_blocks, device=dev)
        r = torch.where(blk == (nb - 1)[:, None, None, None], 2.0, r)
        r = torch.where(blk >= nb[:, None, None, None], -1.0, r)
        top = r.topk(min(k, max_blocks), dim=-1)
        ids = torch.full((B, lists, n, k), -1, dtype=torch.int32, device=dev)
        ids[..., :top.indices.shape[-1]] = torch.where(top.values >= 0, top.indices, -1).to(torch.int32)
        s["ids"] = ids
    return s


# ------------------------------------------------------------- plain forms
def _values(s, codes, scale):
    """f32 values of bytes [..., D / 2] with scales [...]."""
    x = torch.stack([s["e2m1"][(codes & 15).int()], s["e2m1"][(codes >> 4).int()]], -1).flatten(-2)
    return x * scale.float()[..., None]


def _rotate(x, cos, sin, rot, style):
    """f32 x [B, n, H, D] by the angles of cos, sin [B, n, rot / 2]."""
    c, s = cos[:, :, None], sin[:, :, None]
    if style == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * c - b * s, b * c + a * s, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), x[..., rot:]], -1)


def _append(s):
    case = s["case"]
    B, n, Hkv, D, block = (case[x] for x in ("B", "n", "Hkv", "D", "block"))
    dev, table, dt = s["table"].device, s["table"].long(), s["q"].dtype
    lens = s["lens"].long()
    new = s["new"].long() if s["new"] is not None else torch.full((B,), n, device=dev)
    first = lens - new  # slot of the first new token; those before 0 are left out
    slot = first[:, None] + torch.arange(n, device=dev)
    there = (torch.arange(n, device=dev) < new[:, None]) & (slot >= 0)
    at = torch.where(there, slot + (s["offset"].long()[:, None] if s["offset"] is not None else 0), 0)
    cos, sin = s["cos"][at], s["sin"][at]
    k = _rotate(s["k"].float(), cos, sin, case["rot"], case["style"])
    q = _rotate(s["q"].float(), cos, sin, case["rot"], case["style"])
    s["q_out"].copy_(torch.where(there[:, :, None, None], q, 0.0).to(dt))
    slot = torch.where(there, slot, 0)
    page = table.gather(1, slot // block)
    b_, j_ = torch.nonzero(there, as_tuple=True)
    to_page, to_slot = page[b_, j_], (slot % block)[b_, j_]
    held = []
    for x, cache, scale in ((k, s["k_cache"], s["k_scale"]), (s["v"].float(), s["v_cache"], s["v_scale"])):
        t = _scale_of(x.abs().amax(-1))
        cache[to_page, :, to_slot] = _packed(x, t)[b_, j_]
        scale[to_page, :, to_slot] = t.to(torch.bfloat16)[b_, j_]
        y = _values(s, cache[page, :, slot % block], scale[page, :, slot % block])
        held.append(torch.where(there[:, :, None, None], y, 0.0).to(dt))
    # block keys of the blocks that the new tokens reach, from the first one on
    where = first.clamp(min=0)[:, None] // block + torch.arange((n + block - 2) // block + 1, device=dev)
    pos = where[:, :, None] * block + torch.arange(block, device=dev)
    reached = ((pos >= first[:, None, None]) & (pos < lens[:, None, None])).any(-1)
    page = table.gather(1, where.clamp(max=table.shape[1] - 1)).clamp(min=0)
    filled = (pos < lens[:, None, None])[:, :, None]
    y = torch.where(filled[..., None], _values(s, s["k_cache"][page], s["k_scale"][page]), 0.0)
    mean = (y.sum(3) / filled.sum(-1, keepdim=True).clamp(min=1)).to(torch.float16)
    pick = torch.nonzero(reached, as_tuple=True)
    s["kb"][pick[0], :, where[pick]] = mean[pick]
    return {"k": held[0], "v": held[1], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "kb": s["kb"], "q": s["q_out"]}


def _context(s, cache, scale):
    """f32 [B, Hkv, T, D] of the whole context, and its visibility [B, n, T] to each new row."""
    case, table = s["case"], s["table"].long().clamp(min=0)
    x = _values(s, cache[table], scale[table])  # [B, blocks, Hkv, block, D]
    return x.transpose(1, 2).reshape(case["B"], case["Hkv"], -1, case["D"])


def _limit(s):
    """Last slot that each new row sees [B, n]."""
    n = s["case"]["n"]
    return s["lens"].long()[:, None] - n + torch.arange(n, device=s["lens"].device)


def _scores(s):
    """softmax scale * q.k [B, Hkv, R n, T], -inf where a row does not see a token."""
    case = s["case"]
    B, n, Hq, Hkv, D = (case[x] for x in ("B", "n", "Hq", "Hkv", "D"))
    R = Hq // Hkv
    k = _context(s, s["k_cache"], s["k_scale"])
    T = k.shape[2]
    q = s["q"].float().reshape(B, n, Hkv, R, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, R * n, D)
    a = (q @ k.transpose(-1, -2)) * s["scale"]
    seen = torch.arange(T, device=a.device) <= _limit(s)[:, :, None]
    return torch.where(seen[:, None, None], a.reshape(B, Hkv, R, n, T), -math.inf).reshape(B, Hkv, R * n, T)


def _attend(s):
    case = s["case"]
    B, n, Hq, Hkv, D = (case[x] for x in ("B", "n", "Hq", "Hkv", "D"))
    a = _scores(s)
    v = _context(s, s["v_cache"], s["v_scale"])
    v = torch.where((torch.arange(v.shape[2], device=v.device) < s["lens"][:, None])[:, None, :, None], v, 0.0)
    m = a.amax(-1, keepdim=True)
    e = torch.exp(a - torch.where(m == -math.inf, 0.0, m))
    t = e.sum(-1, keepdim=True)
    o = (e @ v) / torch.where(t > 0, t, 1.0)
    return o.reshape(B, Hkv, Hq // Hkv, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D).to(s["q"].dtype)


def _attend_chosen(s):
    case = s["case"]
    B, n, Hq, Hkv, D, block, c = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "block", "k"))
    R, dev = Hq // Hkv, s["table"].device
    ids = s["ids"].long().expand(B, Hkv, n, c)
    page = s["table"].long().gather(1, ids.clamp(min=0).reshape(B, -1)).reshape(B, Hkv, n, c).clamp(min=0)
    h = torch.arange(Hkv, device=dev)[None, :, None, None]
    k = _values(s, s["k_cache"][page, h], s["k_scale"][page, h]).reshape(B, Hkv, n, c * block, D)
    p = (ids[..., None] * block + torch.arange(block, device=dev)).reshape(B, Hkv, n, c * block)
    there = (ids >= 0)[..., None].expand(B, Hkv, n, c, block).reshape(B, Hkv, n, c * block)
    seen = there & (p <= _limit(s)[:, None, :, None])
    q = s["q"].float().reshape(B, n, Hkv, R, D).transpose(1, 2)
    a = (q @ k.transpose(-1, -2)) * s["scale"]  # [B, Hkv, n, R, keys]
    a = torch.where(seen[:, :, :, None], a, -math.inf)
    m = a.amax(-1, keepdim=True)
    e = torch.exp(a - torch.where(m == -math.inf, 0.0, m))
    t = e.sum(-1, keepdim=True)
    v = _values(s, s["v_cache"][page, h], s["v_scale"][page, h]).reshape(B, Hkv, n, c * block, D)
    v = torch.where(seen[..., None], v, 0.0)
    o = (e @ v) / torch.where(t > 0, t, 1.0)
    return o.transpose(1, 2).reshape(B, n, Hq, D).to(s["q"].dtype)


def _weights(s):
    case = s["case"]
    B, n, Hq, Hkv, block = (case[x] for x in ("B", "n", "Hq", "Hkv", "block"))
    a = _scores(s)
    lse = s["lse"].reshape(B, n, Hkv, Hq // Hkv).permute(0, 2, 3, 1).reshape(B, Hkv, -1, 1)
    # rows that see nothing give no token any weight
    p = torch.where(lse == -math.inf, 0.0, torch.exp(a - lse)).sum(2)  # [B, Hkv, T]
    table, t = s["table"].long(), torch.arange(p.shape[-1], device=p.device)
    b_, i_ = torch.nonzero(table >= 0, as_tuple=True)
    page = table[b_, i_]
    p = p.reshape(B, Hkv, -1, block).transpose(1, 2)  # [B, blocks, Hkv, block]
    old = t < s["lens"][:, None] - n
    filled = (t < s["lens"][:, None]).reshape(B, -1, 1, block)
    before = s["weights"][table.clamp(min=0)]
    kept = torch.where(old.reshape(B, -1, 1, block), before * case["decay"], 0.0)
    s["weights"][page] = torch.where(filled, kept + p, before)[b_, i_]
    return s["weights"]


def _evict(s):
    case = s["case"]
    B, Hkv, block, budget = (case[x] for x in ("B", "Hkv", "block", "budget"))
    table, lens = s["table"].long().clamp(min=0), s["lens"].long()[:, None, None]
    w = s["weights"][table].transpose(1, 2).reshape(B, Hkv, -1)
    t = torch.arange(w.shape[-1], device=w.device)
    kept = (t < case["sink"]) | (t >= lens - case["recent"])
    w = torch.where(t >= lens, -1.0, torch.where(kept, math.inf, w))
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget].sort(-1).values
    # order[b, h, i] goes to slot i of the sequences that are too long
    b_, h_, i_ = torch.nonzero((lens > budget).expand(order.shape), as_tuple=True)
    src = order[b_, h_, i_]
    from_page, from_slot, to_page, to_slot = table[b_, src // block], src % block, table[b_, i_ // block], i_ % block
    for x in (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["weights"]):
        x[to_page, h_, to_slot] = x[from_page, h_, from_slot]
    s["lens_out"].copy_(s["lens"].clamp(max=budget))
    s["offset"] += s["lens"] - s["lens_out"]
    return {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"],
            "weights": s["weights"], "lens": s["lens_out"], "offset": s["offset"]}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"append": _append, "attend": _attend, "chosen": _attend_chosen, "weights": _weights, "evict": _evict}[op](s)
    import top_block_selection_gb300 as tbs
    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"])
    if op == "append":
        tbs.qsa_kv4_append(s["k"], s["v"], *cache, cos=s["cos"], sin=s["sin"], interleaved=case["style"] == "pairs",
                           n_new=s["new"], offset=s["offset"], q=s["q"], q_out=s["q_out"], kb=s["kb"])
        k, v = tbs.qsa_kv4_read(*cache, n=case["n"], dtype=s["q"].dtype, n_new=s["new"])
        return {"k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"], "kb": s["kb"], "q": s["q_out"]}
    if op == "weights":
        return tbs.qsa_kv4_weights(s["q"], s["lse"], *cache, s["weights"], scale=s["scale"], decay=case["decay"])
    if op == "evict":
        tbs.qsa_kv4_evict(*cache, s["weights"], budget=case["budget"], sink=case["sink"], recent=case["recent"],
                          offset=s["offset"], lens_out=s["lens_out"])
        return {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"],
                "weights": s["weights"], "lens": s["lens_out"], "offset": s["offset"]}
    return tbs.qsa_kv4_attend(s["q"], *cache, ids=s.get("ids"), scale=s["scale"])


# --------------------------------------------------------- 64-bit results
def _decoded(codes, scale):
    """f64 values of bytes and scales: sign, two bits of exponent (0: no leading one), one behind the point."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    sign, c = torch.where(c >= 8, -1.0, 1.0), c % 8
    e, m = torch.div(c, 2, rounding_mode="floor"), c % 2
    return sign * torch.where(e == 0, m * 0.5, torch.exp2(e - 1) * (1 + m / 2)) * scale.double()[..., None]


def _coded(x):
    """f64 x [..., D] as the cache holds it (values), and the scales."""
    need = (x.abs().amax(-1) / 6).clamp(min=S_MIN)
    unit = torch.exp2(torch.floor(torch.log2(need)) - 7)
    s = torch.ceil(need / unit) * unit
    y = x / s[..., None]
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    return torch.round(y / step) * step * s[..., None], s


def _exact_append(s):
    case = s["case"]
    n, Hkv, D, block, rot = (case[x] for x in ("n", "Hkv", "D", "block", "rot"))
    like = torch.zeros(s["k"].shape, dtype=torch.float64, device=s["k"].device)
    out = {"k": like, "v": like.clone(), "k_scale": s["k_scale"].double(), "v_scale": s["v_scale"].double(),
           "kb": s["kb"].double(), "q": s["q_out"].double()}
    first_of = torch.arange(0, rot // 2, device=like.device) * (2 if case["style"] == "pairs" else 1)
    second_of = first_of + (1 if case["style"] == "pairs" else rot // 2)
    table = s["table"].tolist()
    ahead = s["offset"].tolist() if s["offset"] is not None else [0] * case["B"]
    for b, (length, m) in enumerate(zip(lengths(case), new_counts(case))):
        skip = max(0, m - length)  # rows whose slot would be negative
        p0 = length - m + skip
        if m - skip <= 0:
            continue
        c = s["cos"][p0 + ahead[b]:length + ahead[b]].double()[:, None]
        sn = s["sin"][p0 + ahead[b]:length + ahead[b]].double()[:, None]
        turned = []
        for x in (s["q"], s["k"]):
            y = x[b, skip:m].double()
            z = y.clone()
            z[..., first_of] = y[..., first_of] * c - y[..., second_of] * sn
            z[..., second_of] = y[..., second_of] * c + y[..., first_of] * sn
            turned.append(z)
        out["q"][b, skip:m] = turned[0]
        out["k"][b, skip:m], ks = _coded(turned[1])
        out["v"][b, skip:m], vs = _coded(s["v"][b, skip:m].double())
        for blk in range(p0 // block, (length - 1) // block + 1):
            page, start = table[b][blk], blk * block
            u, w = max(start, p0), min(start + block, length)
            out["k_scale"][page, :, u - start:w - start] = ks[u - p0:w - p0].T
            out["v_scale"][page, :, u - start:w - start] = vs[u - p0:w - p0].T
            older = _decoded(s["k_cache"][page, :, :u - start], s["k_scale"][page, :, :u - start])
            total = older.sum(1) + out["k"][b, skip + u - p0:skip + w - p0].sum(0)
            out["kb"][b, :, blk] = total / (w - start)
    return out


def _exact_attend(s):
    case = s["case"]
    B, n, Hq, Hkv, D, block = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "block"))
    R, dev = Hq // Hkv, s["table"].device
    out = torch.zeros((B, n, Hq, D), dtype=torch.float64, device=dev)
    for b, length in enumerate(lengths(case)):
        page = s["table"][b, :-(-length // block)].long()
        seen = torch.arange(length, device=dev) <= length - n + torch.arange(n, device=dev)[:, None]
        for h in range(Hkv):
            k = _decoded(s["k_cache"][page, h], s["k_scale"][page, h]).reshape(-1, D)[:length]
            v = _decoded(s["v_cache"][page, h], s["v_scale"][page, h]).reshape(-1, D)[:length]
            for r in range(R):
                a = (s["q"][b, :, h * R + r].double() @ k.T) * s["scale"]
                p = torch.softmax(a.masked_fill(~seen, -math.inf), -1)
                out[b, :, h * R + r] = torch.nan_to_num(p) @ v
    return out


def _exact_chosen(s):
    case = s["case"]
    B, n, Hq, Hkv, D, block = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "block"))
    R, dev = Hq // Hkv, s["table"].device
    out = torch.zeros((B, n, Hq, D), dtype=torch.float64, device=dev)
    ids, L = s["ids"].cpu(), lengths(case)
    for b in range(B):
        for j in range(n):
            for h in range(Hkv):
                blk = ids[b, h if case["per_head"] else 0, j]
                blk = blk[blk >= 0].long().to(dev)
                page = s["table"][b, blk].long()
                pos = (blk[:, None] * block + torch.arange(block, device=dev)).flatten()
                k = _decoded(s["k_cache"][page, h], s["k_scale"][page, h]).reshape(-1, D)
                v = _decoded(s["v_cache"][page, h], s["v_scale"][page, h]).reshape(-1, D)
                seen = pos <= L[b] - n + j
                if bool(seen.any()):
                    a = (s["q"][b, j, h * R:(h + 1) * R].double() @ k[seen].T) * s["scale"]
                    out[b, j, h * R:(h + 1) * R] = torch.softmax(a, -1) @ v[seen]
    return out


def _exact_weights(s):
    case = s["case"]
    n, Hq, Hkv, D, block = (case[x] for x in ("n", "Hq", "Hkv", "D", "block"))
    R, dev = Hq // Hkv, s["table"].device
    out = s["weights"].double()
    for b, length in enumerate(lengths(case)):
        page = s["table"][b, :-(-length // block)].long()
        j = torch.arange(n, device=dev)
        seen = torch.arange(length, device=dev) <= length - n + j[:, None]
        for h in range(Hkv):
            k = _decoded(s["k_cache"][page, h], s["k_scale"][page, h]).reshape(-1, D)[:length]
            w = torch.zeros(length, dtype=torch.float64, device=dev)
            w[:max(0, length - n)] = out[page, h].reshape(-1)[:max(0, length - n)] * case["decay"]
            for r in range(R):
                a = (s["q"][b, :, h * R + r].double() @ k.T) * s["scale"] - s["lse"][b, :, h * R + r].double()[:, None]
                w += torch.where(seen & (length - n + j >= 0)[:, None], torch.exp(a), 0.0).sum(0)
            i = torch.arange(length, device=dev)
            out[page[i // block], h, i % block] = w
    return out


def _exact_evict(s):
    case = s["case"]
    block, budget, sink, recent = (case[x] for x in ("block", "budget", "sink", "recent"))
    out = {"k": s["k_cache"].clone(), "v": s["v_cache"].clone(), "k_scale": s["k_scale"].double(),
           "v_scale": s["v_scale"].double(), "weights": s["weights"].double(), "lens": s["lens"].clamp(max=budget),
           "offset": s["offset"] + (s["lens"] - budget).clamp(min=0)}
    to = torch.arange(budget, device=s["lens"].device)
    for b, length in enumerate(lengths(case)):
        if length <= budget:
            continue
        page = s["table"][b].long()
        for h in range(case["Hkv"]):
            w = s["weights"][page.clamp(min=0), h].reshape(-1)[sink:length - recent]
            count = budget - sink - recent
            keep = torch.zeros(length, dtype=torch.bool, device=w.device)
            keep[:sink] = True
            keep[length - recent:] = True
            if count > 0:
                least = w.kthvalue(w.numel() - count + 1).values
                above = w > least
                ties = torch.nonzero(w == least)[:count - int(above.sum()), 0]
                keep[sink:length - recent] = above
                keep[sink + ties] = True
            src = torch.nonzero(keep)[:, 0]
            for name, x in (("k", s["k_cache"]), ("v", s["v_cache"]), ("k_scale", s["k_scale"]),
                            ("v_scale", s["v_scale"]), ("weights", s["weights"])):
                out[name][page[to // block], h, to % block] = x[page[src // block], h, src % block].to(out[name].dtype)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attend" and case["B"] * case["n"] * case["Hq"] * case["hi"] * case["D"] > 1 << 41:
        return None  # minutes in 64 bits
    return {"append": _exact_append, "attend": _exact_attend, "chosen": _exact_chosen, "weights": _exact_weights,
            "evict": _exact_evict}[op](s)
