"""Measured cases of the paged 8-bit cache operators: the append (position
rotation, quantisation, block keys), attention over the whole cached context,
and attention over the blocks a selection step chose for each query.

Where `own` is false, run() computes an operator in elementary torch
operations in 32 bits; where it is true, it calls the library.
"""
import math

import torch

own = False

E_MIN = -100  # smallest exponent of a block's scale
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token of one request: latency of the cache write
        dict(name="append_1_token", op="append", B=1, n=1, Hq=32, Hkv=8, D=128, block=64, lo=4001, hi=4001, rot=128,
             style="half", dtype="f16", ragged=False),
        # a decode step of a full serving batch, contexts of every length
        dict(name="append_decode_64", op="append", B=64, n=1, Hq=32, Hkv=8, D=128, block=64, lo=1, hi=8191, rot=128,
             style="half", dtype="f16", ragged=False),
        # a prefill chunk of the 4096-query batch, behind 28K tokens that are cached already
        dict(name="append_chunk_4096", op="append", B=1, n=4096, Hq=32, Hkv=8, D=128, block=64, lo=32805, hi=32805,
             rot=128, style="half", dtype="f16", ragged=False),
        # chunks of several requests, different counts of new tokens, half the dimensions rotated, small blocks
        dict(name="append_ragged_7x333", op="append", B=7, n=333, Hq=12, Hkv=4, D=64, block=32, lo=200, hi=2999, rot=32,
             style="pairs", dtype="bf16", ragged=True),
        # one decoded token over a short context: latency
        dict(name="attend_1x1000", op="attend", B=1, n=1, Hq=8, Hkv=2, D=128, block=64, lo=1000, hi=1000, dtype="f16"),
        # a decode step of a serving batch, contexts of 1K to 16K tokens
        dict(name="attend_decode_64", op="attend", B=64, n=1, Hq=32, Hkv=8, D=128, block=64, lo=1000, hi=16384,
             dtype="bf16"),
        # two long contexts, one token each, 16 query heads on each KV head
        dict(name="attend_2x131073", op="attend", B=2, n=1, Hq=64, Hkv=4, D=128, block=64, lo=131073, hi=131073,
             dtype="f16"),
        # a chunk of queries over a few thousand cached tokens, below the length where selection pays
        dict(name="attend_chunk_2x129", op="attend", B=2, n=129, Hq=16, Hkv=4, D=64, block=32, lo=2111, hi=4096,
             dtype="f16"),
        # one decoded token over the 32 blocks chosen of the 32768+37 token context, one key head
        dict(name="chosen_1_of_32805", op="chosen", B=1, n=1, Hq=16, Hkv=1, D=128, block=64, lo=32805, hi=32805, k=32,
             per_head=False, dtype="f16"),
        # a decode step of a serving batch, 64 blocks chosen for each KV head of each request
        dict(name="chosen_decode_32", op="chosen", B=32, n=1, Hq=32, Hkv=4, D=128, block=64, lo=8191, hi=32805, k=64,
             per_head=True, dtype="bf16"),
        # the 256-query batch of the 128K context, 64 blocks chosen for each query, 8 KV heads
        dict(name="chosen_256_of_131072", op="chosen", B=1, n=256, Hq=32, Hkv=8, D=128, block=64, lo=131072, hi=131072,
             k=64, per_head=False, dtype="f16"),
        # the 4096-query prefill batch of the 128K context, 16 heads on one key head
        dict(name="chosen_4096_of_131073", op="chosen", B=1, n=4096, Hq=16, Hkv=1, D=128, block=64, lo=131073,
             hi=131073, k=64, per_head=False, dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "chosen"])
    D = rng.choice([64, 128, 128])
    block = rng.choice([32, 64, 64, 128])
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
                    ragged=rng.random() < 0.5)
    elif op == "attend":
        n = rng.choice([1, 1, 1, 2, 4, _log_int(rng, 8, 256)])
        # keys in all: up to those of 64 requests of 8K tokens on 8 heads; keys times rows in all as the chunk's
        B = _log_int(rng, 1, 64 if n < 8 else 4)
        most = min((1 << 22) // (B * Hkv), 131073, (1 << 28) // (B * n * Hkv * R))
        hi = _log_int(rng, max(n, 65), max(n + 65, most))
        case.update(B=B, n=n, lo=max(1, int(hi * rng.uniform(0.05, 1.0))), hi=hi)
    else:
        n = rng.choice([1, 1, _log_int(rng, 2, 2048)])
        B = _log_int(rng, 1, 32) if n == 1 else 1
        k = _log_int(rng, 4, 64)
        # chosen keys in all at most those of 256 queries on 8 KV heads; a cache of at most 1M keys on one head
        while B * n * Hkv * k * block > 256 * 8 * 64 * 64 and n > 1:
            n = max(1, n // 2)
        hi = max(n + block, _log_int(rng, 2000, max(2001, min(131073, (1 << 22) // (B * Hkv)))))
        case.update(B=B, n=n, lo=max(1, int(hi * rng.uniform(0.3, 1.0))) if n == 1 else hi, hi=hi, k=k,
                    per_head=rng.random() < 0.5)
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
    L = lengths(case)
    if case["op"] == "append":
        new = [min(a, b) for a, b in zip(new_counts(case), L)]
        t = sum(new)
        blocks = sum((length - 1) // block - (length - m) // block + 1 for length, m in zip(L, new) if m)
        # a block that was begun earlier has its cached keys read for its block key
        old = sum((length - m) % block for length, m in zip(L, new) if m)
        bytes_ = (t * D * (2 * Hkv * 2 + 2 * Hkv + Hq * 4) + t * case["rot"] * 4 + old * Hkv * D
                  + blocks * Hkv * (D * 2 + 8))
        return {"bytes": bytes_, "flops": t * (Hq + Hkv) * case["rot"] * 3 + t * Hkv * D * 2}
    rows = B * n * Hq * D * 2 * 2
    if case["op"] == "attend":
        keys = sum(L)
        pairs = sum(sum(max(0, length - n + j + 1) for j in range(n)) for length in L)
        return {"bytes": 2 * keys * Hkv * D + keys // block * Hkv * 8 + rows, "flops": 4 * pairs * Hq * D}
    k, lists = case["k"], Hkv if case["per_head"] else 1
    nb = [-(-length // block) for length in L]
    read = sum(min(m, n * min(k, m)) for m in nb) * block * Hkv * D * 2
    pairs = sum(n * min(length, min(k, m) * block) for length, m in zip(L, nb))
    return {"bytes": read + rows + B * n * k * lists * 4, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ inputs
def _scales(amax):
    """2^E, E the smallest with amax <= 448 * 2^E (E >= E_MIN)."""
    m, e = torch.frexp(amax)
    E = torch.where(m <= 0.875, e - 9, e - 8)
    E = torch.where(amax > 0, E, torch.full_like(E, E_MIN)).clamp(min=E_MIN)
    return torch.ldexp(torch.ones_like(amax), E)


def _filled_pages(g, pages, Hkv, block, D, dev):
    """Codes and scales of random keys or values, a spread of magnitudes over heads and blocks."""
    codes = torch.empty((pages, Hkv, block, D), dtype=F8, device=dev)
    scale = torch.empty((pages, Hkv), device=dev)
    step = max(1, (1 << 26) // (Hkv * block * D))
    for i in range(0, pages, step):
        j = min(pages, i + step)
        x = torch.randn((j - i, Hkv, block, D), generator=g, device=dev)
        x *= torch.exp2(torch.randn((j - i, Hkv, 1, 1), generator=g, device=dev) * 0.5)
        s = _scales(x.abs().amax((2, 3)))
        codes[i:j] = (x / s[:, :, None, None]).to(F8)
        scale[i:j] = s
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
             lens=torch.tensor(L, dtype=torch.int32, device=dev))
    if case["op"] == "append":
        # queries, keys and values as one projection leaves them, side by side
        qkv = torch.randn((B, n, Hq + 2 * Hkv, D), generator=g, device=dev)
        qkv[:, :, Hq:] *= torch.exp2(torch.randn((1, 1, 2 * Hkv, 1), generator=g, device=dev))
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        f = 10000.0 ** (-torch.arange(case["rot"] // 2, dtype=torch.float64, device=dev) / (case["rot"] // 2))
        a = torch.arange(max(L), dtype=torch.float64, device=dev)[:, None] * f
        s["cos"], s["sin"] = a.cos().float(), a.sin().float()
        s["new"] = torch.tensor(new_counts(case), dtype=torch.int32, device=dev) if case["ragged"] else None
        s["q_out"] = torch.zeros((B, n, Hq, D), dtype=dt, device=dev)
        s["kb"] = torch.zeros((B, Hkv, max_blocks, D), dtype=torch.float16, device=dev)
        return s
    s["q"] = torch.randn((B, n, Hq, D), generator=g, device=dev).to(dt)
    s["scale"] = D ** -0.5
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
    dev, table = s["table"].device, s["table"].long()
    lens = s["lens"].long()
    new = s["new"].long() if s["new"] is not None else torch.full((B,), n, device=dev)
    first = lens - new  # position of the first new token; those before 0 are left out
    j = torch.arange(n, device=dev)
    pos = first[:, None] + j
    there = (j < new[:, None]) & (pos >= 0)
    at = torch.where(there, pos, 0)
    cos, sin = s["cos"][at], s["sin"][at]
    k = _rotate(s["k"].float(), cos, sin, case["rot"], case["style"])
    v = s["v"].float()
    q = _rotate(s["q"].float(), cos, sin, case["rot"], case["style"])
    s["q_out"].copy_(torch.where(there[:, :, None, None], q, 0.0).to(s["q_out"].dtype))
    # the blocks that the new tokens reach, from the first one on
    blocks = (n + block - 2) // block + 1
    begin = first.clamp(min=0) // block
    where = begin[:, None] + torch.arange(blocks, device=dev)
    slot = where[:, :, None] * block + torch.arange(block, device=dev)  # positions [B, blocks, block]
    from_new = (slot >= first[:, None, None]) & (slot < lens[:, None, None])
    from_old = slot < first[:, None, None].clamp(min=0)
    reached = from_new.any(-1)
    page = table.gather(1, where.clamp(max=table.shape[1] - 1))
    row = (slot - first[:, None, None]).clamp(0, n - 1).flatten(1)
    fresh = (where * block >= first[:, None])[:, :, None]
    pick = torch.nonzero(reached, as_tuple=True)
    to = page[pick]
    for x, cache, scale in ((k, s["k_cache"], s["k_scale"]), (v, s["v_cache"], s["v_scale"])):
        x = x.gather(1, row[:, :, None, None].expand(-1, -1, Hkv, D))
        x = x.reshape(B, blocks, block, Hkv, D).transpose(2, 3)  # [B, blocks, Hkv, block, D]
        old = cache[page.clamp(min=0)].float()
        s_old = scale[page.clamp(min=0)]
        is_new, is_old = from_new[:, :, None, :, None], from_old[:, :, None, :, None]
        s_new = _scales(torch.where(is_new, x.abs(), 0.0).amax((3, 4)))
        t = torch.where(fresh, s_new, torch.maximum(s_old, s_new))
        t5 = t[:, :, :, None, None]
        codes = torch.where(is_new, x / t5, torch.where(is_old, old * (s_old[:, :, :, None, None] / t5), old)).to(F8)
        cache.view(torch.uint8)[to] = codes.view(torch.uint8)[pick]
        scale[to] = t[pick]
        if cache is s["k_cache"]:
            held = is_new | is_old
            total = torch.where(held, codes.float(), 0.0).sum(3)
            mean = total * t[..., None] / held.sum(3).clamp(min=1)
            s["kb"][pick[0], :, where[pick]] = mean.to(torch.float16)[pick]
    return {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "kb": s["kb"],
            "q": s["q_out"]}


def _attend(s):
    case = s["case"]
    B, n, Hq, Hkv, D, block = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "block"))
    R, dev, table = Hq // Hkv, s["table"].device, s["table"].long()
    T = table.shape[1] * block
    k = s["k_cache"][table.clamp(min=0)].float() * s["k_scale"][table.clamp(min=0)][..., None, None]
    k = k.transpose(1, 2).reshape(B, Hkv, T, D)
    v = s["v_cache"][table.clamp(min=0)].float() * s["v_scale"][table.clamp(min=0)][..., None, None]
    v = v.transpose(1, 2).reshape(B, Hkv, T, D)
    lens = s["lens"].long()
    p = torch.arange(T, device=dev)
    limit = lens[:, None] - n + torch.arange(n, device=dev)  # [B, n]
    v = torch.where((p < lens[:, None])[:, None, :, None], v, 0.0)
    q = s["q"].float().reshape(B, n, Hkv, R, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, R * n, D)
    a = (q @ k.transpose(-1, -2)) * s["scale"]
    seen = (p <= limit[:, :, None])[:, None, None].expand(B, Hkv, R, n, T).reshape(B, Hkv, R * n, T)
    a = torch.where(seen, a, -math.inf)
    m = a.amax(-1, keepdim=True)
    e = torch.exp(a - torch.where(m == -math.inf, 0.0, m))
    t = e.sum(-1, keepdim=True)
    o = (e @ v) / torch.where(t > 0, t, 1.0)
    return o.reshape(B, Hkv, R, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D).to(s["q"].dtype)


def _attend_chosen(s):
    case = s["case"]
    B, n, Hq, Hkv, D, block, c = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "block", "k"))
    R, dev = Hq // Hkv, s["table"].device
    ids = s["ids"].long().expand(B, Hkv, n, c)
    page = s["table"].long().gather(1, ids.clamp(min=0).reshape(B, -1)).reshape(B, Hkv, n, c).clamp(min=0)
    h = torch.arange(Hkv, device=dev)[None, :, None, None]
    k = (s["k_cache"][page, h].float() * s["k_scale"][page, h][..., None, None]).reshape(B, Hkv, n, c * block, D)
    p = (ids[..., None] * block + torch.arange(block, device=dev)).reshape(B, Hkv, n, c * block)
    limit = s["lens"].long()[:, None] - n + torch.arange(n, device=dev)  # [B, n]
    there = (ids >= 0)[..., None].expand(B, Hkv, n, c, block).reshape(B, Hkv, n, c * block)
    seen = there & (p <= limit[:, None, :, None])
    q = s["q"].float().reshape(B, n, Hkv, R, D).transpose(1, 2)
    a = (q @ k.transpose(-1, -2)) * s["scale"]  # [B, Hkv, n, R, keys]
    a = torch.where(seen[:, :, :, None], a, -math.inf)
    m = a.amax(-1, keepdim=True)
    e = torch.exp(a - torch.where(m == -math.inf, 0.0, m))
    t = e.sum(-1, keepdim=True)
    v = (s["v_cache"][page, h].float() * s["v_scale"][page, h][..., None, None]).reshape(B, Hkv, n, c * block, D)
    v = torch.where(seen[..., None], v, 0.0)
    o = (e @ v) / torch.where(t > 0, t, 1.0)
    return o.transpose(1, 2).reshape(B, n, Hq, D).to(s["q"].dtype)


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"append": _append, "attend": _attend, "chosen": _attend_chosen}[op](s)
    import top_block_selection_gb300 as tbs
    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"])
    if op == "append":
        tbs.qsa_kv_append(s["k"], s["v"], *cache, cos=s["cos"], sin=s["sin"], interleaved=s["case"]["style"] == "pairs",
                          n_new=s["new"], q=s["q"], q_out=s["q_out"], kb=s["kb"])
        return {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "kb": s["kb"],
                "q": s["q_out"]}
    return tbs.qsa_kv_attend(s["q"], *cache, ids=s.get("ids"), scale=s["scale"])


# --------------------------------------------------------- 64-bit results
def _e4m3(y):
    """Nearest value with 3 bits behind the point, ties to even, quantum 2^-9 at the least, for |y| <= 448."""
    _, e = torch.frexp(y)
    quantum = torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=-6) - 3)
    return torch.round(y / quantum) * quantum


def _exact_append(s):
    case = s["case"]
    n, Hq, Hkv, D, block, rot = (case[x] for x in ("n", "Hq", "Hkv", "D", "block", "rot"))
    out = {"k": s["k_cache"].double(), "v": s["v_cache"].double(), "k_scale": s["k_scale"].double(),
           "v_scale": s["v_scale"].double(), "kb": s["kb"].double(), "q": s["q_out"].double()}
    first_of = torch.arange(0, rot // 2, device=s["table"].device) * (2 if case["style"] == "pairs" else 1)
    second_of = first_of + (1 if case["style"] == "pairs" else rot // 2)
    table = s["table"].tolist()
    for b, (length, m) in enumerate(zip(lengths(case), new_counts(case))):
        skip = max(0, m - length)  # rows whose position would be negative
        p0 = length - m + skip
        if m - skip <= 0:
            continue
        c, sn = s["cos"][p0:length].double()[:, None], s["sin"][p0:length].double()[:, None]
        turned = []
        for x in (s["q"], s["k"]):
            y = x[b, skip:m].double()
            z = y.clone()
            z[..., first_of] = y[..., first_of] * c - y[..., second_of] * sn
            z[..., second_of] = y[..., second_of] * c + y[..., first_of] * sn
            turned.append(z)
        out["q"][b, skip:m] = turned[0]
        v = s["v"][b, skip:m].double()
        for blk in range(p0 // block, (length - 1) // block + 1):
            page, start = table[b][blk], blk * block
            u, w = max(start, p0), min(start + block, length)
            for name, x in (("k", turned[1]), ("v", v)):
                x = x[u - p0:w - p0].transpose(0, 1)  # [Hkv, tokens, D]
                top = x.abs().amax((1, 2))
                E = torch.ceil(torch.log2(top / 448)).clamp(min=E_MIN)
                E = torch.where(torch.exp2(E - 1) * 448 >= top, E - 1, E).clamp(min=E_MIN)
                E = torch.where(torch.exp2(E) * 448 < top, E + 1, E)
                t = torch.exp2(E)
                if u > start:
                    t = torch.maximum(t, out[name + "_scale"][page])
                    held = out[name][page, :, :u - start]
                    out[name][page, :, :u - start] = _e4m3(held * (out[name + "_scale"][page] / t)[:, None, None])
                out[name][page, :, u - start:w - start] = _e4m3(x / t[:, None, None])
                out[name + "_scale"][page] = t
            out["kb"][b, :, blk] = out["k"][page, :, :w - start].mean(1) * out["k_scale"][page][:, None]
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
            k = (s["k_cache"][page, h].double() * s["k_scale"][page, h].double()[:, None, None]).reshape(-1, D)[:length]
            v = (s["v_cache"][page, h].double() * s["v_scale"][page, h].double()[:, None, None]).reshape(-1, D)[:length]
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
    for b, length in enumerate(lengths(case)):
        for h in range(Hkv):
            for i in range(0, n, 256):
                ids = s["ids"][b, h if case["per_head"] else 0, i:i + 256].long()  # [queries, k]
                page = s["table"][b].long()[ids.clamp(min=0)].clamp(min=0)
                p = ids[..., None] * block + torch.arange(block, device=dev)
                j = torch.arange(i, i + ids.shape[0], device=dev)
                seen = ((ids >= 0)[..., None] & (p <= (length - n + j)[:, None, None])).flatten(1)
                x = [(c[page, h].double() * t[page, h].double()[..., None, None]).flatten(1, 2)
                     for c, t in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"]))]
                q = s["q"][b, i:i + 256, h * R:(h + 1) * R].double()
                a = torch.einsum("qrd,qtd->qrt", q, x[0]) * s["scale"]
                w = torch.softmax(a.masked_fill(~seen[:, None], -math.inf), -1)
                out[b, i:i + 256, h * R:(h + 1) * R] = torch.einsum("qrt,qtd->qrd", torch.nan_to_num(w), x[1])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "chosen": _exact_chosen}[case["op"]](s)
