"""GPU parity of the paged 8-bit cache operators with the CPU oracle: the
append bit for bit, attention within the oracle's derived bound plus the
rounding of the result."""
import numpy as np
import pytest

import kv_cases as kc
from oracle import kv_oracle as ko

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"f16": "float16", "bf16": "bfloat16"}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # of the result's rounding (bf16: 8 significant bits)
TINY = {"f16": 2.0 ** -25, "bf16": 0.0}


@pytest.fixture(scope="module")
def tbs():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from top_block_selection_gb300 import _build
    _build.build()
    import top_block_selection_gb300 as m
    m.load_library()
    m.qsa_device_status(clear=True)
    yield m
    assert m.qsa_device_status(clear=True) == (0, 0)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(getattr(torch, DT[dtype]))


def on_gpu(c):
    """The oracle's cache as the binding's positional arguments, and n_new."""
    args = [dev(c[x]) for x in ("k", "v", "k_scale", "v_scale", "table", "lens")]
    return args, None if c["n_new"] is None else dev(c["n_new"])


def same_bits(got, want, what):
    got = got.cpu()
    got = got.view(torch.int16).numpy() if got.dtype in (torch.float16, torch.bfloat16) else got.numpy()
    want = want.view(np.int16) if want.dtype == np.float16 else want
    if got.dtype == np.float32:
        got, want = got.view(np.uint32), np.ascontiguousarray(want, np.float32).view(np.uint32)
    assert got.shape == want.shape and np.array_equal(got, want), (what, int((got != want).sum()), got.size)


# ------------------------------------------------------------------- append
def check_append(tbs, lens, n, Hq, Hkv, D, block, rot, style, dtype, n_new=None, seed=0, old=None, with_kb=True,
                 amp=None, patch=None):
    rng = np.random.default_rng(seed + 1)
    c = kc.make_cache(lens, Hkv, block, D, seed=seed, n_new=n_new, max_blocks=max(1, -(-max(lens) // block) + 1))
    x = rng.standard_normal((len(lens), n, Hq + 2 * Hkv, D)) * (1.0 if amp is None else amp)
    x = kc.ROUND[dtype](x)
    if patch:
        patch(x)
    cos, sin = kc.angles(max(max(lens), 1), rot) if rot else (None, None)
    kb = np.full((len(lens), Hkv, c["table"].shape[1], D), 3.0, np.float16)
    want = kc.copy_cache(c)
    wkb = kb.copy()
    wq = ko.append(want, x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], cos, sin, style == "pairs", x[:, :, :Hq], wkb)
    g = dev(x, dtype)
    args, nn = on_gpu(c)
    gkb = dev(kb) if with_kb else None
    q = tbs.qsa_kv_append(g[:, :, Hq:Hq + Hkv], g[:, :, Hq + Hkv:], *args, cos=None if cos is None else dev(cos),
                          sin=None if sin is None else dev(sin), interleaved=style == "pairs", n_new=nn,
                          q=g[:, :, :Hq], kb=gkb)
    torch.cuda.synchronize()
    for got, name in zip(args, ("k", "v", "k_scale", "v_scale")):
        if name in ("k", "v"):
            w = want[name]
            nan = (w & 0x7F) == 0x7F
            gn = got.cpu().numpy()
            assert np.array_equal((gn & 0x7F) == 0x7F, nan), name  # a NaN's sign is not kept
            assert np.array_equal(gn[~nan], w[~nan]), (name, int((gn[~nan] != w[~nan]).sum()))
        else:
            gs, ws = got.cpu().numpy(), want[name]
            assert np.array_equal(np.isnan(gs), np.isnan(ws)) and np.array_equal(gs[~np.isnan(gs)], ws[~np.isnan(ws)]), name
    if with_kb:
        w = wkb.copy()
        gk = gkb.cpu().numpy()
        assert np.array_equal(np.isnan(gk), np.isnan(w))
        assert np.array_equal(gk[~np.isnan(w)], w[~np.isnan(w)]), "kb"
    wq = torch.from_numpy(wq).to(q.dtype)
    assert torch.equal(torch.nan_to_num(q.cpu()), torch.nan_to_num(wq)), "q"


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("D,rot,style,dtype", [(128, 128, "half", "f16"), (64, 32, "pairs", "bf16"),
                                               (128, 64, "pairs", "f16"), (64, 64, "half", "bf16")])
def test_append_sizes(tbs, block, D, rot, style, dtype):
    # one token; a token that begins a block; chunks that begin and end inside blocks
    for lens, n in (([1, block, block + 1, 3 * block], 1), ([block + 3, 2 * block + 5], block + 2),
                    ([5, 2 * block, 7], 5)):
        check_append(tbs, lens, n, 6, 2, D, block, rot, style, dtype, seed=block + n)


def test_append_ragged_and_missing_rows(tbs):
    # no new token, fewer than n, more than the sequence has, an empty sequence
    check_append(tbs, [70, 41, 3, 0, 130], 9, 4, 1, 128, 64, 128, "half", "f16", n_new=[0, 4, 9, 9, 1])
    check_append(tbs, [0, 0], 3, 4, 2, 64, 32, 0, "half", "bf16")


def test_append_one_head_layouts(tbs):
    check_append(tbs, [100], 37, 1, 1, 128, 64, 128, "half", "f16")
    check_append(tbs, [100], 37, 5, 5, 64, 16, 16, "half", "f16", with_kb=False)


@pytest.mark.parametrize("amp", [1e-4, 1.0, 300.0])
def test_append_scale_growth(tbs, amp):
    """New tokens above, near and below the block's scale so far: growth rounds
    the older codes again, a smaller token leaves them."""
    check_append(tbs, [50, 61, 33], 3, 2, 2, 128, 64, 128, "half", "f16", seed=4, amp=amp)


def test_append_special_values(tbs):
    def patch(x):
        x[0, 0, 2:, :] = 0.0                 # an all-zero token
        x[0, 1, 2, 5] = np.inf
        x[0, 1, 3, 6] = -np.inf
        x[0, 2, 4, 7] = np.nan
        x[0, 3, 2, 8] = 6e-8                 # the smallest fp16
    check_append(tbs, [40], 4, 2, 2, 128, 32, 0, "half", "f16", patch=patch)
    check_append(tbs, [4], 4, 2, 2, 64, 64, 0, "half", "f16", amp=0.0)


def test_append_one_by_one_gives_the_same_scales(tbs):
    """Tokens appended together and one at a time: the same scales; codes and
    block keys equal to the oracle's of each order."""
    Hkv, D, block, n = 2, 64, 32, 70
    x = kc.as_f16(np.random.default_rng(5).standard_normal((1, n, 2 * Hkv, D)) *
                  np.exp2(np.arange(n) % 7 - 3)[None, :, None, None])
    once = kc.make_cache([n], Hkv, block, D, filled=False)
    step = kc.copy_cache(once)
    g = dev(x, "f16")
    args, _ = on_gpu(once)
    tbs.qsa_kv_append(g[:, :, :Hkv], g[:, :, Hkv:], *args)
    sargs, _ = on_gpu(step)
    for i in range(n):
        sargs[5].fill_(i + 1)
        tbs.qsa_kv_append(g[:, i:i + 1, :Hkv], g[:, i:i + 1, Hkv:], *sargs)
        step["lens"][0] = i + 1
        ko.append(step, x[:, i:i + 1, :Hkv], x[:, i:i + 1, Hkv:])
    pages = once["table"][0]
    for a, b in zip(args[2:4], sargs[2:4]):
        assert torch.equal(a[pages.tolist()], b[pages.tolist()])
    same_bits(sargs[0], step["k"], "k")
    same_bits(sargs[1], step["v"], "v")


def test_append_without_queries_and_strides(tbs):
    """k and v with swapped axes, v one row repeated over the heads."""
    Hkv, D, block, n = 3, 64, 16, 20
    rng = np.random.default_rng(8)
    k = kc.as_f16(rng.standard_normal((2, n, Hkv, D)))
    v = kc.as_f16(rng.standard_normal((2, n, 1, D)))
    c = kc.make_cache([30, 20], Hkv, block, D, seed=9)
    want = kc.copy_cache(c)
    ko.append(want, k, np.broadcast_to(v, k.shape))
    args, _ = on_gpu(c)
    gk = dev(k.transpose(0, 2, 1, 3), "f16").transpose(1, 2)
    assert tbs.qsa_kv_append(gk, dev(v, "f16").expand(2, n, Hkv, D), *args) is None
    same_bits(args[0], want["k"], "k")
    same_bits(args[1], want["v"], "v")


def test_append_strided_pages(tbs):
    """Keys and values of a page side by side in one allocation."""
    Hkv, D, block = 2, 128, 32
    c = kc.make_cache([45, 70], Hkv, block, D, seed=3)
    x = kc.as_f16(np.random.default_rng(2).standard_normal((2, 6, 2 * Hkv, D)))
    want = kc.copy_cache(c)
    ko.append(want, x[:, :, :Hkv], x[:, :, Hkv:])
    both = dev(np.stack([c["k"], c["v"]], 1))
    args, _ = on_gpu(c)
    g = dev(x, "f16")
    tbs.qsa_kv_append(g[:, :, :Hkv], g[:, :, Hkv:], both[:, 0], both[:, 1], *args[2:])
    same_bits(both[:, 0].contiguous(), want["k"], "k")
    same_bits(both[:, 1].contiguous(), want["v"], "v")
    q = dev(kc.as_f16(np.random.default_rng(1).standard_normal((2, 1, 4, D))), "f16")
    a = tbs.qsa_kv_attend(q, both[:, 0], both[:, 1], *args[2:])
    b = tbs.qsa_kv_attend(q, dev(want["k"]), dev(want["v"]), *args[2:])
    same_bits(a, b.cpu().numpy(), "attend")


# ------------------------------------------------------------------- attend
def check_attend(tbs, c, n, Hq, dtype, ids=None, scale=None, seed=0, amp=1.0, rows=None):
    D = c["k"].shape[3]
    q = kc.ROUND[dtype](np.random.default_rng(seed + 7).standard_normal((len(c["lens"]), n, Hq, D)) * amp)
    if rows:
        rows(q)
    scale = D ** -0.5 if scale is None else scale
    with np.errstate(invalid="ignore"):
        want, wlse, bound = ko.attend(c, q, scale, ids, terms=3 if dtype == "f16" else 2)
    args, nn = on_gpu(c)
    lse = torch.full(q.shape[:3], 7.0, dtype=torch.float32, device="cuda")
    out = tbs.qsa_kv_attend(dev(q, dtype), *args, ids=None if ids is None else dev(ids), scale=scale, n_new=nn, lse=lse)
    torch.cuda.synchronize()
    got, glse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    err = np.abs(got - want)[ok]
    tol = (bound + (UNIT[dtype] * (np.abs(want) + bound)) + TINY[dtype])[ok]
    assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()), float(err.max()))
    fine = np.isfinite(wlse)
    assert np.array_equal(np.isnan(glse), np.isnan(wlse))
    assert np.array_equal(np.isneginf(glse), np.isneginf(wlse))
    assert np.allclose(glse[fine], wlse[fine], rtol=1e-5, atol=1e-4)
    # whatever the bound allows, the result as a whole is as near as its rounding
    if ok.any() and np.linalg.norm(want[ok]) > 0:
        assert np.linalg.norm((got - want)[ok]) <= 2 * UNIT[dtype] * np.linalg.norm(want[ok])
    return out, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("length", [1, 2, 31, 64, 127, 128, 129, 300, 1000])
def test_attend_one_token(tbs, D, block, length):
    c = kc.make_cache([length], 2, block, D, seed=length)
    check_attend(tbs, c, 1, 8, "f16" if length % 2 else "bf16", seed=length)


@pytest.mark.parametrize("R,Hkv", [(1, 3), (2, 1), (4, 2), (5, 2), (8, 1), (16, 1), (32, 1), (17, 1)])
def test_attend_head_groups(tbs, R, Hkv):
    c = kc.make_cache([77, 200], Hkv, 64, 128, seed=R)
    check_attend(tbs, c, 1, R * Hkv, "f16", seed=R)
    c = kc.make_cache([77, 200], Hkv, 32, 64, seed=R)
    check_attend(tbs, c, 2, R * Hkv, "bf16", seed=R)


@pytest.mark.parametrize("n", [2, 7, 33, 130])
def test_attend_several_queries(tbs, n):
    """Causal rows, the later ones past the earlier ones' last token; a
    sequence shorter than n (rows before its first token)."""
    c = kc.make_cache([n + 40, n, max(1, n // 2)], 1, 32, 64, seed=n)
    check_attend(tbs, c, n, 4, "f16", seed=n)


def test_attend_ragged_batch(tbs):
    lens = [0, 1, 500, 64, 3, 1281, 0, 129]
    c = kc.make_cache(lens, 2, 64, 128, seed=2, n_new=[2, 2, 1, 0, 2, 2, 0, 2])
    out, lse = check_attend(tbs, c, 2, 8, "f16")
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
    assert (out[3] == 0).all() and (out[2, 1] == 0).all()


@pytest.mark.parametrize("lens,Hkv,R,D,block,dtype", [
    ([20011, 9000], 8, 4, 64, 64, "f16"), ([40000], 4, 5, 128, 128, "f16"), ([30001], 8, 16, 64, 32, "f16"),
    ([25000, 1, 17001], 4, 32, 64, 64, "f16"), ([200] * 300, 4, 1, 64, 64, "f16"),
    ([90, 0, 700] * 40, 8, 8, 128, 16, "f16"), ([5, 130, 0, 300] * 200, 2, 3, 64, 64, "bf16"),
    ([21000, 3], 4, 16, 128, 64, "bf16"), ([30000], 3, 32, 128, 64, "bf16"), ([9999, 20000], 8, 8, 128, 32, "bf16")])
def test_attend_many_tiles(tbs, lens, Hkv, R, D, block, dtype):
    """Several turns of every stage, items that begin, lie and end inside a
    CTA's share, and items that span CTAs. A row of each sequence and head is
    compared with the oracle."""
    c = kc.make_long_cache(lens, Hkv, block, D, seed=R)
    q = kc.ROUND[dtype](np.random.default_rng(R).standard_normal((len(lens), 1, Hkv * R, D)))
    args, _ = on_gpu(c)
    g = dev(q, dtype)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")
    out = tbs.qsa_kv_attend(g, *args, lse=lse)
    for _ in range(20):
        assert torch.equal(tbs.qsa_kv_attend(g, *args), out)
    assert not torch.isnan(out).any()
    rows = np.random.default_rng(1).permutation([(b, h) for b in range(len(lens)) for h in range(Hkv)])[:40]
    check_rows(c, q, out, lse, dtype, [(b, 0, h * R + (b + h) % R) for b, h in rows])


def check_rows(c, q, out, lse, dtype, rows, ids=None):
    """These (sequence, row, head) of a result against the oracle."""
    got, D, n = out.double().cpu().numpy(), q.shape[3], q.shape[1]
    R = q.shape[2] // c["k"].shape[1]
    for b, j, hq in rows:
        h = hq // R
        listed = None if ids is None else ids[b, h if ids.shape[1] > 1 else 0, j]
        want, wlse, bound = ko.attend_row(c, q[b, j, hq], b, j, n, h, D ** -0.5, listed, terms=3 if dtype == "f16" else 2)
        err = np.abs(got[b, j, hq] - want)
        assert (err <= bound + UNIT[dtype] * (np.abs(want) + bound) + TINY[dtype]).all(), (b, j, hq)
        assert np.linalg.norm(err) <= 2 * UNIT[dtype] * np.linalg.norm(want)
        if lse is not None:
            g = float(lse[b, j, hq])
            assert wlse == g or abs(wlse - g) <= 1e-4 + 1e-5 * abs(wlse)


@pytest.mark.parametrize("n,Hkv,R,block,k,dtype", [(70, 2, 16, 64, 33, "f16"), (300, 1, 8, 32, 12, "bf16"),
                                                   (33, 4, 4, 128, 9, "f16"), (17, 8, 32, 16, 64, "f16")])
def test_attend_many_lists(tbs, n, Hkv, R, block, k, dtype):
    """Many queries with lists of their own, more items than CTAs and fewer."""
    c = kc.make_long_cache([5003], Hkv, block, 128, seed=n)
    rng = np.random.default_rng(n)
    ids = kc.blocks_of(rng, c, n, Hkv, k, block)
    q = kc.ROUND[dtype](rng.standard_normal((1, n, Hkv * R, 128)))
    args, _ = on_gpu(c)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")
    out = tbs.qsa_kv_attend(dev(q, dtype), *args, ids=dev(ids), lse=lse)
    assert torch.equal(tbs.qsa_kv_attend(dev(q, dtype), *args, ids=dev(ids)), out)
    check_rows(c, q, out, lse, dtype, [(0, int(rng.integers(n)), int(rng.integers(Hkv * R))) for _ in range(40)], ids)


def test_attend_strides_and_given_buffers(tbs):
    """Queries inside a wider projection, with swapped axes, one row for every
    head; a given output and workspace."""
    c = kc.make_cache([150, 70], 2, 32, 64, seed=30)
    args, _ = on_gpu(c)
    wide = torch.randn((2, 3, 12, 64), dtype=torch.float16, device="cuda")
    ws = torch.full((tbs.qsa_kv_attend_workspace_bytes(2, 3, 4, 2, 64),), 255, dtype=torch.uint8, device="cuda")
    for q in (wide[:, :, 5:9], wide.transpose(1, 2)[:, 2:5, :2].transpose(1, 2)[:, :2, :2],
              wide[:, :, :1].expand(2, 3, 4, 64), wide[:1, :, :4].expand(2, 3, 4, 64)):
        want = tbs.qsa_kv_attend(q.contiguous(), *args)
        out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        assert tbs.qsa_kv_attend(q, *args, out=out, workspace=ws) is out
        assert torch.equal(out, want)


@pytest.mark.parametrize("amp", [0.0, 1e-3, 30.0])
def test_attend_score_ranges(tbs, amp):
    """Equal scores, nearly equal ones, and one token above all others."""
    c = kc.make_cache([400], 1, 64, 128, seed=11, spread=2.0)
    check_attend(tbs, c, 1, 8, "f16", amp=amp)
    check_attend(tbs, c, 1, 8, "bf16", amp=amp, scale=0.5)


def test_attend_rows_of_different_size(tbs):
    def rows(q):
        q[0, 0, 0] *= 2.0 ** -12
        q[0, 0, 1] *= 2.0 ** 6
        q[0, 0, 2] = 0.0
        q[0, 0, 3, 1:] = 0.0
    c = kc.make_cache([300], 1, 64, 128, seed=12)
    check_attend(tbs, c, 1, 4, "f16", rows=rows)


def test_attend_nan_is_kept_to_what_sees_it(tbs):
    """NaN codes at positions that some rows see and others do not."""
    c = kc.make_cache([140], 1, 32, 64, seed=13)
    t = c["table"][0]
    c["v"][t[4], 0, 5, 9] = 0x7F       # position 133: rows at 133 and later, dimension 9
    c["k"][t[4], 0, 8, 3] = 0xFF       # position 136: rows at 136 and later, every dimension
    out, lse = check_attend(tbs, c, 12, 2, "f16")
    got = torch.isnan(out[0]).any(1).cpu().numpy()  # [n, D]
    for j in range(12):
        p = 128 + j
        assert got[j].all() if p >= 136 else (got[j].nonzero()[0].tolist() == ([9] if p >= 133 else []))

    def rows(q):
        q[0, 3, 0, 0] = np.nan
    c = kc.make_cache([140], 1, 32, 64, seed=13)
    check_attend(tbs, c, 12, 2, "f16", rows=rows)


@pytest.mark.parametrize("Hkv,lists", [(1, 1), (2, 1), (2, 2)])
@pytest.mark.parametrize("block,D,k", [(64, 128, 5), (16, 64, 9), (128, 128, 1), (32, 64, 40)])
def test_attend_chosen_blocks(tbs, Hkv, lists, block, D, k):
    rng = np.random.default_rng(k)
    n = 3
    c = kc.make_cache([9 * block + 5, 2, 2 * block], Hkv, block, D, seed=k)
    ids = kc.blocks_of(rng, c, n, lists, k, block)
    ids[0, 0, 1] = -1                                  # a row that chose nothing
    check_attend(tbs, c, n, 4 * Hkv, "f16", ids=ids)


def test_attend_chosen_blocks_past_the_row(tbs):
    """Blocks that lie behind the row's own position, and a duplicate."""
    c = kc.make_cache([130], 1, 32, 64, seed=3)
    ids = np.array([[[[4, 3, -1], [4, 4, 0], [4, -1, -1], [0, 1, 2]]]], np.int32).repeat(1, 0)
    check_attend(tbs, c, 4, 4, "f16", ids=ids)


def test_attend_all_blocks_chosen_is_the_whole(tbs):
    c = kc.make_cache([700], 2, 64, 128, seed=21)
    ids = np.arange(11, dtype=np.int32)[None, None, None].repeat(1, 0)
    a = ko.attend(c, np.ones((1, 1, 8, 128)), 0.01, ids)
    b = ko.attend(c, np.ones((1, 1, 8, 128)), 0.01)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    check_attend(tbs, c, 1, 8, "f16", ids=ids)
    check_attend(tbs, c, 1, 8, "f16")


def test_attend_repeats_its_bits(tbs):
    lens = [3000, 100, 1777]
    c = kc.make_cache(lens, 2, 64, 128, seed=5)
    args, _ = on_gpu(c)
    q = torch.randn((3, 4, 16, 128), dtype=torch.float16, device="cuda")
    first = tbs.qsa_kv_attend(q, *args)
    for _ in range(5):
        assert torch.equal(tbs.qsa_kv_attend(q, *args), first)


def test_attend_on_another_stream(tbs):
    c = kc.make_cache([900], 1, 64, 128, seed=6)
    args, _ = on_gpu(c)
    q = torch.randn((1, 1, 8, 128), dtype=torch.float16, device="cuda")
    want = tbs.qsa_kv_attend(q, *args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = tbs.qsa_kv_attend(q, *args)
    s.synchronize()
    assert torch.equal(got, want)


def test_attend_in_a_graph(tbs):
    """Captured once, replayed on other data in the same buffers."""
    c = kc.make_cache([500, 64], 1, 64, 128, seed=16)
    args, _ = on_gpu(c)
    q = torch.randn((2, 1, 8, 128), dtype=torch.float16, device="cuda")
    out, ws = torch.empty_like(q), torch.empty(tbs.qsa_kv_attend_workspace_bytes(2, 1, 8, 1, 128), dtype=torch.uint8,
                                               device="cuda")
    tbs.qsa_kv_attend(q, *args, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tbs.qsa_kv_attend(q, *args, out=out, workspace=ws)
    q.copy_(torch.randn_like(q))
    args[5][0] = 333
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, tbs.qsa_kv_attend(q, *args))


def test_offsets_past_32_bits(tbs):
    """Pages behind 2^32 bytes of a cache, written and read."""
    Hkv, block, D = 8, 128, 128
    per = Hkv * block * D
    pages = (1 << 32) // per + 40
    k = torch.empty((pages, Hkv, block, D), dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    ks = torch.ones((pages, Hkv), device="cuda")
    vs = torch.ones((pages, Hkv), device="cuda")
    c = kc.make_cache([300], Hkv, block, D, seed=1, filled=False)
    table = c["table"] + (pages - 20)
    x = kc.as_f16(np.random.default_rng(3).standard_normal((1, 300, 2 * Hkv, D)))
    g = dev(x, "f16")
    lens = dev(c["lens"])
    tbs.qsa_kv_append(g[:, :, :Hkv], g[:, :, Hkv:], k, v, ks, vs, dev(table), lens)
    ko.append(c, x[:, :, :Hkv], x[:, :, Hkv:])
    at = [int(t) for t in c["table"][0]]
    far = [t + pages - 20 for t in at]
    gk = k[far].cpu().numpy()
    for i, t in enumerate(at):
        held = min(block, 300 - i * block)
        assert np.array_equal(gk[i][:, :held], c["k"][t][:, :held])
    q = torch.randn((1, 1, Hkv, D), dtype=torch.float16, device="cuda")
    a = tbs.qsa_kv_attend(q, k, v, ks, vs, dev(table), lens)
    args, _ = on_gpu(c)
    assert torch.equal(a, tbs.qsa_kv_attend(q, *args))


def test_indexes_outside_are_reported(tbs):
    """A page id, a chosen block and a position outside their buffers: skipped,
    recorded in the status word, everything else as without them."""
    c = kc.make_cache([200], 1, 64, 128, seed=17)
    args, _ = on_gpu(c)
    q = kc.as_f16(np.random.default_rng(18).standard_normal((1, 1, 4, 128)))
    want, _, bound = ko.attend(c, q, 128 ** -0.5, np.array([[[[0, 2]]]], np.int32))
    table = args[4].clone()
    table[0, 1] = 1 << 20
    for tab, listed in ((args[4], [0, 2, 99]), (table, [0, 1, 2])):
        ids = torch.tensor([[[listed]]], dtype=torch.int32, device="cuda")
        got = tbs.qsa_kv_attend(dev(q, "f16"), *args[:4], tab, args[5], ids=ids)
        assert tbs.qsa_device_status(clear=True) == (1, 32)
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= bound + UNIT["f16"] * (np.abs(want) + bound) + TINY["f16"]).all()
    kv = torch.randn((1, 1, 1, 128), dtype=torch.float16, device="cuda")
    before = args[0].clone()
    cos = torch.ones((100, 64), device="cuda")
    tbs.qsa_kv_append(kv, kv, *args, cos=cos, sin=cos)            # position 199 of 100
    assert tbs.qsa_device_status(clear=True) == (1, 32)
    assert torch.equal(args[0], before)
    table[0, 3] = -1
    tbs.qsa_kv_append(kv, kv, *args[:4], table, args[5])
    assert tbs.qsa_device_status(clear=True) == (1, 32)
    assert torch.equal(args[0], before)


def test_binding_refuses_wrong_tensors(tbs):
    c = kc.make_cache([100, 30], 2, 32, 64, seed=17)
    args, _ = on_gpu(c)
    q = torch.zeros((2, 3, 4, 64), dtype=torch.float16, device="cuda")
    kv = torch.zeros((2, 3, 2, 64), dtype=torch.float16, device="cuda")
    cos = torch.ones((100, 32), device="cuda")

    def bad(i, t):
        a = list(args)
        a[i] = t
        return a
    wrong = [bad(0, args[0].half()), bad(1, args[1][:, :1]), bad(1, args[1][:-1]), bad(0, args[0].transpose(2, 3)),
             bad(2, args[2].double()), bad(3, args[3][:-1]), bad(4, args[4].long()), bad(4, args[4][:1]),
             bad(4, args[4].t().contiguous().t()), bad(5, args[5].long()), bad(5, args[5].cpu()), bad(2, args[2].cpu())]
    for a in wrong:
        with pytest.raises(ValueError):
            tbs.qsa_kv_attend(q, *a)
        with pytest.raises(ValueError):
            tbs.qsa_kv_append(kv, kv, *a)
    ids = torch.zeros((2, 1, 3, 4), dtype=torch.int32, device="cuda")
    for kw in (dict(ids=ids.long()), dict(ids=ids[:1]), dict(ids=ids[:, :, :2]), dict(ids=ids[..., :0]), dict(ids=ids[0]),
               dict(ids=ids.expand(2, 2, 3, 4)), dict(ids=torch.zeros((2, 4, 3, 4), dtype=torch.int32, device="cuda")),
               dict(out=q.bfloat16()), dict(out=q[:1]), dict(out=q.cpu()), dict(lse=q[..., 0]),
               dict(lse=torch.zeros((2, 3, 2), device="cuda")), dict(n_new=args[5][:1]), dict(n_new=args[5].cpu()),
               dict(workspace=torch.zeros(8, device="cuda"))):
        with pytest.raises(ValueError):
            tbs.qsa_kv_attend(q, *args, **kw)
    for x in (q.float(), q[:1], q[..., :32], q[0], q.cpu(), q.transpose(2, 3).contiguous().transpose(2, 3)):
        with pytest.raises(ValueError):
            tbs.qsa_kv_attend(x, *args)
    for a, kw in (((kv, kv[:, :2]), {}), ((kv, kv.bfloat16()), {}), ((kv[:, :, :1], kv), {}), ((kv, kv), dict(q_out=q)),
                  ((kv, kv), dict(q=q.bfloat16())), ((kv, kv), dict(q=q, q_out=q[:1])),
                  ((kv, kv), dict(cos=cos, sin=cos[:50])), ((kv, kv), dict(cos=cos.half(), sin=cos.half())),
                  ((kv, kv), dict(kb=torch.zeros((2, 2, 1, 64), dtype=torch.float16, device="cuda")))):
        with pytest.raises(ValueError):
            tbs.qsa_kv_append(*a, *args, **kw)
    with pytest.raises(TypeError):
        tbs.qsa_kv_append(kv, kv, *args, cos=cos)
    with pytest.raises(tbs.QsaError):
        tbs.qsa_kv_attend(q, *args, scale=float("inf"))
    with pytest.raises(tbs.QsaError):
        tbs.qsa_kv_attend(q, *args, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(tbs.QsaError):   # rows that are not 16-byte aligned
        tbs.qsa_kv_attend(torch.zeros(2 * 3 * 4 * 64 + 4, dtype=torch.float16, device="cuda")[4:].view(2, 3, 4, 64), *args)
    with pytest.raises(tbs.QsaError):
        tbs.qsa_kv_append(kv, kv, *args, cos=cos[:, :20].contiguous(), sin=cos[:, :20].contiguous())
    assert tbs.qsa_kv_attend(q[:, :0], *args).shape == (2, 0, 4, 64)


def test_arm_names_the_kernels(tbs):
    c = kc.make_cache([200], 1, 64, 128, seed=17)
    args, _ = on_gpu(c)
    tbs.qsa_kv_attend(torch.randn((1, 1, 4, 128), dtype=torch.float16, device="cuda"), *args)
    assert "kv_attend_kernel" in tbs.qsa_arm()
    kv = torch.randn((1, 1, 1, 128), dtype=torch.float16, device="cuda")
    tbs.qsa_kv_append(kv, kv, *args)
    assert "1 launch: kv_append_kernel" in tbs.qsa_arm()
