"""GPU parity of the 4-bit cache operators with the CPU oracle: append, read
and evict bit for bit (block keys within the rounding of an fp32 sum),
attention and weights within the oracle's derived bounds."""
import numpy as np
import pytest

import kv4_cases as kc
from oracle import kv4_oracle as ko

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"f16": "float16", "bf16": "bfloat16"}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # of the result's rounding
TINY = {"f16": 2.0 ** -25, "bf16": 0.0}
NAMES = ("k", "v", "k_scale", "v_scale", "table", "lens")


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
    args = [dev(c[x], "bf16" if x.endswith("scale") else None) for x in NAMES]
    return args, None if c["n_new"] is None else dev(c["n_new"])


def same(got, want, what):
    got = got.float().cpu().numpy() if got.dtype != torch.uint8 and got.dtype != torch.int32 else got.cpu().numpy()
    if got.dtype == np.float32:
        want = want.astype(np.float32)
        nan = np.isnan(want)
        assert np.array_equal(np.isnan(got), nan), what
        got, want = np.where(nan, 0, got).view(np.uint32), np.where(nan, np.float32(0), want).view(np.uint32)
    assert got.shape == want.shape and np.array_equal(got, want), (what, int((got != want).sum()), got.size)


# ------------------------------------------------------------ append, read
def check_append(tbs, lens, n, Hq, Hkv, D, block, rot, style, dtype, n_new=None, seed=0, with_kb=True, amp=1.0,
                 patch=None, offset=None):
    rng = np.random.default_rng(seed + 1)
    c = kc.make_cache(lens, Hkv, block, D, seed=seed, n_new=n_new, max_blocks=max(1, -(-max(lens) // block) + 1))
    x = kc.ROUND[dtype](rng.standard_normal((len(lens), n, Hq + 2 * Hkv, D)) * amp)
    if patch:
        patch(x)
    ahead = 0 if offset is None else max(offset)
    cos, sin = kc.angles(max(max(lens), 1) + ahead, rot) if rot else (None, None)
    want = kc.copy_cache(c)
    wkb = np.full((len(lens), Hkv, c["table"].shape[1], D), 3.0)
    gkb = dev(wkb.astype(np.float16)) if with_kb else None
    wq = ko.append(want, x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], cos, sin, style == "pairs", x[:, :, :Hq], wkb, offset)
    g = dev(x, dtype)
    args, nn = on_gpu(c)
    q = tbs.qsa_kv4_append(g[:, :, Hq:Hq + Hkv], g[:, :, Hq + Hkv:], *args, cos=None if cos is None else dev(cos),
                           sin=None if sin is None else dev(sin), interleaved=style == "pairs", n_new=nn,
                           q=g[:, :, :Hq], kb=gkb, offset=None if offset is None else dev(np.array(offset, np.int32)))
    for got, name in zip(args, NAMES):
        same(got, want[name], name)
    wq = torch.from_numpy(wq).to(q.dtype)
    assert torch.equal(torch.nan_to_num(q.cpu()), torch.nan_to_num(wq)), "q"
    if with_kb:
        # fp32 sums of at most 128 products, each below the largest scale times 6,
        # 7 + 7 roundings deep, the quotient's, and the fp16's
        gk, big = gkb.cpu().numpy().astype(np.float64), 6 * np.nanmax(np.where(np.isfinite(want["k_scale"]), want["k_scale"], 0))
        assert np.array_equal(np.isnan(gk), np.isnan(wkb))
        over = np.abs(wkb) >= 65520.0  # of an fp16
        assert np.array_equal(gk[over], np.copysign(np.inf, wkb[over]))
        ok = ~np.isnan(wkb) & ~over
        lim = 2.0 ** -11 * np.abs(wkb) + 2.0 ** -25 + 16 * 2.0 ** -24 * big
        assert bool((np.abs(gk - wkb)[ok] <= lim[ok]).all()), float((np.abs(gk - wkb) / lim)[ok].max())
    k, v = tbs.qsa_kv4_read(*args, n=n, dtype=g.dtype, n_new=nn)
    for got, w in zip((k, v), ko.read(want, n)):
        same(got, torch.from_numpy(w.astype(np.float32)).to(g.dtype).float().numpy(), "read")


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


def test_append_offsets_and_one_head(tbs):
    check_append(tbs, [100, 30], 37, 1, 1, 128, 64, 128, "half", "f16", offset=[0, 200])
    check_append(tbs, [100], 37, 5, 5, 64, 16, 16, "half", "f16", with_kb=False, offset=[77])


@pytest.mark.parametrize("amp", [1e-7, 1e-3, 300.0])
def test_append_magnitudes(tbs, amp):
    check_append(tbs, [50, 61, 33], 3, 2, 2, 128, 64, 128, "half", "f16", seed=4, amp=amp)
    check_append(tbs, [50, 61, 33], 3, 2, 2, 64, 64, 0, "half", "bf16", seed=4, amp=amp * 1e30)


def test_append_special_values(tbs):
    def patch(x):
        x[0, 0, 2:, :] = 0.0                 # an all-zero token
        x[0, 1, 2, 5] = np.inf
        x[0, 1, 3, 6] = -np.inf
        x[0, 2, 4, 7] = np.nan
        x[0, 3, 2, 8] = 6e-8                 # the smallest fp16
    check_append(tbs, [40], 4, 2, 2, 128, 32, 0, "half", "f16", patch=patch)
    check_append(tbs, [4], 4, 2, 2, 64, 64, 0, "half", "f16", amp=0.0)


def test_codes_at_borders(tbs):
    """Every border between two codes, times scales with all mantissas, and its neighbours in fp32."""
    border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    c = kc.make_cache([128], 1, 128, 128, filled=False)
    k = np.zeros((1, 128, 1, 128), np.float32)
    for t in range(128):
        s = (128 + t) / 128.0
        row = np.concatenate([border * s * f for f in (1.0, 1 - 2.0 ** -8, 1 + 2.0 ** -8, -1.0)] + [[6 * s]])
        k[0, t, 0, :len(row)] = kc.as_bf16(row)
    want = kc.copy_cache(c)
    ko.append(want, k, k)
    args, _ = on_gpu(c)
    tbs.qsa_kv4_append(dev(k, "bf16"), dev(k, "bf16"), *args)
    for got, name in zip(args, NAMES):
        same(got, want[name], name)


def test_append_one_by_one_gives_the_same_bits(tbs):
    Hkv, D, block, n = 2, 64, 32, 70
    x = dev(kc.ROUND["f16"](np.random.default_rng(5).standard_normal((1, n, 2 * Hkv, D))), "f16")
    c = kc.make_cache([n], Hkv, block, D, filled=False)
    once, _ = on_gpu(c)
    step, _ = on_gpu(c)
    kb = [torch.zeros((1, Hkv, 3, D), dtype=torch.float16, device="cuda") for _ in range(2)]
    tbs.qsa_kv4_append(x[:, :, :Hkv], x[:, :, Hkv:], *once, kb=kb[0])
    for t in range(n):
        step[5].fill_(t + 1)
        tbs.qsa_kv4_append(x[:, t:t + 1, :Hkv], x[:, t:t + 1, Hkv:], *step, kb=kb[1])
    for a, b in zip(once[:4], step[:4]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(kb[0], kb[1])


# --------------------------------------------------------------- attention
def check_attend(tbs, lens, n, Hq, Hkv, D, block, dtype, ids=None, n_new=None, seed=0, spread=1.0, scale=None,
                 patch=None, plan=None, c=None):
    rng = np.random.default_rng(seed + 7)
    c = c or kc.make_cache(lens, Hkv, block, D, seed=seed, n_new=n_new, spread=spread)
    q = kc.ROUND[dtype](rng.standard_normal((len(lens), n, Hq, D)))
    if patch:
        patch(c, q)
    scale = D ** -0.5 if scale is None else scale
    if isinstance(ids, tuple):
        ids = kc.blocks_of(rng, c, n, ids[0], ids[1], block)
    want, wlse, bound = ko.attend(c, q, scale, ids, terms=3 if dtype == "f16" else 2)
    args, nn = on_gpu(c)
    lse = torch.full((len(lens), n, Hq), 7.0, device="cuda")
    out = tbs.qsa_kv4_attend(dev(q, dtype), *args, ids=None if ids is None else dev(ids), scale=scale, n_new=nn, lse=lse)
    if plan:
        arm = tbs.load_library().qsa_arm().decode()
        assert plan in arm, arm
    got = out.float().cpu().numpy().astype(np.float64)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    lim = bound + UNIT[dtype] * (np.abs(want) + bound) + TINY[dtype]
    err = np.abs(got - want)
    assert (err[~nan] <= lim[~nan]).all(), (float((err / lim)[~nan].max()), float(err[~nan].max()))
    gl = lse.cpu().numpy().astype(np.float64)
    fine = np.isfinite(wlse)
    assert np.array_equal(gl[~fine & ~np.isnan(wlse)], wlse[~fine & ~np.isnan(wlse)])
    assert np.array_equal(np.isnan(gl), np.isnan(wlse))
    assert (np.abs(gl - wlse)[fine] <= 1e-4 + 1e-5 * np.abs(wlse[fine])).all()
    return out, lse


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_lengths(tbs, D, block, dtype):
    check_attend(tbs, [1, 2, 127, 128, 129, 257, 600, 0], 1, 4, 2, D, block, dtype, seed=block, plan="kv4_attend_kernel")


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 1), (10, 2), (16, 1), (32, 2)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_heads(tbs, Hq, Hkv, D, dtype):
    check_attend(tbs, [300, 5], 1, Hq, Hkv, D, 32, dtype, seed=Hq)
    check_attend(tbs, [300, 5], 3, Hq, Hkv, D, 64, dtype, seed=Hq)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("R", [9, 20, 24, 31, 32])
def test_attend_many_heads_on_one(tbs, R, D, dtype):
    check_attend(tbs, [300, 5], 2, R, 1, D, 64, dtype, seed=R)
    check_attend(tbs, [300, 45], 1, 2 * R, 2, D, 32, dtype, ids=(2, 3), seed=R)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,R", [(64, 12), (64, 16), (64, 32), (128, 24), (128, 32)])
@pytest.mark.parametrize("room", [4096, 1300000])
def test_attend_heads_split_or_whole(tbs, D, R, dtype, room):
    """More than 16 columns, over tables with room for few tiles a CTA and for many."""
    c = kc.make_cache([4000, 100], 1, 128, D, seed=R, max_blocks=room // 128)
    check_attend(tbs, [4000, 100], 1, R, 1, D, 128, dtype, plan="kv_combine_kernel", c=c)


@pytest.mark.parametrize("D", [64, 128])
def test_attend_rows_that_are_not_there(tbs, D):
    check_attend(tbs, [70, 41, 3, 0, 130], 9, 4, 1, D, 64, "f16", n_new=[0, 4, 9, 9, 1])
    check_attend(tbs, [260, 4], 6, 2, 2, D, 32, "bf16")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,n,Hq,Hkv", [([2500, 70, 1300], 1, 8, 2), ([2300, 2200], 3, 12, 4), ([40000], 1, 2, 1)])
def test_attend_split_items(tbs, D, dtype, lens, n, Hq, Hkv):
    """Items of more tiles than a CTA takes, in two parts to one for nearly every CTA."""
    check_attend(tbs, lens, n, Hq, Hkv, D, 64, dtype, plan="kv_combine_kernel", seed=n)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,k,plan", [(1, 40, "kv_combine_kernel"), (20, 40, "kv_combine_kernel"), (75, 40, None), (1, 5, None)])
def test_attend_chosen_items_split_or_not(tbs, D, B, k, plan):
    check_attend(tbs, [3000] + [200] * (B - 1), 1, 4, 2, D, 64, "f16", ids=(2, k * 128 // D), seed=B, plan=plan or "kv4_attend_kernel")
    assert ("combine" in tbs.qsa_arm()) == (plan is not None)


@pytest.mark.parametrize("D,lists,dtype", [(64, 1, "f16"), (128, 2, "bf16"), (64, 2, "bf16"), (128, 1, "f16")])
@pytest.mark.parametrize("block,k", [(16, 9), (64, 3), (128, 5)])
def test_attend_chosen(tbs, D, lists, dtype, block, k):
    check_attend(tbs, [900, 17, 333], 1, 8, 2, D, block, dtype, ids=(lists, k), seed=k)
    check_attend(tbs, [700, 40], 5, 8, 2, D, block, dtype, ids=(lists, k), seed=k)


def test_attend_chosen_nothing_and_twice(tbs):
    ids = np.full((2, 1, 1, 4), -1, np.int32)
    ids[1, 0, 0] = [2, 2, -1, 0]
    check_attend(tbs, [300, 300], 1, 4, 2, 128, 64, "f16", ids=ids)
    check_attend(tbs, [300, 300], 1, 4, 2, 64, 64, "bf16", ids=ids)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 5])
def test_attend_nan_scales(tbs, D, n):
    """A NaN scale reaches the rows that see its token, and no others."""
    def patch(c, q):
        page, off = ko.place(c, 0, 297)
        c["v_scale"][page, 0, off] = np.nan
        page, off = ko.place(c, 1, 200)
        c["k_scale"][page, 1, off] = np.nan
    check_attend(tbs, [300, 220], n, 4, 2, D, 32, "f16", patch=patch)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_scales_far_apart(tbs, D, dtype):
    check_attend(tbs, [500], 1, 4, 1, D, 64, dtype, spread=8.0)
    check_attend(tbs, [500], 1, 4, 1, D, 64, dtype, scale=-3.0)


def test_attend_repeats_its_bits(tbs):
    c = kc.make_cache([2000, 900], 2, 64, 128)
    args, _ = on_gpu(c)
    q = torch.randn((2, 1, 16, 128), device="cuda").half()
    first = tbs.qsa_kv4_attend(q, *args)
    for _ in range(5):
        assert torch.equal(first, tbs.qsa_kv4_attend(q, *args))


MANY = [([256 + 37], 128, 16, 2, 128, "f16"), ([700], 130, 16, 2, 64, "bf16"), ([600, 300], 150, 8, 1, 128, "bf16"),
        ([310, 290], 140, 8, 2, 64, "f16")]


@pytest.mark.parametrize("lens,n,Hq,Hkv,D,dtype", MANY, ids=[str(i) for i in range(len(MANY))])
@pytest.mark.parametrize("block", [16, 64, 128])
def test_attend_many_rows(tbs, lens, n, Hq, Hkv, D, dtype, block):
    c = kc.roomy(kc.make_cache(lens, Hkv, block, D), len(lens) * n * Hq)
    check_attend(tbs, lens, n, Hq, Hkv, D, block, dtype, plan="kv4_attend_many_kernel", c=c)


@pytest.mark.parametrize("D,few,many", [(64, 2000, 2048), (128, 5000, 5120)])
def test_attend_many_rows_by_room(tbs, D, few, many):
    """2,048 rows: a table's room decides, not what it holds."""
    for room, plan in ((few, "kv4_attend_kernel"), (many, "kv4_attend_many_kernel")):
        c = kc.make_cache([300], 1, 16, D, max_blocks=room // 16)
        check_attend(tbs, [300], 128, 16, 1, D, 16, "f16", plan=plan, c=c)


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16")])
def test_attend_many_rows_nan_and_ragged(tbs, D, dtype):
    def patch(c, q):
        page, off = ko.place(c, 0, 170)
        c["v_scale"][page, 0, off] = np.nan
        page, off = ko.place(c, 1, 60)
        c["k_scale"][page, 1, off] = np.nan
    c = kc.roomy(kc.make_cache([200, 150], 2, 32, D, n_new=[128, 100], spread=4.0), 4096)
    check_attend(tbs, [200, 150], 128, 16, 2, D, 32, dtype, patch=patch, plan="kv4_attend_many_kernel", c=c)


# ----------------------------------------------------------------- weights
def check_weights(tbs, lens, n, Hq, Hkv, D, block, dtype, decay, n_new=None, seed=0, scale=None):
    rng = np.random.default_rng(seed + 9)
    c = kc.make_cache(lens, Hkv, block, D, seed=seed, n_new=n_new)
    q = kc.ROUND[dtype](rng.standard_normal((len(lens), n, Hq, D)))
    scale = D ** -0.5 if scale is None else scale
    _, lse, _ = ko.attend(c, q, scale)
    lse = lse.astype(np.float32)
    want, bound = ko.weights(c, q, lse, c["w"], scale, decay, terms=3 if dtype == "f16" else 2)
    args, nn = on_gpu(c)
    w = dev(c["w"])
    assert tbs.qsa_kv4_weights(dev(q, dtype), dev(lse), *args, w, scale=scale, n_new=nn, decay=decay) is w
    got = w.cpu().numpy().astype(np.float64)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    err = np.abs(got - want)
    assert (err[~nan] <= bound[~nan]).all(), (float(err[~nan].max()), float((err / np.maximum(bound, 1e-300))[~nan].max()))
    again = dev(c["w"])
    tbs.qsa_kv4_weights(dev(q, dtype), dev(lse), *args, again, scale=scale, n_new=nn, decay=decay)
    assert torch.equal(w.view(torch.int32), again.view(torch.int32))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_weights_lengths(tbs, D, dtype, block):
    check_weights(tbs, [1, 2, 127, 128, 129, 300, 0, 513], 1, 4, 2, D, block, dtype, 1.0, seed=block)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 1), (16, 2), (16, 1)])
@pytest.mark.parametrize("n", [1, 7, 40])
@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16"), (128, "f16")])
def test_weights_rows(tbs, Hq, Hkv, n, D, dtype):
    check_weights(tbs, [350, 60], n, Hq, Hkv, D, 32, dtype, 0.75, seed=n + Hq)


def test_weights_rows_that_are_not_there(tbs):
    check_weights(tbs, [70, 41, 3, 0, 130], 9, 4, 1, 128, 64, "f16", 0.5, n_new=[0, 4, 9, 9, 1])
    check_weights(tbs, [70, 41, 3, 0, 130], 9, 4, 1, 64, 64, "bf16", 0.0, n_new=[0, 4, 9, 9, 1])
    check_weights(tbs, [300], 32, 32, 1, 128, 64, "f16", 0.0)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16")])
def test_weights_of_silent_rows(tbs, D, dtype, n):
    """Rows with lse -inf, and a NaN key scale before the call's tokens: no weight
    from these rows, and NaN only if another row of the KV head sees the token."""
    c = kc.make_cache([300, 200], 2, 64, D, seed=n)
    page = c["table"][0, 1]
    c["k_scale"][page, :, 5] = np.nan
    args, _ = on_gpu(c)
    q = kc.ROUND[dtype](np.random.default_rng(n).standard_normal((2, n, 8, D)))
    lse = np.full((2, n, 8), 3.0, np.float32)
    lse[0, :, :4] = -np.inf       # all rows of head 0
    lse[0, n // 2, 5] = -np.inf   # one of head 1
    lse[1, :, 6] = -np.inf
    want, bound = ko.weights(c, q, lse, c["w"], D ** -0.5, 0.5, terms=3 if dtype == "f16" else 2)
    w = dev(c["w"])
    tbs.qsa_kv4_weights(dev(q, dtype), dev(lse), *args, w, decay=0.5)
    got = w.cpu().numpy().astype(np.float64)
    ok = ~np.isnan(want)
    assert np.array_equal(np.isnan(got), ~ok) and (np.abs(got - want)[ok] <= bound[ok]).all()
    assert got[page, 0, 5] == 0.5 * c["w"][page, 0, 5] and np.isnan(got[page, 1, 5])


@pytest.mark.parametrize("R", [11, 24, 31, 32])
@pytest.mark.parametrize("n", [1, 5])
def test_weights_many_heads_on_one(tbs, R, n):
    check_weights(tbs, [300, 40], n, R, 1, 64, 64, "f16", 1.0, seed=R)
    check_weights(tbs, [300, 40], n, 2 * R, 2, 128, 32, "bf16", 1.0, seed=R)


# ------------------------------------------------------------------- evict
def check_evict(tbs, lens, Hkv, D, block, budget, sink, recent, seed=0, ties=False, patch=None, max_blocks=None):
    c = kc.make_cache(lens, Hkv, block, D, seed=seed, max_blocks=max_blocks)
    if ties:
        c["w"] = np.round(c["w"] * 0.5).astype(np.float32)
    if patch:
        patch(c)
    want = kc.copy_cache(c)
    now, gone = ko.evict(want, want["w"], budget, sink, recent)
    args, _ = on_gpu(c)
    w, offset = dev(c["w"]), torch.full((len(lens),), 5, dtype=torch.int32, device="cuda")
    got = tbs.qsa_kv4_evict(*args, w, budget, sink, recent, offset=offset)
    for x, name in zip(args + [w], NAMES + ("w",)):
        same(x, want[name], name)
    assert np.array_equal(got.cpu().numpy(), now) and np.array_equal(offset.cpu().numpy(), 5 + gone)


@pytest.mark.parametrize("block,D", [(16, 128), (32, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("budget,sink,recent", [(100, 4, 20), (7, 0, 0), (64, 0, 64), (64, 64, 0), (50, 25, 25), (1, 0, 1)])
def test_evict_sizes(tbs, block, D, budget, sink, recent):
    check_evict(tbs, [300, 101, 99, 0, 1, 640], 3, D, block, budget, sink, recent, seed=budget)


def test_evict_ties_and_special_weights(tbs):
    check_evict(tbs, [500, 260], 2, 128, 64, 120, 3, 9, ties=True)

    def patch(c):
        for t, x in ((10, np.nan), (11, np.inf), (12, -np.inf), (13, -1.0), (14, -0.0), (200, np.nan)):
            page, off = ko.place(c, 0, t)
            c["w"][page, :, off] = x
        page = c["table"][1]
        c["w"][page] = 0.0
    check_evict(tbs, [400, 300], 2, 64, 32, 90, 0, 10, patch=patch)


@pytest.mark.parametrize("length,max_blocks", [(5000, None), (9000, 512)])
def test_evict_long(tbs, length, max_blocks):
    """Clusters of several CTAs; of one CTA an item, with more room than tokens."""
    check_evict(tbs, [length], 1, 64, 64, length // 3, 10, 500, max_blocks=max_blocks)
    check_evict(tbs, [length], 1, 128, 64, length - 40, 4, 100, ties=True, max_blocks=max_blocks)
