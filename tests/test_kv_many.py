"""GPU parity of the cache attention of many rows (chunks of prompts: 128 rows
and more on a KV head, 2,048 and more in all) with the CPU oracle, within the same derived bound as
the other forms: its probabilities are nearer than theirs."""
import numpy as np
import pytest

import kv_cases as kc
from oracle import kv_oracle as ko
from test_kv_parity import TINY, UNIT, check_attend, check_rows, dev, on_gpu, tbs  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def run(tbs, c, q, dtype, seed=0, count=60, **kw):
    """The call on queries q, repeated, and some of its rows against the oracle."""
    args, nn = on_gpu(c)
    g = dev(q, dtype)
    lse = torch.full(q.shape[:3], 7.0, dtype=torch.float32, device="cuda")
    out = tbs.qsa_kv_attend(g, *args, n_new=nn, lse=lse, **kw)
    assert "kv_attend_many_kernel" in tbs.qsa_arm()
    for _ in range(5):
        assert torch.equal(tbs.qsa_kv_attend(g, *args, n_new=nn, **kw), out)
    rng = np.random.default_rng(seed)
    B, n, Hq = q.shape[:3]
    at = [(int(rng.integers(B)), int(rng.integers(n)), int(rng.integers(Hq))) for _ in range(count)]
    at += [(b, j, h) for b in range(B) for j in (0, n - 1) for h in (0, Hq - 1)][:40]
    check_rows(c, q, out, lse, dtype, at)
    return out, lse


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,block", [(64, 16), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("n,R,Hkv", [(130, 1, 2), (67, 5, 1), (33, 8, 2), (9, 32, 1), (26, 5, 2)])
def test_many_head_groups(tbs, dtype, D, block, n, R, Hkv):  # noqa: F811
    """Row tiles that are full, that end inside a tile and that R does not divide."""
    B = -(-2048 // (n * R * Hkv))
    c = kc.make_long_cache([n + 211, n, n + 3, 2 * n][:B] + [n + 1] * (B - 4), Hkv, block, D, seed=n)
    q = kc.ROUND[dtype](np.random.default_rng(R).standard_normal((B, n, Hkv * R, D)))
    run(tbs, c, q, dtype, seed=n)


@pytest.mark.parametrize("length", [128, 129, 255, 256, 257, 400])
def test_many_every_row(tbs, length):  # noqa: F811
    """Rows from the first token on: every row of a call against the oracle."""
    c = kc.make_cache([length, 128], 1, 32, 64, seed=length)
    check_attend(tbs, c, 128, 8, "f16" if length % 2 else "bf16", seed=length)


def test_many_ragged(tbs):  # noqa: F811
    """Sequences with fewer new tokens than rows, without any, shorter than n."""
    lens = [300, 40, 0, 513, 130, 7]
    c = kc.make_cache(lens, 1, 64, 64, seed=2, n_new=[70, 70, 70, 0, 1, 33])
    out, lse = check_attend(tbs, c, 70, 5, "f16")
    assert (out[2] == 0).all() and (out[3] == 0).all() and torch.isneginf(lse[3]).all()
    assert (out[4, 1:] == 0).all() and (out[0, 69] != 0).any()
    # 40 tokens, 70 of them new: the first 30 rows stand before position 0
    assert (out[1, :30] == 0).all() and (out[1, 30] != 0).any()


@pytest.mark.parametrize("lens,n,Hkv,R,D,block,dtype", [
    ([9000, 5001], 300, 4, 4, 64, 32, "f16"), ([20011], 520, 2, 8, 128, 64, "f16"),
    ([700] * 9, 257, 8, 2, 128, 16, "bf16"), ([3001, 129, 900] * 4, 129, 2, 3, 64, 64, "f16"),
    ([16390], 16, 8, 16, 128, 128, "bf16"), ([131, 140] * 40, 64, 2, 2, 64, 64, "f16")])
def test_many_tiles(tbs, lens, n, Hkv, R, D, block, dtype):  # noqa: F811
    """Items that begin, lie and end inside a CTA's share, items that span CTAs."""
    c = kc.make_long_cache(lens, Hkv, block, D, seed=R)
    q = kc.ROUND[dtype](np.random.default_rng(n).standard_normal((len(lens), n, Hkv * R, D)))
    run(tbs, c, q, dtype, seed=R)


@pytest.mark.parametrize("amp", [0.0, 1e-3, 30.0])
@pytest.mark.parametrize("scale", [0.125, -0.3])
def test_many_score_ranges(tbs, amp, scale):  # noqa: F811
    """Equal scores, nearly equal ones, one token above all others; blocks of
    very different scales; a negative scale."""
    c = kc.make_cache([500], 1, 64, 64, seed=11, spread=3.0)
    check_attend(tbs, c, 130, 16, "f16", amp=amp, scale=scale)
    check_attend(tbs, c, 130, 16, "bf16", amp=amp, scale=scale)


def test_many_rows_of_different_size(tbs):  # noqa: F811
    def rows(q):
        q[0, 0] *= 2.0 ** -12
        q[0, 1] *= 2.0 ** 6
        q[0, 2] = 0.0
        q[0, 3, :, 1:] = 0.0
    c = kc.make_cache([300], 1, 64, 128, seed=12)
    check_attend(tbs, c, 64, 32, "f16", rows=rows)

    def far(q):  # bf16 far outside the range of fp32 products of codes
        rows(q)
        q[0, 4] *= 2.0 ** 120
        q[0, 5] *= 2.0 ** -100
    check_attend(tbs, c, 64, 32, "bf16", rows=far)


def test_many_nan_is_kept_to_what_sees_it(tbs):  # noqa: F811
    c = kc.make_cache([140], 1, 32, 64, seed=13)
    t = c["table"][0]
    c["v"][t[4], 0, 5, 9] = 0x7F       # position 133: rows at 133 and later, dimension 9
    c["k"][t[4], 0, 8, 3] = 0xFF       # position 136: rows at 136 and later, every dimension
    out, lse = check_attend(tbs, c, 70, 30, "f16")
    got = torch.isnan(out[0]).any(1).cpu().numpy()  # [n, D]
    for j in range(70):
        p = 70 + j
        assert got[j].all() if p >= 136 else (got[j].nonzero()[0].tolist() == ([9] if p >= 133 else []))

    c = kc.make_cache([440], 1, 32, 64, seed=14)
    c["v"][c["table"][0][2], 0, 5, 9] = 0xFF  # seen by every row
    out, _ = check_attend(tbs, c, 70, 30, "bf16")
    assert torch.isnan(out[:, :, :, 9]).all() and not torch.isnan(out[:, :, :, 10]).any()

    def rows(q):
        q[0, 3, 0, 0] = np.nan
    c = kc.make_cache([140], 1, 32, 64, seed=13)
    check_attend(tbs, c, 70, 30, "f16", rows=rows)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_many_infinite_query(tbs, dtype):  # noqa: F811
    """An infinite query makes its row NaN, whatever the keys' signs."""
    c = kc.make_cache([200], 1, 64, 64, seed=15)
    for p in c["table"][0]:
        c["k"][p, 0, :, 0] |= 0x80  # every key negative there
    q = torch.randn((1, 130, 16, 64), device="cuda").to(getattr(torch, {"f16": "float16", "bf16": "bfloat16"}[dtype]))
    q[0, 7, :, 0] = float("inf")
    q[0, 9, :, 3] = -float("inf")
    args, _ = on_gpu(c)
    bad = torch.isnan(tbs.qsa_kv_attend(q, *args)).all(-1)[0].all(-1).nonzero().flatten().tolist()
    assert bad == [7, 9]


def test_many_pages_outside_are_left_out(tbs):  # noqa: F811
    """A page id outside the cache, in blocks of 16: recorded, its tokens not
    there for any row."""
    c = kc.make_cache([300], 1, 16, 64, seed=16)
    args, _ = on_gpu(c)
    q = kc.as_f16(np.random.default_rng(1).standard_normal((1, 128, 16, 64)))
    table = args[4].clone()
    table[0, 3] = 1 << 20
    table[0, 8] = -1
    got = tbs.qsa_kv_attend(dev(q, "f16"), *args[:4], table, args[5])
    assert tbs.qsa_device_status(clear=True) == (1, 32)
    listed = [i for i in range(19) if i not in (3, 8)]
    ids = np.array([[[listed] * 128]], np.int32)
    want, _, bound = ko.attend(c, q, 0.125, ids)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= bound + UNIT["f16"] * (np.abs(want) + bound) + TINY["f16"]).all()


def test_many_strides_and_streams(tbs):  # noqa: F811
    """Queries inside a wider projection, one row for every head; a given
    output and workspace; another stream; a graph."""
    c = kc.make_cache([350, 270], 2, 32, 64, seed=30)
    args, _ = on_gpu(c)
    wide = torch.randn((2, 140, 16, 64), dtype=torch.float16, device="cuda")
    ws = torch.full((tbs.qsa_kv_attend_workspace_bytes(2, 140, 8, 2, 64),), 255, dtype=torch.uint8, device="cuda")
    for q in (wide[:, :, 5:13], wide[:, :, :1].expand(2, 140, 8, 64), wide[:1, :, :8].expand(2, 140, 8, 64)):
        want = tbs.qsa_kv_attend(q.contiguous(), *args)
        out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        assert tbs.qsa_kv_attend(q, *args, out=out, workspace=ws) is out
        assert "kv_attend_many_kernel" in tbs.qsa_arm()
        assert torch.equal(out, want)
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            there = tbs.qsa_kv_attend(q, *args)
        other.synchronize()
        assert torch.equal(there, want)
    q = wide[:, :, :8].clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        tbs.qsa_kv_attend(q, *args, out=out, workspace=ws)
    for _ in range(3):
        q.normal_()
        graph.replay()
        assert torch.equal(out, tbs.qsa_kv_attend(q, *args))


def test_many_and_few_rows_agree(tbs):  # noqa: F811
    """The same rows in one call of many and in calls of one token each."""
    c = kc.make_long_cache([1500], 2, 64, 128, seed=40)
    args, _ = on_gpu(c)
    q = torch.randn((1, 64, 32, 128), dtype=torch.float16, device="cuda")
    many = tbs.qsa_kv_attend(q, *args)
    assert "kv_attend_many_kernel" in tbs.qsa_arm()
    lens = args[5].clone()
    for j in (0, 31, 63):
        lens[0] = 1500 - 63 + j
        one = tbs.qsa_kv_attend(q[:, j:j + 1], *args[:5], lens)
        diff = (one.double() - many[:, j:j + 1].double()).norm() / one.double().norm()
        assert float(diff) <= 4 * UNIT["f16"]


def test_many_offsets_past_32_bits(tbs):  # noqa: F811
    """Pages behind 2^32 bytes of a cache."""
    Hkv, block, D = 8, 128, 128
    pages = (1 << 32) // (Hkv * block * D) + 10
    c = kc.make_cache([300], Hkv, block, D, seed=1)
    args, _ = on_gpu(c)
    used = args[0].shape[0]
    far = []
    for t in args[:4]:
        f = torch.zeros((pages, *t.shape[1:]), dtype=t.dtype, device="cuda")
        f[pages - used:] = t
        far.append(f)
    table = torch.where(args[4] >= 0, args[4] + pages - used, args[4])
    q = torch.randn((1, 128, 2 * Hkv, D), dtype=torch.float16, device="cuda")
    assert torch.equal(tbs.qsa_kv_attend(q, *far, table, args[5]), tbs.qsa_kv_attend(q, *args))
    assert "kv_attend_many_kernel" in tbs.qsa_arm()


@pytest.mark.parametrize("lens,n,Hkv,R,D", [([60] * 40 + [6000] * 6, 1, 4, 4, 64), ([9000] + [3] * 300, 1, 2, 2, 128),
                                            ([100, 2000] * 20, 3, 2, 5, 64), ([1] * 700 + [129], 1, 1, 8, 64)])
def test_mixed_lengths(tbs, lens, n, Hkv, R, D):  # noqa: F811
    """Short and long sequences in one call of few rows: shares that begin or
    end in the cost of an item, or hold nothing else."""
    c = kc.make_long_cache(lens, Hkv, 32, D, seed=R)
    q = kc.ROUND["f16"](np.random.default_rng(n).standard_normal((len(lens), n, Hkv * R, D)))
    args, _ = on_gpu(c)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")
    out = tbs.qsa_kv_attend(dev(q, "f16"), *args, lse=lse)
    assert "kv_attend_kernel" in tbs.qsa_arm()
    assert torch.equal(tbs.qsa_kv_attend(dev(q, "f16"), *args), out)
    rng = np.random.default_rng(7)
    at = [(int(rng.integers(len(lens))), int(rng.integers(n)), int(rng.integers(Hkv * R))) for _ in range(80)]
    check_rows(c, q, out, lse, "f16", at + [(len(lens) - 1, 0, 0), (0, 0, 0)])
