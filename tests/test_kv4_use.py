"""GPU tests of the 4-bit cache's calls as a program makes them: together in a
loop, on streams, in graphs, with strided pages, far pages and indexes outside;
and of what the binding refuses."""
import importlib.util
import os

import numpy as np
import pytest

import kv4_cases as kc
from oracle import kv4_oracle as ko
from test_kv4_parity import NAMES, TINY, UNIT, dev, on_gpu, same, tbs  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def close(got, want, bound, dtype):
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= bound + UNIT[dtype] * (np.abs(want) + bound) + TINY[dtype]).all(), float(err.max())


# ------------------------------------------------------------- all together
@pytest.mark.parametrize("D,dtype,block", [(128, "bf16", 32), (64, "f16", 64)])
def test_a_run_of_them_together(tbs, D, dtype, block):  # noqa: F811
    """Prompts, weights, eviction and steps, each call's results against the
    oracle's on the cache as the GPU has it."""
    rng = np.random.default_rng(1)
    B, Hq, Hkv, n, budget = 2, 8, 2, 70, 48
    c = kc.make_cache([n, n - 13], Hkv, block, D, filled=False, max_blocks=-(-90 // block), n_new=[n, n - 13])
    c["table"] = np.arange(c["table"].size, dtype=np.int32)[::-1].reshape(B, -1).copy()
    pages = c["table"].size
    for name, shape in (("k", (pages, Hkv, block, D // 2)), ("v", (pages, Hkv, block, D // 2))):
        c[name] = np.zeros(shape, np.uint8)
    for name in ("k_scale", "v_scale", "w"):
        c[name] = np.full((pages, Hkv, block), np.nan, np.float32)
    cos, sin = kc.angles(120, D)
    args, nn = on_gpu(c)
    w, offset = dev(c["w"]), torch.zeros(B, dtype=torch.int32, device="cuda")
    gone = np.zeros(B, np.int32)
    terms = 3 if dtype == "f16" else 2

    def pull():
        for t, name in zip(args, NAMES):
            c[name] = t.float().cpu().numpy() if name.endswith("scale") else t.cpu().numpy()

    def rows(x, name):
        return kc.ROUND[dtype](x), name

    for step in range(12):
        m = n if step == 0 else 1
        if step:
            c["n_new"] = nn = None
            args[5] += 1
            c["lens"] = args[5].cpu().numpy()
        x = kc.ROUND[dtype](rng.standard_normal((B, m, Hq + 2 * Hkv, D)))
        g = dev(x, dtype)
        kb, wkb = torch.zeros((B, Hkv, c["table"].shape[1], D), dtype=torch.float16, device="cuda"), None
        q = tbs.qsa_kv4_append(g[:, :, Hq:Hq + Hkv], g[:, :, Hq + Hkv:], *args, cos=dev(cos), sin=dev(sin), n_new=nn,
                               offset=offset, q=g[:, :, :Hq], kb=kb)
        wq = ko.append(c, x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], cos, sin, q=x[:, :, :Hq], kb=wkb, offset=gone)
        for t, name in zip(args, NAMES):
            same(t, c[name], (step, name))
        assert torch.equal(q.cpu(), torch.from_numpy(wq).to(q.dtype))
        lse = torch.zeros((B, m, Hq), device="cuda")
        out = tbs.qsa_kv4_attend(q, *args, n_new=nn, lse=lse)
        qn = q.double().cpu().numpy()
        want, _, bound = ko.attend(c, qn, D ** -0.5, terms=terms)
        close(out, want, bound, dtype)
        c["w"] = w.cpu().numpy()
        tbs.qsa_kv4_weights(q, lse, *args, w, n_new=nn, decay=0.0 if step == 0 else 0.9)
        want, bound = ko.weights(c, qn, lse.cpu().numpy(), c["w"], D ** -0.5, 0.0 if step == 0 else 0.9, terms=terms)
        got = w.cpu().numpy().astype(np.float64)
        ok = ~np.isnan(want)
        assert np.array_equal(np.isnan(got), ~ok) and (np.abs(got - want)[ok] <= bound[ok]).all()
        if step % 5 == 0:
            c["w"] = w.cpu().numpy()
            args[5] = tbs.qsa_kv4_evict(*args, w, budget, 2, 10, offset=offset)
            now, went = ko.evict(c, c["w"], budget, 2, 10)
            gone += went
            c["lens"] = now.astype(np.int32)
            for t, name in zip(args + [w], NAMES + ("w",)):
                same(t, c[name], (step, name))
            assert np.array_equal(offset.cpu().numpy(), gone)
    assert gone.max() > n - budget


def test_example(tbs):  # noqa: F811
    spec = importlib.util.spec_from_file_location("paged4_decode", os.path.join(ROOT, "examples", "paged4_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    layer, q, out = m.decode(2, 300, 40, budget=128, slack=8, Hq=8, Hkv=2, D=64, block=32)
    torch.cuda.synchronize()
    # 300 -> 128, then 8 more and back again, every 8 steps
    assert layer.lens.tolist() == [128, 128] and layer.offset.tolist() == [212, 212]
    c = dict(k=layer.k.cpu().numpy(), v=layer.v.cpu().numpy(), k_scale=layer.k_scale.float().cpu().numpy(),
             v_scale=layer.v_scale.float().cpu().numpy(), table=layer.table.cpu().numpy(),
             lens=layer.lens.cpu().numpy(), n_new=None)
    got = tbs.qsa_kv4_attend(q, *layer.cache())
    want, _, bound = ko.attend(c, q.double().cpu().numpy(), 0.125, terms=2)
    close(got, want, bound, "bf16")
    w = layer.weights.cpu().numpy()[layer.table.cpu().numpy()].transpose(0, 2, 1, 3).reshape(2, 2, -1)[:, :, :128]
    assert np.isfinite(w).all() and (w >= 0).all() and out.shape == q.shape


# --------------------------------------------------------- streams, graphs
def calls(tbs, args, q, kv, w, out, lse, ws, ews, lens_out, offset, cos):  # noqa: F811
    tbs.qsa_kv4_append(kv, kv, *args, cos=cos, sin=cos, offset=offset)
    tbs.qsa_kv4_attend(q, *args, out=out, lse=lse, workspace=ws)
    tbs.qsa_kv4_weights(q, lse, *args, w)
    tbs.qsa_kv4_evict(*args, w, 200, 3, 20, offset=offset, lens_out=lens_out, workspace=ews)
    return tbs.qsa_kv4_read(*args[:5], lens_out, n=4)


def problem(tbs, seed, D=128, lens=(500, 64)):  # noqa: F811
    c = kc.make_cache(list(lens), 2, 64, D, seed=seed)
    args, _ = on_gpu(c)
    torch.manual_seed(seed)
    B = len(lens)
    q = torch.randn((B, 1, 8, D), device="cuda").half()
    kv = torch.randn((B, 1, 2, D), device="cuda").half()
    return (args, q, kv, dev(c["w"]), torch.zeros_like(q), torch.zeros((B, 1, 8), device="cuda"),
            torch.zeros(tbs.qsa_kv4_attend_workspace_bytes(B, 1, 8, 2, D), dtype=torch.uint8, device="cuda"),
            torch.zeros(tbs.qsa_kv4_evict_workspace_bytes(B, 2, 200), dtype=torch.uint8, device="cuda"),
            torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda"),
            torch.rand((9001, D // 2), device="cuda"))


def state(p):
    args, q, kv, w, out, lse, ws, ews, lens_out, offset, cos = p
    return [t.view(torch.uint8).clone() for t in (*args[:4], w, out, lse, lens_out, offset)]


@pytest.mark.parametrize("D", [64, 128])
def test_on_another_stream(tbs, D):  # noqa: F811
    a, b = problem(tbs, 3, D), problem(tbs, 3, D)
    want = calls(tbs, *a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = calls(tbs, *b)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(state(a), state(b)))
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_two_streams_at_once(tbs):  # noqa: F811
    """The same calls on different data, workspaces apart, side by side."""
    alone = []
    for seed in (5, 6):
        p = problem(tbs, seed, lens=(9000, 3000))
        for _ in range(4):
            calls(tbs, *p)
        torch.cuda.synchronize()
        alone.append(state(p))
    ps = [problem(tbs, seed, lens=(9000, 3000)) for seed in (5, 6)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(4):
        for p, s in zip(ps, streams):
            with torch.cuda.stream(s):
                calls(tbs, *p)
    torch.cuda.synchronize()
    for p, want in zip(ps, alone):
        assert all(torch.equal(x, y) for x, y in zip(state(p), want))


@pytest.mark.parametrize("D", [64, 128])
def test_in_a_graph(tbs, D):  # noqa: F811
    """Captured once, replayed on other data in the same buffers; a second graph
    shares the workspaces."""
    p, ref = problem(tbs, 8, D), problem(tbs, 9, D)
    calls(tbs, *p)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls(tbs, *p)
        graphs.append(g)
    fresh = problem(tbs, 9, D)
    for x, y in zip(p[0], fresh[0]):
        x.copy_(y)
    for i in (1, 2, 3, 8, 9, 10):
        p[i].copy_(fresh[i])
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _ in range(2):
        calls(tbs, *ref)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(state(p), state(ref)))


# ----------------------------------------------------- layouts and indexes
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f16")])
@pytest.mark.parametrize("n,Hq", [(1, 4), (130, 16)])
def test_strided_pages_and_rows(tbs, D, dtype, n, Hq):  # noqa: F811
    """Pages with room between them, queries of a wider projection."""
    lens = [n + 90, n + 1]
    c = kc.make_cache(lens, 1, 32, D, seed=2)
    if n > 1:
        kc.roomy(c, 2 * n * Hq)
    args, _ = on_gpu(c)
    for i in (0, 1):
        wide = torch.full((args[i].shape[0], 3, 32, D // 2), 0xFF, dtype=torch.uint8, device="cuda")
        wide[:, 1:2] = args[i]
        args[i] = wide[:, 1:2]
    rng = np.random.default_rng(3)
    q = kc.ROUND[dtype](rng.standard_normal((2, n, Hq + 2, D)))
    g = dev(q, dtype)
    lse = torch.zeros((2, n, Hq), device="cuda")
    out = tbs.qsa_kv4_attend(g[:, :, :Hq], *args, lse=lse)
    want, wlse, bound = ko.attend(c, q[:, :, :Hq], D ** -0.5, terms=3 if dtype == "f16" else 2)
    close(out, want, bound, dtype)
    w = dev(c["w"])
    tbs.qsa_kv4_weights(g[:, :, :Hq], lse, *args, w)
    ww, wb = ko.weights(c, q[:, :, :Hq], lse.cpu().numpy(), c["w"], D ** -0.5, 1.0, terms=3 if dtype == "f16" else 2)
    ok = ~np.isnan(ww)
    assert (np.abs(w.cpu().numpy() - ww)[ok] <= wb[ok]).all()
    now, _ = ko.evict(c, ww32 := w.cpu().numpy(), 40, 1, 7)
    assert np.array_equal(tbs.qsa_kv4_evict(*args, w, 40, 1, 7).cpu().numpy(), now)
    same(args[0].contiguous(), c["k"], "k")
    same(args[1].contiguous(), c["v"], "v")
    same(w, ww32, "w")
    x = dev(kc.ROUND[dtype](rng.standard_normal((2, 3, 2, D))), dtype)
    lens_t = dev(now.astype(np.int32))
    tbs.qsa_kv4_append(x[:, :, :1], x[:, :, 1:], *args[:5], lens_t)
    c["lens"] = now.astype(np.int32)
    ko.append(c, x[:, :, :1].float().cpu().numpy(), x[:, :, 1:].float().cpu().numpy())
    same(args[0].contiguous(), c["k"], "k")
    k, _ = tbs.qsa_kv4_read(*args[:5], lens_t, n=3)
    same(k, torch.from_numpy(ko.read(c, 3)[0].astype(np.float32)).half().float().numpy(), "read")


def test_offsets_past_32_bits(tbs):  # noqa: F811
    """Pages behind 2^32 bytes of a cache."""
    Hkv, block, D = 8, 128, 128
    pages = (1 << 32) // (Hkv * block * D // 2) + 40
    k = torch.empty((pages, Hkv, block, D // 2), dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    ks = torch.empty((pages, Hkv, block), dtype=torch.bfloat16, device="cuda")
    vs, w = torch.empty_like(ks), torch.empty((pages, Hkv, block), device="cuda")
    c = kc.roomy(kc.make_cache([300], Hkv, block, D, seed=1, filled=False), 129 * 2 * Hkv)
    near, _ = on_gpu(c)
    table, lens = dev(c["table"] + (pages - 20)), dev(c["lens"])
    far = [k, v, ks, vs, table, lens]
    x = torch.randn((1, 300, 2 * Hkv, D), device="cuda").half()
    q = torch.randn((1, 1, Hkv, D), device="cuda").half()
    got = []
    for args, weights in ((far, w), (near, torch.empty(c["w"].shape, device="cuda"))):
        tbs.qsa_kv4_append(x[:, :, :Hkv], x[:, :, Hkv:], *args)
        lse = torch.zeros((1, 1, Hkv), device="cuda")
        out = [tbs.qsa_kv4_attend(q, *args, lse=lse), tbs.qsa_kv4_attend(x[:, -129:, :Hkv].repeat(1, 1, 2, 1), *args)]
        tbs.qsa_kv4_weights(q, lse, *args, weights, decay=0.0)
        args[5] = tbs.qsa_kv4_evict(*args, weights, 150, 2, 30)
        got.append(out + list(tbs.qsa_kv4_read(*args, n=150)))
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,Hq", [(1, 4), (3, 8), (128, 16)])
def test_longer_than_the_page_table(tbs, D, n, Hq):  # noqa: F811
    """400 tokens, a table for 320: what the table holds, and a record of it."""
    c = kc.make_cache([400], 1, 64, D, seed=n)
    c["table"] = np.ascontiguousarray(c["table"][:, :5])
    args, _ = on_gpu(c)
    q = kc.as_f16(np.random.default_rng(1).standard_normal((1, n, Hq, D)))
    lse = torch.zeros((1, n, Hq), device="cuda")
    got = tbs.qsa_kv4_attend(dev(q, "f16"), *args, lse=lse)
    assert tbs.qsa_device_status(clear=True) == (1, 32)
    want, _, bound = ko.attend(c, q, D ** -0.5, np.array([[[[0, 1, 2, 3, 4]] * n]], np.int32))
    close(got, want, bound, "f16")
    w = dev(c["w"])
    tbs.qsa_kv4_weights(dev(q, "f16"), lse, *args, w)
    assert tbs.qsa_device_status(clear=True) == (1, 32)
    now = tbs.qsa_kv4_evict(*args, w, 350, 0, 0)
    assert tbs.qsa_device_status(clear=True) == (1, 32) and now.tolist() == [320]
    x = torch.zeros((1, 1, 1, D), dtype=torch.float16, device="cuda")
    before = [t.clone() for t in args]
    tbs.qsa_kv4_append(x, x, *args)
    assert tbs.qsa_device_status(clear=True) == (1, 32)
    k, _ = tbs.qsa_kv4_read(*args, n=1)
    assert tbs.qsa_device_status(clear=True) == (1, 32) and (k == 0).all()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(args, before))


@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_longer_than_the_page_table(tbs, D):  # noqa: F811
    """6,000 tokens, a table for 5,120."""
    c = kc.make_cache([6000], 1, 128, D, seed=4)
    c["table"] = np.ascontiguousarray(c["table"][:, :40])
    args, _ = on_gpu(c)
    q = kc.as_f16(np.random.default_rng(1).standard_normal((1, 128, 16, D)))
    got = tbs.qsa_kv4_attend(dev(q, "f16"), *args)
    assert "kv4_attend_many_kernel" in tbs.qsa_arm() and tbs.qsa_device_status(clear=True) == (1, 32)
    want, _, bound = ko.attend(c, q[:, -3:], D ** -0.5, np.array([[[list(range(40))] * 3]], np.int32))
    close(got[:, -3:], want, bound, "f16")


@pytest.mark.parametrize("block", [16, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_pages_outside(tbs, block, D):  # noqa: F811
    """One page id outside the cache, at each of the blocks in turn."""
    blocks = 256 // block + 2
    L = blocks * block - 3
    c = kc.roomy(kc.make_cache([L], 1, block, D, seed=block), 130 * 16)
    args, _ = on_gpu(c)
    q = kc.as_f16(np.random.default_rng(2).standard_normal((1, 130, 16, D)))
    for i in range(blocks):
        table = args[4].clone()
        table[0, i] = -1 if i % 2 else c["k"].shape[0]
        cache = [*args[:4], table, args[5]]
        rest = [k for k in range(blocks) if k != i]
        lse = torch.zeros((1, 1, 4), device="cuda")
        got = tbs.qsa_kv4_attend(dev(q[:, :1, :4], "f16"), *cache, lse=lse)
        assert tbs.qsa_device_status(clear=True) == (1, 32), i
        want, wlse, bound = ko.attend(c, q[:, :1, :4], D ** -0.5, np.array([[[rest]]], np.int32))
        close(got, want, bound, "f16")
        w = dev(c["w"])
        tbs.qsa_kv4_weights(dev(q[:, :1, :4], "f16"), lse, *cache, w)
        assert tbs.qsa_device_status(clear=True) == (1, 32), i
        page = c["table"][0, i]
        same(w[page], c["w"][page], "weights of the page that was not named")
        if i in (0, blocks - 1):
            got = tbs.qsa_kv4_attend(dev(q, "f16"), *cache)
            assert tbs.qsa_device_status(clear=True) == (1, 32), i
            want, _, bound = ko.attend(c, q[:, :, :2], D ** -0.5, np.array([[[rest]] * 130], np.int32).reshape(1, 1, 130, -1))
            heads = got.reshape(1, 130, 16, D)[:, :, :2]
            close(heads, want, bound, "f16")
        copies = [t.clone() for t in args[:4]]
        tbs.qsa_kv4_evict(*copies, table, args[5], dev(c["w"]), L - 5, 0, 3)
        assert tbs.qsa_device_status(clear=True) == (1, 32), i
        for got_t, was in zip(copies, args):
            assert torch.equal(got_t[page].view(torch.uint8), was[page].view(torch.uint8))


def test_positions_outside_the_angles(tbs):  # noqa: F811
    c = kc.make_cache([200], 1, 64, 128, seed=17)
    args, _ = on_gpu(c)
    kv = torch.randn((1, 3, 1, 128), device="cuda").half()
    before = [t.clone() for t in args[:4]]
    cos = torch.rand((230, 64), device="cuda")
    for off in (-1, 1000, 2 ** 31 - 1):
        offset = torch.tensor([off], dtype=torch.int32, device="cuda")
        q = tbs.qsa_kv4_append(kv, kv, *args, cos=cos, sin=cos, offset=offset, q=kv)
        assert tbs.qsa_device_status(clear=True) == (1, 32), off
        assert (q == 0).all() and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(args, before))
    # the last of three tokens past the tables: the first two are stored
    tbs.qsa_kv4_append(kv, kv, *args, cos=cos, sin=cos, offset=torch.tensor([31], dtype=torch.int32, device="cuda"))
    assert tbs.qsa_device_status(clear=True) == (1, 32)
    page = int(c["table"][0, 3])
    assert torch.equal(args[0][page, 0, 7], before[0][page, 0, 7])
    assert not torch.equal(args[0][page, 0, 5:7], before[0][page, 0, 5:7])


# ---------------------------------------------------------------- refusals
def test_binding_refuses_wrong_tensors(tbs):  # noqa: F811
    c = kc.make_cache([100, 30], 2, 32, 64, seed=17)
    args, _ = on_gpu(c)
    q = torch.zeros((2, 3, 4, 64), dtype=torch.float16, device="cuda")
    kv = torch.zeros((2, 3, 2, 64), dtype=torch.float16, device="cuda")
    w, lse = dev(c["w"]), torch.zeros((2, 3, 4), device="cuda")

    def bad(i, t):
        a = list(args)
        a[i] = t
        return a
    wrong = [bad(0, args[0].view(torch.int8)), bad(1, args[1][:, :1]), bad(1, args[1][:-1]), bad(0, args[0].transpose(2, 3)),
             bad(2, args[2].float()), bad(2, args[2].half()), bad(3, args[3][:-1]), bad(3, args[3][..., 0]),
             bad(4, args[4].long()), bad(4, args[4][:1]), bad(5, args[5].long()), bad(5, args[5].cpu()), bad(2, args[2].cpu())]
    for a in wrong:
        for call in (lambda: tbs.qsa_kv4_attend(q, *a), lambda: tbs.qsa_kv4_append(kv, kv, *a),
                     lambda: tbs.qsa_kv4_read(*a, n=1), lambda: tbs.qsa_kv4_weights(q, lse, *a, w),
                     lambda: tbs.qsa_kv4_evict(*a, w, 8)):
            with pytest.raises(ValueError):
                call()
    ids = torch.zeros((2, 1, 3, 4), dtype=torch.int32, device="cuda")
    for kw in (dict(ids=ids.long()), dict(ids=ids[:, :, :2]), dict(out=q.bfloat16()), dict(lse=lse[..., 0]),
               dict(n_new=args[5][:1]), dict(workspace=torch.zeros(8, device="cuda"))):
        with pytest.raises(ValueError):
            tbs.qsa_kv4_attend(q, *args, **kw)
    for x in (q.float(), q[:1], q[..., :32], q[0], q.cpu()):
        with pytest.raises(ValueError):
            tbs.qsa_kv4_attend(x, *args)
        with pytest.raises(ValueError):
            tbs.qsa_kv4_weights(x, lse, *args, w)
    for kw in (dict(offset=args[5].long()), dict(offset=args[5][:1]), dict(kb=q), dict(n_new=args[5].cpu()), dict(q_out=q)):
        with pytest.raises(ValueError):
            tbs.qsa_kv4_append(kv, kv, *args, **kw)
    for kw in (dict(n=-1), dict(n=2 ** 31), dict(n=1, dtype=torch.float32), dict(n=1, k_out=kv), dict(n=3, v_out=kv.bfloat16())):
        with pytest.raises(ValueError):
            tbs.qsa_kv4_read(*args, **kw)
    for x, y in ((lse[:, :2], w), (lse.half(), w), (lse, w[:1]), (lse, w.half()), (lse, w[..., 0]), (lse.cpu(), w)):
        with pytest.raises(ValueError):
            tbs.qsa_kv4_weights(q, x, *args, y)
    for kw in (dict(budget=-1), dict(budget=8, sink=-1), dict(budget=2 ** 31), dict(budget=8, offset=args[5].long()),
               dict(budget=8, lens_out=args[5][:1]), dict(budget=8, workspace=torch.zeros(8, device="cuda"))):
        with pytest.raises(ValueError):
            tbs.qsa_kv4_evict(*args, w, **kw)
    for kw in (dict(budget=0), dict(budget=8, sink=5, recent=4), dict(budget=8, lens_out=args[5]),
               dict(budget=8, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(tbs.QsaError):
            tbs.qsa_kv4_evict(*args, w, **kw)
    with pytest.raises(tbs.QsaError):
        tbs.qsa_kv4_weights(q, lse, *args, w, decay=-1.0)
    with pytest.raises(tbs.QsaError):
        tbs.qsa_kv4_attend(q, *args, scale=float("inf"))
    with pytest.raises(tbs.QsaError):   # pages that are not on 32 bytes
        raw = torch.zeros(args[0].numel() + 16, dtype=torch.uint8, device="cuda")[16:].view(args[0].shape)
        tbs.qsa_kv4_attend(q, raw, *args[1:])
    with pytest.raises(TypeError):
        tbs.qsa_kv4_read(*args, n="1")
    assert tbs.qsa_kv4_attend(q[:, :0], *args).shape == (2, 0, 4, 64)
    assert tbs.qsa_kv4_read(*args, n=0)[0].shape == (2, 0, 2, 64)


def test_arm_names_the_kernels(tbs):  # noqa: F811
    p = problem(tbs, 1)
    args, q, kv, w, lse = p[0], p[1], p[2], p[3], p[5]
    for call, name in ((lambda: tbs.qsa_kv4_append(kv, kv, *args), "1 launch: kv4_append_kernel"),
                       (lambda: tbs.qsa_kv4_read(*args, n=1), "1 launch: kv4_read_kernel"),
                       (lambda: tbs.qsa_kv4_attend(q, *args), "1 launch: kv4_attend_kernel"),
                       (lambda: tbs.qsa_kv4_weights(q, lse, *args, w), "1 launch: kv4_weights_kernel"),
                       (lambda: tbs.qsa_kv4_evict(*args, w, 100), "1 launch: kv4_evict_kernel")):
        call()
        assert name in tbs.qsa_arm(), tbs.qsa_arm()
    args, q = problem(tbs, 1, lens=(3000, 5))[:2]  # items long enough to be split and joined
    tbs.qsa_kv4_attend(q, *args)
    assert "2 launches: kv4_attend_kernel -> kv_combine_kernel" in tbs.qsa_arm()
