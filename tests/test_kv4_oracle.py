"""CPU pins of the 4-bit cache's oracle: e2m1 by exhaustion, scales, a
hand-worked append, attention and weights against second, direct computations,
eviction by hand."""
import numpy as np

import kv4_cases as kc
from oracle import kv4_oracle as ko


def packed(n):
    n = np.asarray(n, np.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def test_decode_and_encode():
    n = np.arange(16, dtype=np.uint8)
    x = ko.decode(packed(n))
    assert x.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]
    assert np.array_equal(ko.encode(x), packed(n)) and np.signbit(x[8])
    for lo in range(7):  # midpoints go to the even code, anything past them to the nearer one
        mid = (x[lo] + x[lo + 1]) / 2
        even = lo if lo % 2 == 0 else lo + 1
        for v, want in ((mid, even), (np.nextafter(mid, 0), lo), (np.nextafter(mid, 9), lo + 1)):
            assert ko.encode(np.array([v, -v]))[0] == (want | (want | 8) << 4)
    assert ko.encode(np.array([1e30, -np.inf]))[0] == 0xF7 and ko.encode(np.array([np.nan, -1e-30]))[0] == 0x80


def test_scale_is_the_smallest_bf16():
    assert ko.scale_of(6.0) == 1.0 and ko.scale_of(6.0001) == 1 + 2.0 ** -7 and ko.scale_of(0.0) == 2.0 ** -100
    assert ko.scale_of(np.inf) == ko.scale_of(float(np.finfo(np.float32).max))
    for x in np.exp2(np.random.default_rng(0).uniform(-30, 30, 200)):
        s = ko.scale_of(x)
        assert np.float32(s) == kc.as_bf16(np.array([s], np.float32))[0]
        below = np.array([np.float32(s)]).view(np.uint32) - 0x10000
        assert x <= 6 * s and x > 6 * float(below.view(np.float32)[0])


def test_append_by_hand():
    c = dict(k=np.full((1, 1, 16, 32), 0x11, np.uint8), v=np.full((1, 1, 16, 32), 0x11, np.uint8),
             k_scale=np.full((1, 1, 16), 2.0, np.float32), v_scale=np.full((1, 1, 16), 4.0, np.float32),
             table=np.zeros((1, 1), np.int32), lens=np.array([3], np.int32), n_new=None)
    k, v = np.zeros((1, 2, 1, 64), np.float32), np.zeros((1, 2, 1, 64), np.float32)
    k[0, 0, 0, :3] = [12.0, -3.0, 0.4]      # scale 2: codes 6, -1.5, 0 (0.2)
    v[0, 0, 0, 5] = np.nan
    v[0, 1, 0, :2] = [np.inf, -1.0]
    kb = np.zeros((1, 1, 1, 64))
    ko.append(c, k, v, kb=kb)
    assert c["k_scale"][0, 0, :4].tolist() == [2.0, 2.0, 2.0 ** -100, 2.0]
    assert ko.decode(c["k"])[0, 0, 1, :4].tolist() == [6, -1.5, 0, 0] and (c["k"][0, 0, 0] == 0x11).all()
    assert np.isnan(c["v_scale"][0, 0, 1]) and (c["v"][0, 0, 1] == 0).all()
    assert ko.decode(c["v"])[0, 0, 2, :2].tolist() == [6, 0]
    assert kb[0, 0, 0, :3].tolist() == [(1 + 12 + 0) / 3, (1 - 3) / 3, 1 / 3]
    r = ko.read(c, 3)
    assert r[0, 0, 0, 0].tolist() == [1.0] * 64 and r[0, 0, 1, 0, :2].tolist() == [12, -3]
    assert np.isnan(r[1, 0, 1]).all()


def direct(c, q, scale):
    """Attention with all heads' keys and values laid out, in float64."""
    B, n, Hq, D = q.shape
    R = Hq // c["k"].shape[1]
    out, p_all = np.zeros(q.shape), {}
    for b in range(B):
        L = int(c["lens"][b])
        s = np.arange(L)
        page, off = c["table"][b, s // c["k"].shape[2]], s % c["k"].shape[2]
        k = ko.decode(c["k"])[page, :, off] * c["k_scale"][page, :, off, None]
        v = ko.decode(c["v"])[page, :, off] * c["v_scale"][page, :, off, None]
        for j in range(n):
            if L - n + j < 0:
                continue
            for h in range(Hq):
                x = scale * (k[:L - n + j + 1, h // R] @ q[b, j, h])
                p = np.exp(x - x.max())
                p_all[b, j, h] = p / p.sum()
                out[b, j, h] = p_all[b, j, h] @ v[:L - n + j + 1, h // R]
    return out, p_all


def test_attention_and_weights():
    c = kc.make_cache([40, 5, 17], 2, 16, 64, seed=3)
    q = np.random.default_rng(4).standard_normal((3, 2, 6, 64))
    out, lse, bound = ko.attend(c, q, 0.2)
    want, p = direct(c, q, 0.2)
    assert np.abs(out - want).max() < 1e-12 and (bound > 0).all()
    for decay in (0.0, 0.5):
        new, err = ko.weights(c, q, lse, c["w"], 0.2, decay)
        for b, L in enumerate(c["lens"]):
            for t in range(L):
                page, off = ko.place(c, b, t)
                for h in range(2):
                    old = decay * c["w"][page, h, off] if t < L - 2 and decay else 0.0
                    got = sum(p[b, j, i][t] for j in range(2) for i in range(3 * h, 3 * h + 3) if t < len(p[b, j, i]))
                    assert abs(new[page, h, off] - old - got) < 1e-12 and err[page, h, off] > 0
        # every row's weights add up to one
        if decay == 0:
            assert abs(np.nansum(new) - 3 * 2 * 6) < 1e-9
    ids = np.array([[[[2, 0], [0, -1]]]] * 3, np.int32)
    c2 = kc.make_cache([40, 40, 40], 2, 16, 64, seed=5)
    out, lse, _ = ko.attend(c2, q, 0.2, ids)
    one = dict(c2, lens=np.array([16, 16, 16], np.int32))  # the second row's block alone
    assert np.abs(out[:, 1] - ko.attend(one, q[:, 1:], 0.2)[0][:, 0]).max() < 1e-12


def test_rows_that_are_not_there():
    c = kc.make_cache([3, 0], 1, 16, 64, n_new=[9, 1])
    q = np.ones((2, 4, 2, 64))
    out, lse, _ = ko.attend(c, q, 0.1)
    assert ko.rows_of(c, 0, 4) == [] and ko.rows_of(c, 1, 4) == []
    c["n_new"] = np.array([4, 1], np.int32)
    assert ko.rows_of(c, 0, 4) == [(1, 0), (2, 1), (3, 2)]
    assert (out == 0).all() and np.isneginf(lse).all()


def test_evict_by_hand():
    c = kc.make_cache([9, 4], 1, 16, 64, seed=8)
    page = c["table"][0, 0]
    c["w"][page, 0, :9] = [0, 5, 1, 5, 2, np.nan, 2, 0, 0]
    before = kc.copy_cache(c)
    now, gone = ko.evict(c, c["w"], 5, 1, 1)
    # kept: 0 (first), 8 (last); of the others NaN, then 5 and 5
    for to, src in enumerate([0, 1, 3, 5, 8]):
        for name in ("k", "v", "k_scale", "v_scale", "w"):
            assert np.array_equal(c[name][page, 0, to], before[name][page, 0, src], equal_nan=name not in ("k", "v"))
    assert np.array_equal(c["k"][page, 0, 5:], before["k"][page, 0, 5:])
    assert now.tolist() == [5, 4] and gone.tolist() == [4, 0]
    c = kc.copy_cache(before)
    c["w"][page, 0, :9] = 1.0   # all equal: the lowest slots
    ko.evict(c, c["w"], 4, 0, 2)
    assert all(np.array_equal(c["k"][page, 0, t], before["k"][page, 0, s]) for t, s in enumerate([0, 1, 7, 8]))
