"""CPU pins of the paged-cache oracle: e4m3 by exhaustion and against closed
forms, scales, rotation, a hand-worked append and attention against a second,
direct computation in exact rationals or float64."""
import math
from fractions import Fraction

import numpy as np
import pytest

import kv_cases as kc
from oracle import kv_oracle as ko


def test_decode_table():
    assert ko.E4M3[0] == 0 and ko.E4M3[1] == 2.0 ** -9 and ko.E4M3[8] == 2.0 ** -6 and ko.E4M3[0x38] == 1.0
    assert ko.E4M3[0x7E] == 448 and np.isnan(ko.E4M3[0x7F]) and np.isnan(ko.E4M3[0xFF])
    assert np.array_equal(ko.E4M3[128:255], -ko.E4M3[:127])
    assert (np.diff(ko.E4M3[:127]) > 0).all()


def test_encode_is_nearest_even():
    codes = np.array([c for c in range(256) if (c & 0x7F) != 0x7F], np.uint8)
    assert np.array_equal(ko.encode(ko.E4M3[codes]), codes)
    for c in range(126):  # midpoints go to the even code, anything past them to the nearer one
        lo, hi = ko.E4M3[c], ko.E4M3[c + 1]
        mid = (lo + hi) / 2
        assert ko.encode(mid) == (c if c % 2 == 0 else c + 1)
        assert ko.encode(np.nextafter(mid, 0)) == c and ko.encode(np.nextafter(mid, 1e9)) == c + 1
    assert ko.encode(1e30) == 0x7E and ko.encode(-np.inf) == 0xFE and ko.encode(np.nan) == 0x7F
    assert ko.encode(-1e-30) == 0x80


def test_scale_is_the_smallest_power_of_two():
    assert ko.scale_of(448.0) == 1.0 and ko.scale_of(448.1) == 2.0 and ko.scale_of(224.0) == 0.5
    assert ko.scale_of(0.0) == 2.0 ** -100 and ko.scale_of(np.inf) == 2.0 ** 120
    for x in np.exp2(np.random.default_rng(0).uniform(-20, 20, 50)):
        s = ko.scale_of(x)
        assert x <= 448 * s and x > 448 * s / 2


def test_rotation_keeps_lengths_and_pairs():
    x = np.arange(8, dtype=np.float32)
    c, s = np.zeros(2, np.float32), np.ones(2, np.float32)   # a quarter turn of the first 4 elements
    assert ko.rotate_f32(x, c, s, False).tolist() == [-2, -3, 0, 1, 4, 5, 6, 7]
    assert ko.rotate_f32(x, c, s, True).tolist() == [-1, 0, -3, 2, 4, 5, 6, 7]


def test_append_by_hand():
    """Block of 16, three tokens after one: the scale grows from 2^-2 to 1 and
    the old codes are rounded again."""
    c = dict(k=np.zeros((1, 1, 16, 64), np.uint8), v=np.zeros((1, 1, 16, 64), np.uint8),
             k_scale=np.full((1, 1), 0.25, np.float32), v_scale=np.full((1, 1), 4.0, np.float32),
             table=np.zeros((1, 1), np.int32), lens=np.array([4], np.int32), n_new=None)
    c["k"][0, 0, 0, :3] = [0x7E, 0x39, 0x01]       # 448, 1.125, 2^-9, times 0.25
    k = np.zeros((1, 3, 1, 64), np.float32)
    k[0, 0, 0, 0], k[0, 1, 0, 1], k[0, 2, 0, 2] = 300.0, 17.0, -0.001
    v = np.ones((1, 3, 1, 64), np.float32)
    kb = np.zeros((1, 1, 1, 64), np.float16)
    ko.append(c, k, v, kb=kb)
    assert c["k_scale"][0, 0] == 1.0 and c["v_scale"][0, 0] == 4.0
    assert ko.decode(c["k"][0, 0, 0, :3]).tolist() == [112.0, 0.28125, 0.0]   # 2^-11 rounds to 0
    assert ko.decode(c["k"][0, 0, 1, 0]) == 288.0 and ko.decode(c["k"][0, 0, 2, 1]) == 16.0  # ties to even
    assert ko.decode(c["k"][0, 0, 3, 2]) == -(2.0 ** -9)                   # 0.512 of a quantum
    assert ko.decode(c["v"][0, 0, 1:4]).min() == 0.25
    assert float(kb[0, 0, 0, 0]) == 100.0


def test_attend_against_a_direct_sum():
    c = kc.make_cache([70, 5], 2, 32, 64, seed=1)
    rng = np.random.default_rng(2)
    q = rng.standard_normal((2, 3, 4, 64))
    out, lse, bound = ko.attend(c, q, 0.125)
    for b, j, h in ((0, 0, 0), (0, 2, 3), (1, 1, 2)):
        p = int(c["lens"][b]) - 3 + j
        num, den = np.zeros(64), 0.0
        for t in range(p + 1):
            page, o, kv = c["table"][b, t // 32], t % 32, h // 2
            key = ko.E4M3[c["k"][page, kv, o]] * float(c["k_scale"][page, kv])
            w = math.exp(0.125 * math.fsum(key * q[b, j, h]))
            num += w * ko.E4M3[c["v"][page, kv, o]] * float(c["v_scale"][page, kv])
            den += w
        assert np.allclose(out[b, j, h], num / den, rtol=1e-12, atol=1e-13)
        assert abs(lse[b, j, h] - math.log(den)) < 1e-12
        assert (bound[b, j, h] > 0).all() and (bound[b, j, h] < 0.05 * np.abs(num / den).max() + 0.05).all()


def test_attend_of_equal_scores_is_the_mean_exactly():
    c = kc.make_cache([9], 1, 16, 64, seed=3)
    out, lse, _ = ko.attend(c, np.zeros((1, 1, 1, 64)), 1.0)
    page = c["table"][0, 0]
    for d in range(64):
        mean = sum(Fraction(float(ko.E4M3[c["v"][page, 0, t, d]] * c["v_scale"][page, 0])) for t in range(9)) / 9
        assert abs(out[0, 0, 0, d] - float(mean)) < 1e-14
    assert abs(lse[0, 0, 0] - math.log(9)) < 1e-14


def test_rows_that_see_nothing():
    c = kc.make_cache([0, 2, 40], 1, 32, 64, seed=4, n_new=[3, 3, 1])
    out, lse, _ = ko.attend(c, np.ones((3, 3, 2, 64)), 1.0)
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all()
    assert (out[1, 0] == 0).all() and not np.isneginf(lse[1, 1]).any()   # row 0 would stand at -1
    assert (out[2, 1:] == 0).all() and np.isfinite(lse[2, 0]).all()
    ids = np.full((3, 1, 3, 2), -1, np.int32)
    out, lse, _ = ko.attend(c, np.ones((3, 3, 2, 64)), 1.0, ids)
    assert (out == 0).all() and np.isneginf(lse).all()


@pytest.mark.parametrize("seed", range(3))
def test_chosen_order_does_not_matter(seed):
    c = kc.make_cache([130], 1, 32, 64, seed=seed)
    q = np.random.default_rng(seed).standard_normal((1, 1, 2, 64))
    a = ko.attend(c, q, 0.3, np.array([[[[0, 4, 2]]]], np.int32))
    b = ko.attend(c, q, 0.3, np.array([[[[-1, 2, 0, 4]]]], np.int32))
    assert np.allclose(a[0], b[0], rtol=1e-13) and np.allclose(a[1], b[1], rtol=1e-13)


def test_bound_sees_a_wrong_result():
    """The bound rejects a result that lost a token, or took its scale twice."""
    c = kc.make_cache([60], 1, 32, 64, seed=5)
    q = np.random.default_rng(6).standard_normal((1, 1, 1, 64))
    out, _, bound = ko.attend(c, q, 0.125)
    c["lens"][0] = 59
    less, _, _ = ko.attend(c, q, 0.125)
    assert (np.abs(less - out) > bound + 2.0 ** -11 * np.abs(out)).any()
    c["lens"][0] = 60
    c["v_scale"][c["table"][0, 1]] *= 2
    twice, _, _ = ko.attend(c, q, 0.125)
    assert (np.abs(twice - out) > bound + 2.0 ** -11 * np.abs(out)).any()
