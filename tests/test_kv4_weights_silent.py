"""GPU tests of the attention weights of calls whose rows give nothing: rows that
are not there (fewer new tokens than rows) beside rows of lse -inf, over tokens
whose key scale is NaN."""
import numpy as np
import pytest

import kv4_cases as kc
from oracle import kv4_oracle as ko
from test_kv4_parity import dev, on_gpu, tbs  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("lens,n_new", [([300, 200], [1, 40]), ([300, 200], [0, 33]), ([300, 20], [9, 40])])
@pytest.mark.parametrize("D,dtype,R", [(64, "f16", 4), (128, "bf16", 4), (128, "f16", 5), (64, "bf16", 24)])
def test_rows_that_are_not_there_give_nothing(tbs, D, dtype, R, lens, n_new):  # noqa: F811
    """All rows of sequence 0 are silent or not there: a token's NaN scale leaves its weight alone."""
    n = 40
    c = kc.make_cache(lens, 2, 64, D, seed=n, n_new=n_new)
    page = c["table"][0, 1]
    c["k_scale"][page, :, 5] = np.nan
    c["k_scale"][c["table"][1, 0], 1, 7] = np.nan
    args, nn = on_gpu(c)
    q = kc.ROUND[dtype](np.random.default_rng(n).standard_normal((2, n, 2 * R, D)))
    lse = np.full((2, n, 2 * R), 3.0, np.float32)
    lse[0] = -np.inf
    want, bound = ko.weights(c, q, lse, c["w"], D ** -0.5, 0.5, terms=3 if dtype == "f16" else 2)
    w = dev(c["w"])
    tbs.qsa_kv4_weights(dev(q, dtype), dev(lse), *args, w, n_new=nn, decay=0.5)
    got = w.cpu().numpy().astype(np.float64)
    ok = ~np.isnan(want)
    assert np.array_equal(got[page, :, 5], 0.5 * c["w"][page, :, 5].astype(np.float64))
    assert np.array_equal(np.isnan(got), ~ok) and (np.abs(got - want)[ok] <= bound[ok]).all()
    assert np.isnan(got[c["table"][1, 0], 1, 7]) and ok[page, :, 5].all()
