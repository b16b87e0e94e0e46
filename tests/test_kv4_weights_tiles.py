"""GPU parity of the attention weights where a CTA has many tiles: both warpgroups
and all loading warps take tiles in turn, stages and places for scores come round
again, and a CTA's share begins and ends inside items."""
import numpy as np
import pytest

import kv4_cases as kc
from oracle import kv4_oracle as ko
from test_kv4_parity import dev, on_gpu, tbs  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LENS = [20011, 128, 0, 7003, 1, 5121, 129, 3000, 64, 2049, 999, 4096, 300, 513, 1500, 31]


def check(tbs, lens, n, R, Hkv, D, block, dtype, decay, tiles_each, n_new=None, seed=0):  # noqa: F811
    tokens = 128 * 128 // D  # of a tile
    tiles = Hkv * sum(-(-length // tokens) for length in lens)
    assert tiles > tiles_each * torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(seed)
    c = kc.make_cache(lens, Hkv, block, D, seed=seed, n_new=n_new)
    q = kc.ROUND[dtype](rng.standard_normal((len(lens), n, R * Hkv, D)))
    lse = (3 + rng.standard_normal(q.shape[:3])).astype(np.float32)
    args, nn = on_gpu(c)
    w = dev(c["w"])
    tbs.qsa_kv4_weights(dev(q, dtype), dev(lse), *args, w, n_new=nn, decay=decay)
    want, bound = ko.weights(c, q, lse, c["w"], D ** -0.5, decay, terms=3 if dtype == "f16" else 2)
    got = w.cpu().numpy().astype(np.float64)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)  # slots without a token keep their NaN
    err = np.abs(got - want)[~nan]
    assert (err <= bound[~nan]).all(), (float(err.max()), int((err > bound[~nan]).sum()))


# Forms of 8, 16 and 32 columns: rows times the tokens of an operand row.
@pytest.mark.parametrize("D,R,dtype,block,decay", [(128, 4, "f16", 64, 0.75), (128, 8, "bf16", 16, 0.0),
                                                   (128, 12, "bf16", 32, 0.75), (128, 20, "f16", 128, 1.0),
                                                   (64, 4, "bf16", 128, 0.75), (64, 6, "f16", 16, 0.0),
                                                   (64, 16, "bf16", 64, 0.75)])
def test_one_row(tbs, D, R, dtype, block, decay):  # noqa: F811
    check(tbs, LENS if D == 128 else 2 * LENS, 1, R, 4, D, block, dtype, decay, 8, seed=R)


@pytest.mark.parametrize("D,dtype", [(128, "f16"), (64, "bf16")])
def test_several_passes(tbs, D, dtype):  # noqa: F811
    """160 rows of a KV head are two passes (or three) over a CTA's tiles; one sequence has none, one a few of them."""
    lens = [9000, 70, 3001, 40, 2500]
    check(tbs, lens if D == 128 else 2 * lens, 40, 4, 4, D, 64, dtype, 0.5, 2, seed=1,
          n_new=[40, 0, 7, 40, 33] * (1 if D == 128 else 2))
