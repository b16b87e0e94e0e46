"""GPU tests of device-side indexes of the cache attention that lie outside the
cache: left out and recorded, whichever kernel takes the call and wherever in a
tile they stand."""
import numpy as np
import pytest

import kv_cases as kc
from oracle import kv_oracle as ko
from test_kv_parity import TINY, UNIT, dev, on_gpu, tbs  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def close(got, c, q, dtype, ids):
    """The result against the oracle's over the listed blocks."""
    want, _, bound = ko.attend(c, q, q.shape[-1] ** -0.5, np.array(ids, np.int32), terms=3 if dtype == "f16" else 2)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= bound + UNIT[dtype] * (np.abs(want) + bound) + TINY[dtype]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,Hq", [(1, 4), (3, 8), (128, 16)])
def test_longer_than_the_page_table(tbs, D, dtype, n, Hq):  # noqa: F811
    """400 tokens, a table for 320: attention over what the table holds."""
    c = kc.make_cache([400], 1, 64, D, seed=n)
    c["table"] = np.ascontiguousarray(c["table"][:, :5])
    args, _ = on_gpu(c)
    q = kc.ROUND[dtype](np.random.default_rng(1).standard_normal((1, n, Hq, D)))
    got = tbs.qsa_kv_attend(dev(q, dtype), *args)
    assert ("many" in tbs.qsa_arm()) == (n == 128)
    assert tbs.qsa_device_status(clear=True) == (1, 32)
    close(got, c, q, dtype, [[[[0, 1, 2, 3, 4]] * n]])
    # as long as the table: nothing to record
    args[5].fill_(320)
    tbs.qsa_kv_attend(dev(q, dtype), *args)
    assert tbs.qsa_device_status(clear=True) == (0, 0)


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("n,Hq", [(1, 4), (128, 16)])
def test_pages_outside_in_any_place_of_a_tile(tbs, block, n, Hq):  # noqa: F811
    """One page id outside the cache, at each of the blocks in turn."""
    blocks = 256 // block + 2
    c = kc.make_cache([blocks * block - 3], 1, block, 64, seed=block)
    args, _ = on_gpu(c)
    q = kc.as_f16(np.random.default_rng(2).standard_normal((1, n, Hq, 64)))
    for i in range(blocks):
        table = args[4].clone()
        table[0, i] = -1 if i % 2 else c["k"].shape[0]
        got = tbs.qsa_kv_attend(dev(q, "f16"), *args[:4], table, args[5])
        assert tbs.qsa_device_status(clear=True) == (1, 32), i
        if n == 1 or i in (0, 1, blocks - 1):
            close(got, c, q, "f16", [[[[k for k in range(blocks) if k != i]] * n]])
