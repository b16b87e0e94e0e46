"""GPU test of an append whose positions run past the angle tables: those
positions are skipped and recorded, the others of the same block stored."""
import numpy as np
import pytest

import kv_cases as kc
from oracle import kv_oracle as ko
from test_kv_parity import dev, on_gpu, same_bits, tbs  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("held,n,table", [(70, 20, 55), (70, 20, 50), (70, 70, 64), (70, 70, 65), (40, 3, 38), (200, 150, 199)])
def test_positions_past_the_angles(tbs, held, n, table):  # noqa: F811
    Hkv, D, block = 2, 64, 32
    c = kc.make_cache([held], Hkv, block, D, seed=n)
    x = kc.as_f16(np.random.default_rng(n).standard_normal((1, n, 3 * Hkv, D)))
    cos, sin = kc.angles(table, D)
    blocks = c["table"].shape[1]
    kb = np.full((1, Hkv, blocks, D), 3.0, np.float16)
    args, _ = on_gpu(c)
    gkb = dev(kb)
    g = dev(x, "f16")
    q = tbs.qsa_kv_append(g[:, :, :Hkv], g[:, :, Hkv:2 * Hkv], *args, cos=dev(cos), sin=dev(sin), q=g[:, :, 2 * Hkv:],
                          kb=gkb)
    assert tbs.qsa_device_status(clear=True) == (1, 32)
    # as if the sequence ended with the table
    there = n - (held - table)
    c["lens"][0] = table
    wq = ko.append(c, x[:, :there, :Hkv], x[:, :there, Hkv:2 * Hkv], cos, sin, False, x[:, :there, 2 * Hkv:], kb)
    for got, name in zip(args, ("k", "v", "k_scale", "v_scale")):
        same_bits(got, c[name], name)
    same_bits(gkb, kb, "kb")
    assert torch.equal(q[:, :there].cpu(), torch.from_numpy(wq).half()) and (q[:, there:] == 0).all()
