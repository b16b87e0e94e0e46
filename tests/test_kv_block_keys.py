"""GPU tests of the block keys that the append makes: the fp16 mean of the
block's stored keys, the same however its sum is split over threads, and what a
selection next on the stream reads."""
import numpy as np
import pytest

import kv_cases as kc
from oracle import kv_oracle as ko
from test_kv_parity import dev, on_gpu, same_bits, tbs  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cut", [0, 1, 40, 64, 100, 127])
@pytest.mark.parametrize("seed", range(3))
def test_a_sum_past_24_bits(tbs, D, cut, seed):  # noqa: F811
    """A block of 128 tokens whose codes add up to 35,600 + 3 x 2^-9, a little
    above the middle of two fp16 means: the 2^-9 count although each is less
    than half of the sum's last fp32 bit. The codes stand in any order, and the
    first `cut` tokens were appended before the others."""
    rng = np.random.default_rng(seed)
    x = np.zeros((128, D), np.float32)
    for d in range(D):
        col = np.zeros(128)
        col[:79], col[79], col[80:83] = 448.0, 208.0, 2.0 ** -9
        x[:, d] = col if seed == 0 else rng.permutation(col)
        if seed == 0:  # large codes in the tokens of the first threads of each pass
            order = np.argsort(np.arange(128) % 32, kind="stable")
            x[order, d] = col[np.r_[0:80, 83:96, 80, 83 + 13:83 + 13 + 15, 81, 111:127, 82, 127]]
    c = kc.make_cache([128], 1, 128, D, filled=False)
    kv = kc.as_f16(x)[None, :, None]
    kb = np.zeros((1, 1, 1, D), np.float16)
    args, _ = on_gpu(c)
    gkb = dev(kb)
    for lo, hi in ((0, cut), (cut, 128)):
        if hi == lo:
            continue
        c["lens"][0] = hi
        args[5].fill_(hi)
        ko.append(c, kv[:, lo:hi], kv[:, lo:hi], kb=kb)
        tbs.qsa_kv_append(dev(kv[:, lo:hi], "f16"), dev(kv[:, lo:hi], "f16"), *args, kb=gkb)
    assert (kb == 278.25).all()
    same_bits(args[0], c["k"], "k")
    same_bits(gkb, kb, "kb")


def test_a_nan_key_makes_its_mean_nan(tbs):  # noqa: F811
    c = kc.make_cache([128], 1, 128, 64, filled=False)
    x = kc.as_f16(np.random.default_rng(1).standard_normal((1, 128, 1, 64)))
    x[0, 77, 0, 9] = np.nan
    args, _ = on_gpu(c)
    kb = dev(np.zeros((1, 1, 1, 64), np.float16))
    tbs.qsa_kv_append(dev(x, "f16"), dev(x, "f16"), *args, kb=kb)
    assert torch.isnan(kb).flatten().nonzero().flatten().tolist() == [9]


@pytest.mark.parametrize("nq,n", [(1, 1), (16, 40), (300, 300)])
def test_selection_reads_what_the_append_before_it_wrote(tbs, nq, n):  # noqa: F811
    """Append with block keys and a selection over them, in a stream without a
    wait between them, against the same with one."""
    Hkv, D, block, k = 4, 128, 64, 8
    c = kc.make_cache([n + 2000], Hkv, block, D, seed=n, spread=1.0)
    g = torch.Generator(device="cuda").manual_seed(n)
    q = torch.randn((Hkv, nq, 2, D), generator=g, device="cuda").half()
    blocks = c["table"].shape[1]
    for i in range(10):
        x = torch.randn((1, n, 2 * Hkv, D), generator=g, device="cuda", dtype=torch.float16)
        ids = []
        for wait in (False, True):
            args, _ = on_gpu(c)
            kb = torch.randn((1, Hkv, blocks, D), generator=torch.Generator(device="cuda").manual_seed(i),
                             device="cuda").half()
            torch.cuda.synchronize()
            tbs.qsa_kv_append(x[:, :, :Hkv], x[:, :, Hkv:], *args, kb=kb)
            if wait:
                torch.cuda.synchronize()
            ids.append(tbs.qsa_score_select_batched(q, kb[0], n + 2000, k, block))
        for a, b in zip(*ids):
            assert torch.equal(a, b)
