"""GPU test of the cache attention of many rows where the warps of a row tile
run far apart: every key tile moves the references of one warp's rows, and the
other warps' never, so that these reach the end of an item well ahead."""
import numpy as np
import pytest

import kv_cases as kc
from oracle import kv_oracle as ko
from test_kv_parity import check_rows, dev, on_gpu, tbs  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def shared_cache(B, tokens, D, block, seed, codes):
    """B sequences of `tokens` tokens in the same pages (one KV head, scales 2^-4);
    codes(k) changes the key values [tokens, D] before they are encoded."""
    rng = np.random.default_rng(seed)
    pages = -(-tokens // block)
    order = rng.permutation(pages).astype(np.int32)
    out = dict(table=np.broadcast_to(order, (B, pages)).copy(), lens=np.full(B, tokens, np.int32), n_new=None)
    for name in ("k", "v"):
        x = rng.standard_normal((tokens, D)) * 16.0
        if name == "k":
            codes(x)
        full = np.full((pages, 1, block, D), 0x7F, np.uint8)
        c = ko.encode(x)
        for i in range(pages):
            held = min(block, tokens - i * block)
            full[order[i], 0, :held] = c[i * block:i * block + held]
        out[name] = full
        out[name + "_scale"] = np.full((pages, 1), 2.0 ** -4, np.float32)
    return out


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("slow", [0, 3])
def test_warps_of_a_row_tile_run_apart(tbs, D, dtype, slow):  # noqa: F811
    """One item of 17 tiles a CTA. Dimension 0 of the keys grows by 16 codes a
    tile (x 2^-4 x 16 = 16 in the score: 23 in log2), which only the queries of
    warp `slow` of each row tile (two of eight, 16 heads) look at."""
    B, tokens, n, R = 19, 17 * 128, 128, 16

    def rising(k):
        k[:, 0] = 16.0 * (np.arange(tokens) // 128)
    c = shared_cache(B, tokens, D, 64, D, rising)
    rng = np.random.default_rng(slow)
    q = rng.standard_normal((B, n, R, D))
    q[..., 0] = np.where(np.arange(n) % 8 // 2 == slow, 16.0 / D ** -0.5 / 16.0, 0.0)[None, :, None]
    q = kc.ROUND[dtype](q)
    args, _ = on_gpu(c)
    g = dev(q, dtype)
    out = tbs.qsa_kv_attend(g, *args)
    assert "kv_attend_many_kernel" in tbs.qsa_arm()
    for _ in range(50):
        assert torch.equal(tbs.qsa_kv_attend(g, *args), out)
    at = [(int(rng.integers(B)), int(rng.integers(n)), int(rng.integers(R))) for _ in range(60)]
    check_rows(c, q, out, None, dtype, at)
