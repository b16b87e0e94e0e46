"""The eviction's forms, each over several chunks of its move: one CTA an item,
small and large CTAs in clusters, and parts of more keys than shared memory
holds. The expected cache is computed here, whole arrays at a time, and pinned to
the oracle on small cases."""
import numpy as np
import pytest

import kv4_cases as kc
from oracle import kv4_oracle as ko

torch = pytest.importorskip("torch")

NAMES = ("k", "v", "k_scale", "v_scale", "w")


def evict(c, budget, sink, recent):
    """oracle.kv4_oracle.evict of the cache and its weights, for long sequences."""
    block = c["k"].shape[2]
    for b, length in enumerate(c["lens"]):
        if length <= budget:
            continue
        slots = np.arange(length)
        page, off = c["table"][b, slots // block], slots % block
        for h in range(c["k"].shape[1]):
            w = c["w"][page, h, off][sink:length - recent].astype(np.float64)
            order = np.lexsort((-np.where(np.isnan(w), 0.0, w), ~np.isnan(w)))  # stable: equal ones by slot
            kept = np.concatenate([slots[:sink], np.sort(sink + order[:budget - sink - recent]), slots[length - recent:]])
            for name in NAMES:
                c[name][page[:budget], h, off[:budget]] = c[name][page[kept], h, off[kept]]
    return np.minimum(c["lens"], budget)


def cache(lens, Hkv, block, D, seed, ties=False, max_blocks=None):
    c = kc.make_cache(lens, Hkv, block, D, seed=seed, max_blocks=max_blocks)
    if ties:
        c["w"] = np.round(c["w"] * 0.5).astype(np.float32)
    return c


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("budget,sink,recent", [(100, 4, 20), (7, 0, 0), (64, 0, 64), (64, 64, 0), (50, 25, 25)])
def test_expected(budget, sink, recent, ties):
    c = cache([300, 101, 99, 0, 640], 2, 16, 64, budget, ties)
    for t, x in ((30, np.nan), (31, np.inf), (32, -np.inf), (33, -1.0), (34, -0.0), (200, np.nan)):
        page, off = ko.place(c, 0, t)
        c["w"][page, :, off] = x
    want = kc.copy_cache(c)
    now, _ = ko.evict(want, want["w"], budget, sink, recent)
    assert np.array_equal(evict(c, budget, sink, recent), now)
    for name in NAMES:
        assert np.array_equal(c[name], want[name], equal_nan=c[name].dtype == np.float32), name


def check(c, budget, sink, recent):
    import top_block_selection_gb300 as tbs
    from test_kv4_parity import dev, on_gpu, same
    args, _ = on_gpu(c)
    w, offset = dev(c["w"]), torch.full((len(c["lens"]),), 5, dtype=torch.int32, device="cuda")
    got = tbs.qsa_kv4_evict(*args, w, budget, sink, recent, offset=offset)
    now = evict(c, budget, sink, recent)
    assert np.array_equal(got.cpu().numpy(), now) and np.array_equal(offset.cpu().numpy(), 5 + c["lens"] - now)
    for x, name in zip(args[:4] + [w], NAMES):
        same(x, c[name], name)
    assert tbs.qsa_device_status(clear=True) == (0, 0)


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.gpu
@pytest.mark.parametrize("D,block,ties", [(64, 32, True), (128, 64, False), (128, 16, True)])
@pytest.mark.parametrize("budget,sink,recent", [(4096, 4, 512), (4096, 0, 0), (1100, 64, 0), (2500, 10, 2400)])
def test_a_cta_an_item(D, block, ties, budget, sink, recent):
    """Chunks of 512 or 1,024 tokens."""
    lens = [4160, 4097, 5000, 4096, 1, 4500, 0, 3000, 2200, 6000] * 4
    assert len(lens) * 4 > sms()
    check(cache(lens, 4, block, D, budget + D, ties), budget, sink, recent)


@pytest.mark.gpu
@pytest.mark.parametrize("B,ctas", [(4, 8), (10, 4), (30, 2)])
@pytest.mark.parametrize("D,budget,sink,recent", [(64, 8000, 4, 100), (128, 16200, 0, 1000), (128, 3000, 1, 0)])
def test_small_ctas_in_clusters(B, ctas, D, budget, sink, recent):
    """4 heads; tables of 16,384 tokens."""
    assert sms() // 2 < 4 * B * ctas <= 2 * sms() and (ctas == 8 or 4 * B * 2 * ctas > 2 * sms())
    lens = [16384, 16201, 9000, 3001, 12345][:B] + [100] * (B - 5)
    check(cache(lens, 4, 64, D, B, ties=D == 128, max_blocks=256), budget, sink, recent)


@pytest.mark.gpu
@pytest.mark.parametrize("length,budget,recent", [(131072, 32768, 2048), (70001, 70000, 0)])
def test_large_ctas_in_clusters(length, budget, recent):
    check(cache([length], 2, 64, 64, 3), budget, 64, recent)


@pytest.mark.gpu
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("lens,budget", [([45000, 300] + [50] * 38, 20000), ([345000], 100000)])
def test_more_keys_than_shared_memory_holds(lens, budget, ties):
    """Parts of more than 40,960 keys, of a CTA alone and in a cluster of eight."""
    Hkv = 4 if len(lens) > 1 else 1
    assert len(lens) == 1 or len(lens) * Hkv > sms()
    check(cache(lens, Hkv, 128, 64, 5, ties), budget, 10, 1000)
