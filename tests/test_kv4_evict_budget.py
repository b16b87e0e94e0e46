"""Budgets of the eviction that no sequence can outgrow: nothing goes, and no
workspace is needed for what would have moved."""
import numpy as np
import pytest

import kv4_cases as kc
import test_kv4_boundary as host
from test_kv4_boundary import A, INVALID, MISALIGNED, cache, lib  # noqa: F401

torch = pytest.importorskip("torch")
ROOM = 5 * 64  # of the boundary tests' page table


@pytest.mark.parametrize("budget", [ROOM, ROOM + 1, (1 << 31) - 1])
def test_needs_no_workspace(lib, budget):  # noqa: F811
    for kw in (dict(ws=None, size=0), dict(size=0), dict(size=16)):
        assert host.evict(lib, budget=budget, w=A + 8, **kw) == MISALIGNED  # the next check
        assert host.evict(lib, budget=ROOM - 1, w=A + 8, **kw) == INVALID
    assert host.evict(lib, budget=budget, sink=budget, recent=1, ws=None, size=0) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("budget,sink,recent", [(320, 320, 0), (321, 300, 21), ((1 << 31) - 1, 4, 1 << 30)])
def test_takes_nothing_out(budget, sink, recent):
    """64 sequences on 16 heads, whose workspace for the largest budget would be 8 TB."""
    import top_block_selection_gb300 as tbs
    from test_kv4_parity import on_gpu
    c = kc.make_cache([320, 0, 17, 319] * 16, 16, 64, 64, max_blocks=5)
    args, _ = on_gpu(c)
    w = torch.from_numpy(c["w"]).cuda()
    offset = torch.full((64,), 5, dtype=torch.int32, device="cuda")
    got = tbs.qsa_kv4_evict(*args, w, budget, sink, recent, offset=offset)
    assert np.array_equal(got.cpu().numpy(), c["lens"]) and (offset == 5).all()
    for t, name in zip(args[:4] + [w], ("k", "v", "k_scale", "v_scale", "w")):
        x = t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()
        assert np.array_equal(x, c[name], equal_nan=x.dtype == np.float32), name
    assert tbs.qsa_device_status(clear=True) == (0, 0)


def test_lengths_and_offsets_that_overlap_are_refused(lib):  # noqa: F811
    for kw in (dict(lens=A), dict(lens=A + 4), dict(lens=A - 4), dict(offset=A + 4), dict(offset=2 * A - 4),
               dict(offset=2 * A + 4), dict(offset=2 * A), dict(lens=A + 4, offset=4 * A)):
        assert host.evict(lib, **kw) == INVALID, kw
