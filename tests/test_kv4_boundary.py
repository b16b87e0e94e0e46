"""CPU tests of the 4-bit cache's entry points: argument checks happen on the
host, in order, before any CUDA call; empty work succeeds."""
import ctypes

import pytest

import top_block_selection_gb300 as tbs
from test_kv_boundary import BAD_ROWS, Cache, GEOM, INVALID, MISALIGNED, OK, A, rows
from top_block_selection_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return tbs.load_library()


def cache(**kw):
    """A qsa_kv4_cache: the fields are those of a qsa_kv_cache."""
    f = dict(k=A, v=A, k_scale=A, v_scale=A, page_table=A, lens=A, n_new=None, page_stride=8 * 64 * 64, n_pages=10,
             max_blocks=5, B=2, Hkv=8, block=64, D=128)
    f.update(kw)
    if "page_stride" not in kw:
        f["page_stride"] = f["Hkv"] * f["block"] * f["D"] // 2
    return Cache(*[f[n] for n, _ in Cache._fields_])


def ref(s):
    return None if s is None else ctypes.byref(s)


def append(lib, c=None, k=None, v=None, q=None, n=1, Hq=8, dtype=0, cos=A, sin=A, rot=128, max_pos=100, offset=None,
           q_out=None, kb=None):
    return lib.qsa_kv4_append(ref(c or cache()), ref(k or rows()), ref(v or rows()), ref(q), n, Hq, dtype, cos, sin, rot,
                              max_pos, 0, offset, q_out, kb, None)


def read(lib, c=None, n=1, dtype=0, k=A, v=A):
    return lib.qsa_kv4_read(ref(c or cache()), n, dtype, k, v, None)


def attend(lib, c=None, q=None, n=1, Hq=32, dtype=0, scale=0.1, ids=None, lists=1, k=4, out=A, lse=None, ws=A, size=1 << 30):
    return lib.qsa_kv4_attend(ref(c or cache()), ref(q or rows()), n, Hq, dtype, scale, ids, lists, k, out, lse, ws, size,
                              None)


def weights(lib, c=None, q=None, n=1, Hq=32, dtype=0, scale=0.1, lse=A, decay=1.0, w=A):
    return lib.qsa_kv4_weights(ref(c or cache()), ref(q or rows()), n, Hq, dtype, scale, lse, decay, w, None)


def evict(lib, c=None, w=A, budget=64, sink=4, recent=10, lens=2 * A, offset=None, ws=A, size=1 << 30):
    return lib.qsa_kv4_evict(ref(c or cache()), w, budget, sink, recent, lens, offset, ws, size, None)


ALL = (append, read, attend, weights, evict)
BAD_CACHES = [(dict(B=-1), INVALID), (dict(n_pages=-1), INVALID), (dict(max_blocks=-1), INVALID), (dict(Hkv=0), INVALID),
              (dict(block=0), INVALID), (dict(D=0), INVALID), (dict(D=96), GEOM), (dict(D=256), GEOM), (dict(block=48), GEOM),
              (dict(block=8), GEOM), (dict(Hkv=65536), GEOM), (dict(max_blocks=1 << 25), GEOM),
              (dict(page_stride=8 * 64 * 64 - 32), INVALID), (dict(page_stride=8 * 64 * 64 + 16), MISALIGNED),
              (dict(page_stride=1 << 40), GEOM), (dict(lens=None), INVALID), (dict(page_table=None), INVALID),
              (dict(k=None), INVALID), (dict(k_scale=None), INVALID), (dict(k=A + 16), MISALIGNED),
              (dict(v=A + 16), MISALIGNED), (dict(k_scale=A + 8), MISALIGNED), (dict(v_scale=A + 2), MISALIGNED),
              (dict(page_table=A + 2), MISALIGNED), (dict(lens=A + 1), MISALIGNED), (dict(n_new=A + 2), MISALIGNED)]


@pytest.mark.parametrize("change,status", BAD_CACHES, ids=[f"{list(c)[0]}-{i}" for i, (c, _) in enumerate(BAD_CACHES)])
def test_bad_caches_are_rejected(lib, change, status):
    for f in ALL:
        assert f(lib, cache(**change)) == status, f.__name__


def test_values_are_needed_but_for_weights(lib):
    for change in (dict(v=None), dict(v_scale=None)):
        for f in (append, read, attend, evict):
            assert f(lib, cache(**change)) == INVALID
        assert weights(lib, cache(**change), w=A + 4) == MISALIGNED  # the next check


@pytest.mark.parametrize("change,status", BAD_ROWS)
def test_bad_rows_are_rejected(lib, change, status):
    bad = rows(**change)
    assert append(lib, k=bad) == status
    assert append(lib, v=bad) == status
    assert append(lib, q=bad, q_out=A) == status
    assert attend(lib, q=bad) == status
    assert weights(lib, q=bad) == status


def test_append_and_read_reject_bad_arguments(lib):
    assert append(lib, n=-1) == INVALID and read(lib, n=-1) == INVALID
    assert append(lib, dtype=2) == INVALID and read(lib, dtype=2) == INVALID
    assert append(lib, rot=-16) == INVALID and append(lib, max_pos=-1) == INVALID
    assert append(lib, rot=24) == GEOM and append(lib, rot=144) == GEOM
    assert append(lib, cache(B=1 << 20), n=1 << 12) == GEOM and read(lib, cache(B=1 << 20), n=1 << 12) == GEOM
    assert append(lib, cache(B=1 << 16, Hkv=65535)) == GEOM and read(lib, cache(B=1 << 18, Hkv=65535), n=8) == GEOM
    assert append(lib, cos=None) == INVALID and append(lib, sin=None) == INVALID
    assert append(lib, cos=A + 4) == MISALIGNED and append(lib, kb=A + 1) == MISALIGNED
    assert append(lib, offset=A + 2) == MISALIGNED
    assert append(lib, q=rows(), q_out=None) == INVALID and append(lib, q_out=A) == INVALID
    assert append(lib, q=rows(), q_out=A, Hq=0) == INVALID and append(lib, q=rows(), q_out=A + 8) == MISALIGNED
    assert read(lib, k=None) == INVALID and read(lib, v=None) == INVALID
    assert read(lib, k=A + 8) == MISALIGNED and read(lib, v=A + 2) == MISALIGNED


def test_attend_and_weights_reject_bad_arguments(lib):
    for f in (attend, weights):
        assert f(lib, n=-1) == INVALID
        assert f(lib, Hq=0) == INVALID
        assert f(lib, Hq=12) == INVALID            # not a multiple of Hkv
        assert f(lib, Hq=8 * 33) == GEOM
        assert f(lib, dtype=-1) == INVALID
        assert f(lib, scale=float("nan")) == INVALID and f(lib, scale=float("inf")) == INVALID
        assert f(lib, cache(n_pages=0)) == INVALID and f(lib, cache(max_blocks=0)) == INVALID
    assert attend(lib, ids=A, k=0) == INVALID and attend(lib, ids=A, lists=2) == INVALID
    assert attend(lib, ids=A, k=(1 << 20) + 1) == GEOM and attend(lib, ids=A + 2) == MISALIGNED
    assert attend(lib, out=None) == INVALID and attend(lib, out=A + 8) == MISALIGNED
    assert attend(lib, lse=A + 2) == MISALIGNED
    assert attend(lib, ws=None) == INVALID and attend(lib, ws=A + 4) == MISALIGNED
    assert attend(lib, size=tbs.qsa_kv4_attend_workspace_bytes(2, 1, 32, 8, 128) - 1) == INVALID
    assert weights(lib, lse=None) == INVALID and weights(lib, w=None) == INVALID
    assert weights(lib, lse=A + 2) == MISALIGNED and weights(lib, w=A + 4) == MISALIGNED
    for decay in (-0.5, float("nan"), float("inf")):
        assert weights(lib, decay=decay) == INVALID


def test_evict_rejects_bad_arguments(lib):
    for kw in (dict(budget=0), dict(budget=-1), dict(sink=-1), dict(recent=-1), dict(sink=60, recent=5), dict(w=None),
               dict(sink=(1 << 31) - 1, recent=(1 << 31) - 1), dict(lens=None), dict(lens=A), dict(offset=2 * A), dict(offset=A), dict(ws=None),
               dict(size=2 * 8 * 64 * 4 - 1)):
        assert evict(lib, **kw) == INVALID, kw
    for kw in (dict(w=A + 8), dict(lens=A + 2), dict(offset=A + 1), dict(ws=A + 8)):
        assert evict(lib, **kw) == MISALIGNED, kw
    assert evict(lib, cache(n_pages=0)) == INVALID and evict(lib, cache(max_blocks=0)) == INVALID
    assert evict(lib, cache(B=1 << 16, Hkv=4096)) == GEOM


def test_empty_work_succeeds_without_pointers(lib):
    none = dict(k=None, v=None, k_scale=None, v_scale=None, page_table=None, lens=None, n_pages=0, max_blocks=0)
    for c, n in ((cache(B=0, **none), 1), (cache(**none), 0)):
        assert append(lib, c, rows(data=None), n=n) == OK
        assert read(lib, c, n=n, k=None, v=None) == OK
        assert attend(lib, c, n=n, out=None, ws=None, size=0) == OK
        assert weights(lib, c, n=n, lse=None, w=None) == OK
    assert evict(lib, cache(B=0, **none), w=None, lens=None, ws=None, size=0) == OK


def test_workspace_sizes(lib):
    assert tbs.qsa_kv4_attend_workspace_bytes(1, 1, 8, 2, 128) > 0
    assert tbs.qsa_kv4_attend_workspace_bytes(1, 1, 64, 2, 64) > 0
    for bad in ((-1, 1, 8, 2, 128), (1, -1, 8, 2, 128), (1, 1, 0, 2, 128), (1, 1, 8, 0, 128), (1, 1, 9, 2, 128),
                (1, 1, 66, 2, 128), (1, 1, 8, 2, 96)):
        assert tbs.qsa_kv4_attend_workspace_bytes(*bad) == 0
    assert tbs.qsa_kv4_evict_workspace_bytes(3, 2, 100) == 3 * 2 * 100 * 4
    assert tbs.qsa_kv4_evict_workspace_bytes(-1, 2, 100) == tbs.qsa_kv4_evict_workspace_bytes(1, 2, 0) == 0


def test_binding_rejects_host_tensors(lib):
    torch = pytest.importorskip("torch")
    k = torch.zeros((2, 1, 64, 64), dtype=torch.uint8)
    s = torch.ones((2, 1, 64), dtype=torch.bfloat16)
    w, t, n = torch.ones((2, 1, 64)), torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q = torch.zeros((1, 1, 4, 128), dtype=torch.float16)
    c = (k, k, s, s, t, n)
    for call in (lambda: tbs.qsa_kv4_append(q[:, :, :1], q[:, :, :1], *c), lambda: tbs.qsa_kv4_read(*c, n=1),
                 lambda: tbs.qsa_kv4_attend(q, *c), lambda: tbs.qsa_kv4_weights(q, w, *c, w),
                 lambda: tbs.qsa_kv4_evict(*c, w, 8), lambda: tbs.qsa_kv4_read(*c, n=1, dtype=torch.float32)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        tbs.qsa_kv4_attend(q, None, *c[1:])
