"""CPU tests of the paged-cache entry points: argument checks happen on the
host, in order, before any CUDA call; empty work succeeds."""
import ctypes

import pytest

import top_block_selection_gb300 as tbs
from top_block_selection_gb300 import _build

OK, INVALID, GEOM, ARCH, MISALIGNED, CUDA, TIMEOUT = range(7)
A = 1 << 20  # a fake, aligned address; never dereferenced


class Cache(ctypes.Structure):
    _fields_ = [(x, ctypes.c_void_p) for x in ("k", "v", "k_scale", "v_scale", "page_table", "lens", "n_new")] \
        + [("page_stride", ctypes.c_int64)] \
        + [(x, ctypes.c_int32) for x in ("n_pages", "max_blocks", "B", "Hkv", "block", "D")]


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + [(x, ctypes.c_int64) for x in ("stride_b", "stride_n", "stride_h")]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return tbs.load_library()


def cache(**kw):
    f = dict(k=A, v=A, k_scale=A, v_scale=A, page_table=A, lens=A, n_new=None, page_stride=8 * 64 * 128, n_pages=10,
             max_blocks=5, B=2, Hkv=8, block=64, D=128)
    f.update(kw)
    if "page_stride" not in kw:
        f["page_stride"] = f["Hkv"] * f["block"] * f["D"]
    return Cache(*[f[n] for n, _ in Cache._fields_])


def rows(**kw):
    f = dict(data=A, stride_b=1024, stride_n=1024, stride_h=128)
    f.update(kw)
    return Rows(*[f[n] for n, _ in Rows._fields_])


def append(lib, c=None, k=None, v=None, q=None, n=1, Hq=8, dtype=0, cos=A, sin=A, rot=128, max_pos=100, q_out=None, kb=None):
    ref = lambda s: None if s is None else ctypes.byref(s)
    return lib.qsa_kv_append(ref(c if c is not None else cache()), ref(k or rows()), ref(v or rows()), ref(q), n, Hq,
                             dtype, cos, sin, rot, max_pos, 0, q_out, kb, None)


def attend(lib, c=None, q=None, n=1, Hq=32, dtype=0, scale=0.1, ids=None, lists=1, k=4, out=A, lse=None, ws=A, size=1 << 30):
    return lib.qsa_kv_attend(ctypes.byref(c if c is not None else cache()), ctypes.byref(q or rows()), n, Hq, dtype,
                             scale, ids, lists, k, out, lse, ws, size, None)


BAD_CACHES = [(dict(B=-1), INVALID), (dict(n_pages=-1), INVALID), (dict(max_blocks=-1), INVALID), (dict(Hkv=0), INVALID),
              (dict(block=0), INVALID), (dict(D=0), INVALID), (dict(D=96), GEOM), (dict(D=256), GEOM), (dict(block=48), GEOM),
              (dict(block=256), GEOM), (dict(Hkv=65536), GEOM), (dict(max_blocks=1 << 25), GEOM),
              (dict(page_stride=8 * 64 * 128 - 16), INVALID), (dict(page_stride=8 * 64 * 128 + 8), MISALIGNED),
              (dict(page_stride=1 << 40), GEOM), (dict(lens=None), INVALID), (dict(page_table=None), INVALID),
              (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k_scale=None), INVALID),
              (dict(v_scale=None), INVALID), (dict(k=A + 8), MISALIGNED), (dict(v=A + 4), MISALIGNED),
              (dict(k_scale=A + 2), MISALIGNED), (dict(v_scale=A + 1), MISALIGNED), (dict(page_table=A + 2), MISALIGNED),
              (dict(lens=A + 1), MISALIGNED), (dict(n_new=A + 2), MISALIGNED)]


@pytest.mark.parametrize("change,status", BAD_CACHES, ids=[f"{list(c)[0]}-{i}" for i, (c, _) in enumerate(BAD_CACHES)])
def test_bad_caches_are_rejected(lib, change, status):
    assert append(lib, cache(**change)) == status
    assert attend(lib, cache(**change)) == status


BAD_ROWS = [(dict(data=None), INVALID), (dict(stride_b=-8), INVALID), (dict(stride_n=-8), INVALID),
            (dict(stride_h=-8), INVALID), (dict(data=A + 8), MISALIGNED), (dict(stride_b=1028), MISALIGNED),
            (dict(stride_n=1), MISALIGNED), (dict(stride_h=132), MISALIGNED)]


@pytest.mark.parametrize("change,status", BAD_ROWS)
def test_bad_rows_are_rejected(lib, change, status):
    bad = rows(**change)
    assert append(lib, k=bad) == status
    assert append(lib, v=bad) == status
    assert append(lib, q=bad, q_out=A) == status
    assert attend(lib, q=bad) == status


def test_append_rejects_bad_arguments(lib):
    assert append(lib, n=-1) == INVALID
    assert append(lib, dtype=2) == INVALID
    assert append(lib, rot=-16) == INVALID
    assert append(lib, max_pos=-1) == INVALID
    assert append(lib, rot=24) == GEOM
    assert append(lib, rot=144) == GEOM
    assert append(lib, cache(B=1 << 20), n=1 << 12) == GEOM
    assert append(lib, cache(B=1 << 16, Hkv=65535), n=1) == GEOM
    assert append(lib, cos=None) == INVALID
    assert append(lib, sin=None) == INVALID
    assert append(lib, cos=A + 4) == MISALIGNED
    assert append(lib, kb=A + 1) == MISALIGNED
    assert append(lib, q=rows(), q_out=None) == INVALID
    assert append(lib, q=rows(), q_out=A, Hq=0) == INVALID
    assert append(lib, q=rows(), q_out=A + 8) == MISALIGNED
    assert append(lib, q_out=A) == INVALID
    assert lib.qsa_kv_append(None, ctypes.byref(rows()), ctypes.byref(rows()), None, 1, 0, 0, None, None, 0, 0, 0, None,
                             None, None) == INVALID


def test_attend_rejects_bad_arguments(lib):
    assert attend(lib, n=-1) == INVALID
    assert attend(lib, Hq=0) == INVALID
    assert attend(lib, Hq=12) == INVALID           # not a multiple of Hkv
    assert attend(lib, Hq=8 * 33) == GEOM
    assert attend(lib, dtype=-1) == INVALID
    assert attend(lib, scale=float("nan")) == INVALID
    assert attend(lib, scale=float("inf")) == INVALID
    assert attend(lib, ids=A, k=0) == INVALID
    assert attend(lib, ids=A, lists=2) == INVALID
    assert attend(lib, ids=A, k=(1 << 20) + 1) == GEOM
    assert attend(lib, ids=A + 2) == MISALIGNED
    assert attend(lib, out=None) == INVALID
    assert attend(lib, out=A + 8) == MISALIGNED
    assert attend(lib, lse=A + 2) == MISALIGNED
    assert attend(lib, ws=None) == INVALID
    assert attend(lib, ws=A + 4) == MISALIGNED
    assert attend(lib, size=tbs.qsa_kv_attend_workspace_bytes(2, 1, 32, 8, 128) - 1) == INVALID
    assert attend(lib, cache(n_pages=0)) == INVALID
    assert attend(lib, cache(max_blocks=0)) == INVALID


def test_empty_work_succeeds_without_pointers(lib):
    none = dict(k=None, v=None, k_scale=None, v_scale=None, page_table=None, lens=None, n_pages=0, max_blocks=0)
    assert append(lib, cache(B=0, **none), rows(data=None)) == OK
    assert append(lib, cache(**none), n=0) == OK
    assert attend(lib, cache(B=0, **none), rows(data=None), out=None, ws=None, size=0) == OK
    assert attend(lib, cache(**none), n=0, out=None, ws=None, size=0) == OK


def test_workspace_size(lib):
    assert tbs.qsa_kv_attend_workspace_bytes(1, 1, 8, 2, 128) > 0
    for bad in ((-1, 1, 8, 2, 128), (1, -1, 8, 2, 128), (1, 1, 0, 2, 128), (1, 1, 8, 0, 128), (1, 1, 9, 2, 128),
                (1, 1, 66, 2, 128), (1, 1, 8, 2, 96)):
        assert tbs.qsa_kv_attend_workspace_bytes(*bad) == 0


def test_binding_rejects_host_tensors(lib):
    torch = pytest.importorskip("torch")
    k = torch.zeros((2, 1, 64, 128), dtype=torch.uint8)
    s, t, n = torch.ones((2, 1)), torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q = torch.zeros((1, 1, 4, 128), dtype=torch.float16)
    with pytest.raises(ValueError):
        tbs.qsa_kv_attend(q, k, k, s, s, t, n)
    with pytest.raises(ValueError):
        tbs.qsa_kv_append(q[:, :, :1], q[:, :, :1], k, k, s, s, t, n)
    with pytest.raises(TypeError):
        tbs.qsa_kv_attend(q, None, k, s, s, t, n)
