"""CPU tests of the build: the C library needs neither PyTorch nor Python's
headers, and the module that takes PyTorch tensors is built anew for another
PyTorch or Python."""
import importlib.metadata
import importlib.util
import sysconfig

import pytest

from top_block_selection_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


@pytest.mark.parametrize("missing", ["torch", "headers"])
def test_the_library_builds_without_the_binding(monkeypatch, tmp_path, capsys, missing):
    monkeypatch.setattr(_build, "BINDINGPATH", str(tmp_path / "_qsa_kv.so"))
    if missing == "torch":
        find = importlib.util.find_spec
        monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    else:
        paths = dict(sysconfig.get_paths(), include=str(tmp_path))
        monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: paths)
    assert _build.build() == _build.LIBPATH
    assert "_qsa_kv.so not built" in capsys.readouterr().err
    assert not (tmp_path / "_qsa_kv.so").exists()


def test_the_binding_is_stale_for_another_torch_or_python(monkeypatch):
    pytest.importorskip("torch")
    assert not _build._binding_stale()
    with monkeypatch.context() as m:
        version = importlib.metadata.version
        m.setattr(importlib.metadata, "version", lambda name: "0.0" if name == "torch" else version(name))
        assert _build._binding_stale()
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: ".cpython-0-none.so")
        assert _build._binding_stale()
    assert not _build._binding_stale()
