"""libgdn.so needs nvcc alone: it is built where _marshal.so, the module against torch's and Python's headers,
cannot be."""
import os

import pytest

from hybrid_gated_deltanet_gb300 import build as gbuild


@pytest.fixture()
def small(monkeypatch, tmp_path):
    """A build of one source into a folder of its own."""
    monkeypatch.setattr(gbuild, "SOURCES", ["gdn_tables.cu"])
    for name, path in (("LIB", "libgdn.so"), ("MARSHAL", "_marshal.so"), ("BUILD", "_build")):
        monkeypatch.setattr(gbuild, name, str(tmp_path / path))
    return tmp_path


def test_the_library_is_built_though_the_module_is_not(small, monkeypatch):
    def fails():
        raise RuntimeError("no such header")

    monkeypatch.setattr(gbuild, "_build_marshal", fails)
    with pytest.raises(RuntimeError, match="no such header"):
        gbuild.build()
    assert gbuild._current(gbuild.LIB) and not os.path.exists(gbuild.MARSHAL)


def test_headers_that_are_missing(small, monkeypatch):
    monkeypatch.setattr(gbuild.sysconfig, "get_paths", lambda: {"include": str(small)})
    with pytest.warns(UserWarning, match="Python.h not found"):
        assert gbuild.build() == gbuild.LIB
    assert gbuild._current(gbuild.LIB) and not os.path.exists(gbuild.MARSHAL)
    before = os.path.getmtime(gbuild.LIB)
    monkeypatch.setattr(gbuild.importlib.util, "find_spec", lambda name: None)  # no torch: no one to use it, no warning
    assert gbuild.build() == gbuild.LIB and os.path.getmtime(gbuild.LIB) == before
