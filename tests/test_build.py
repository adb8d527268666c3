"""libgdn.so needs nvcc alone: it is built where _marshal.so, the module against torch's and Python's headers,
cannot be."""
import os
import subprocess
import sys

import pytest
import torch

from hybrid_gated_deltanet_gb300 import binding as gb
from hybrid_gated_deltanet_gb300 import build as gbuild


@pytest.fixture()
def small(monkeypatch, tmp_path):
    """A build of one source into a folder of its own."""
    monkeypatch.setattr(gbuild, "SOURCES", ["gdn_tables.cu"])
    for name, path in (("LIB", "libgdn.so"), ("MARSHAL", "_marshal.so"), ("STAMP", "_marshal.stamp"), ("BUILD", "_build")):
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


def test_the_module_of_another_torch_or_python(small, monkeypatch):
    """A module compiled against another torch or Python, or with no word of which, is built again, and never loaded
    by the binding."""
    gbuild._build_lib(False, False)
    built = []

    def stands_in():
        built.append(gbuild.marshal_key())
        with open(gbuild.LIB, "rb") as lib, open(gbuild.MARSHAL, "wb") as f:
            f.write(lib.read(64))
        with open(gbuild.STAMP, "w") as f:
            f.write(built[-1])

    monkeypatch.setattr(gbuild, "_build_marshal", stands_in)
    key = gbuild.marshal_key()
    changes = [lambda: None, lambda: os.remove(gbuild.STAMP)]
    changes += [lambda other=other: monkeypatch.setattr(gbuild, "marshal_key", lambda: other)
                for other in (key + ".1", key.replace("cpython", "pypy"), key)]
    for n, change in enumerate(changes):
        change()
        assert not gbuild.marshal_fits()
        with pytest.raises(RuntimeError, match="_marshal.so is not built for this Python and torch"):
            gb._load_marshal()
        for _ in range(2):  # (the second finds it current)
            gbuild.build()
            assert gbuild.marshal_fits() and len(built) == n + 1 and built[-1] == gbuild.marshal_key()


def test_the_stamp_names_torch_as_it_is_imported():
    assert gbuild.marshal_key().endswith(f" torch {torch.__version__}")


def test_import_under_a_torch_without_cuda():
    """The package imports (its generators and the tests' oracle need no GPU) where torch was built without CUDA."""
    code = ("import torch\nfor name in [n for n in dir(torch._C) if n.startswith('_cuda_')]: delattr(torch._C, name)\n"
            "import hybrid_gated_deltanet_gb300 as g\nfrom hybrid_gated_deltanet_gb300 import synth\n"
            "try:\n    g.gdn_page_tables(16, 4, *[torch.zeros(1, dtype=torch.int32)] * 4, torch.zeros(1, 1), *[torch.zeros(2)] * 3)\n"
            "except ValueError as e:\n    assert 'required one CUDA device' in str(e)\nelse:\n    raise SystemExit('no error')\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=gbuild.ROOT)
