"""The build: the C library and the module that reads the tensors of small calls."""

import os

import pytest


@pytest.fixture
def small(tmp_path, monkeypatch):
    """The build module on a tree of two small sources."""
    from affine_bit_matmul_gb300 import build as b

    (tmp_path / "a.cu").write_text('extern "C" int answer() { return 42; }\n')
    (tmp_path / "c.cpp").write_text("#include <Python.h>\n"
                                    'static PyModuleDef m = {PyModuleDef_HEAD_INIT, "_calls", 0, -1, 0, 0, 0, 0, 0};\n'
                                    "PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&m); }\n")
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(b, "sources", lambda: [str(tmp_path / "a.cu")])
    monkeypatch.setattr(b, "calls_source", lambda: str(tmp_path / "c.cpp"))
    return b


def test_the_library_is_built_where_the_module_cannot_be(small):
    with open(small.calls_source(), "w") as f:
        f.write("#error no torch here\n")
    with pytest.raises(RuntimeError, match="no torch here"):
        small.build(force=True)
    assert os.path.exists(small.LIB) and not os.path.exists(small.CALLS)


def test_the_module_is_built_anew_for_another_torch(small, monkeypatch):
    small.build(force=True)
    assert small.up_to_date()
    first = os.stat(small.LIB).st_mtime_ns, os.stat(small.CALLS).st_mtime_ns
    small.build()
    assert first == (os.stat(small.LIB).st_mtime_ns, os.stat(small.CALLS).st_mtime_ns)
    import importlib.metadata

    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0 of another time")
    assert not small.up_to_date()
    small.build()
    assert small.up_to_date()
    assert os.stat(small.LIB).st_mtime_ns == first[0] and os.stat(small.CALLS).st_mtime_ns > first[1]


def test_a_module_that_does_not_load_is_not_called_missing(small, monkeypatch):
    import affine_bit_matmul_gb300 as mxq

    def fails(name, package=None):
        raise ImportError("undefined symbol: of_another_torch")

    monkeypatch.setattr(mxq, "_calls_module", None)
    monkeypatch.setattr(mxq, "lib", lambda: None)
    monkeypatch.setattr(mxq.importlib, "import_module", fails)
    with pytest.raises(RuntimeError, match="undefined symbol: of_another_torch"):
        mxq._direct()
